"""The 4-bit cache without a GPU: the oracle's rounding against a brute-force search, exactness of
the stored values, and the refusals of the C entry points and of the binding."""

import numpy as np
import pytest
import torch

import attention_tiled_attn_b200 as attn
from attention_tiled_attn_b200 import build as attn_build
from oracle import kv4 as orc4

import kv4_util as ku


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.load_library()


def brute_nearest(grid, x):
    d = np.abs(grid - x)
    best = np.flatnonzero(d == d.min())
    return int(best[best % 2 == 0][0]) if len(best) > 1 else int(best[0])


def test_scales_are_the_upper_bits_of_fp16():
    bits = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(bits, orc4.SCALES)
    assert orc4.SCALES[226] == 10240 and 6 * orc4.SCALES[226] < np.finfo(np.float16).max
    assert np.isnan((np.array([255], dtype=np.uint16) << 7).view(np.float16)[0])


def test_every_stored_value_is_exact_in_16_bits():
    v = np.multiply.outer(orc4.SCALES, orc4.ELEMENTS)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    assert np.array_equal(ku.f64(torch.from_numpy(v).to(torch.bfloat16)), v)


def test_nearest_against_brute_force():
    rng = np.random.default_rng(0)
    mids = (orc4.SCALES[1:] + orc4.SCALES[:-1]) / 2
    xs = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, np.inf), orc4.SCALES,
                         np.exp(rng.uniform(-14, 11, 500)), [0.0, 1e9]])
    assert [brute_nearest(orc4.SCALES, x) for x in xs] == orc4.nearest(orc4.SCALES, xs).tolist()
    mids = (orc4.ELEMENTS[1:] + orc4.ELEMENTS[:-1]) / 2
    xs = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 9), orc4.ELEMENTS, rng.uniform(0, 8, 500)])
    assert [brute_nearest(orc4.ELEMENTS, x) for x in xs] == orc4.nearest(orc4.ELEMENTS, xs).tolist()


def test_rounding_a_row_by_hand():
    x = np.zeros(32)
    x[:4] = [6.0, -1.25, 0.75, 5.0]      # scale 1: 6, -1 (tie to even), 1 (tie to even), 4 (tie to even)
    x[16:18] = [np.nan, 3.0]             # a block with a NaN
    codes, scales = orc4.quantise(x)
    assert scales.tolist() == [15 << 3, 255]
    got = orc4.dequantise(codes, scales)
    assert got[:4].tolist() == [6.0, -1.0, 1.0, 4.0] and np.all(got[4:16] == 0)
    assert np.isnan(got[16:]).all()
    codes, scales = orc4.quantise(np.full(16, 1e30))
    assert scales[0] == 226 and np.all(orc4.dequantise(codes, scales) == 61440)


def test_rounding_error_is_at_most_a_half_step():
    rng = np.random.default_rng(1)
    x = ku.f64(ku.random_rows(rng, (200, 64)))
    codes, scales = orc4.quantise(x)
    y = orc4.dequantise(codes, scales)
    s = np.repeat(orc4.SCALES[scales], 16, -1)
    # half of the widest step (4 to 6) is 1 s; max|x| / 6 is at most 1 + 2^-4 above s, so saturation loses at most 6 s / 16
    assert np.all(np.abs(x - y) <= s * (1 + 2 ** -52))


P = 0x10000  # a 16-byte aligned fake device address; never dereferenced on the error paths


def call_write(**kw):
    a = dict(k=P, v=P, kc=P, ks=P, vc=P, vs=P, N=2, H=2, L=3, C=32, E=64, Ev=64, kst=(384, 192, 64), vst=(384, 192, 64),
             start=0, pos=None, count=None, dtype=0)
    a.update(kw)
    return attn.attn_kv4_write_raw(a["k"], a["v"], a["kc"], a["ks"], a["vc"], a["vs"], a["N"], a["H"], a["L"], a["C"],
                                   a["E"], a["Ev"], a["kst"], a["vst"], a["start"], a["pos"], a["count"], a["dtype"],
                                   None)


def call_read(**kw):
    a = dict(kc=P, ks=P, vc=P, vs=P, k=P, v=P, N=2, H=2, rows=3, C=32, E=64, Ev=64, start=0, pos=None, kv_len=None,
             dtype=0)
    a.update(kw)
    return attn.attn_kv4_read_raw(a["kc"], a["ks"], a["vc"], a["vs"], a["k"], a["v"], a["N"], a["H"], a["rows"], a["C"],
                                  a["E"], a["Ev"], a["start"], a["pos"], a["kv_len"], a["dtype"], None)


def call_decode(**kw):
    a = dict(q=P, kc=P, ks=P, vc=P, vs=P, out=P, lse=P, N=1, Hq=2 * max(1, kw.get("H", 1)), H=1, L=1, S=20, C=32, E=64, Ev=64, scale=0.125,
             mode=0, sink=None, mask_kind=0, window=0, keep=0, kv_len=None, ws=P,
             ws_bytes=attn.load_library().attn_decode_kv4_workspace_bytes())
    a.update(kw)
    return attn.attn_decode_kv4_raw(a["q"], a["kc"], a["ks"], a["vc"], a["vs"], a["out"], a["lse"], a["N"], a["Hq"],
                                    a["H"], a["L"], a["S"], a["C"], a["E"], a["Ev"], a["scale"], a["mode"], a["sink"],
                                    a["mask_kind"], a["window"], a["keep"], a["kv_len"], a["ws"], a["ws_bytes"], None)


COMMON = [
    (dict(kc=None), -1), (dict(ks=None), -1), (dict(vc=None), -1), (dict(vs=None), -1),
    (dict(N=0), -2), (dict(H=-1), -2), (dict(N=1 << 16, H=1 << 15), -2),
    (dict(E=96), -4), (dict(Ev=16), -4),
    (dict(C=0), -19), (dict(C=40), -19), (dict(C=-16), -19),
    (dict(kc=P + 8), -11), (dict(ks=P + 4), -11), (dict(vc=P + 8), -11), (dict(vs=P + 1), -11),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(L=0), -2), (dict(N=1 << 10, H=1 << 10, L=1 << 12), -2),
    (dict(dtype=2), -10), (dict(dtype=-1), -10),
    (dict(k=P + 2), -11), (dict(v=P + 8), -11), (dict(pos=P + 2), -11), (dict(count=P + 1), -11),
    (dict(kst=(384, 192, 68)), -11), (dict(vst=(384, 196, 64)), -11), (dict(kst=(388, 192, 64)), -11),
    (dict(dtype=1, vst=(384, 192, 66)), -11),
])
def test_write_refusals(lib, kw, status):
    assert call_write(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(rows=0), -2), (dict(N=1 << 10, H=1 << 10, rows=1 << 12), -2),
    (dict(dtype=2), -10), (dict(k=P + 8), -11), (dict(v=P + 4), -11), (dict(pos=P + 2), -11), (dict(kv_len=P + 3), -11),
])
def test_read_refusals(lib, kw, status):
    assert call_read(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(L=0), -2), (dict(S=0), -2),
    (dict(S=33), -19), (dict(Hq=3, H=2), -3), (dict(scale=0.0), -5), (dict(scale=float("nan")), -5),
    (dict(mode=3), -6), (dict(mode=2), -9), (dict(mask_kind=3), -7), (dict(mask_kind=2, window=0), -8),
    (dict(keep=-1, mask_kind=2, window=1), -18), (dict(keep=4), -18), (dict(keep=4, mask_kind=1), -18),
    (dict(Hq=17), -17), (dict(Hq=4, L=5), -17), (dict(q=P + 8), -11), (dict(lse=P + 2), -11), (dict(sink=P + 2), -11),
    (dict(kv_len=P + 2), -11), (dict(ws=P + 8), -11), (dict(ws_bytes=0), -20),
    (dict(N=1 << 20, C=1 << 24, S=5), -2),
])
def test_decode_refusals(lib, kw, status):
    assert call_decode(**kw) == status


@pytest.mark.parametrize("N", [(1 << 30) - 1, 1 << 29])
def test_decode_refuses_more_small_sequences_than_it_numbers(lib, N):
    # a sequence of one chunk takes 5 positions of the 32-bit work list
    assert call_decode(N=N, Hq=1, S=16, C=16) == -2


def test_status_texts(lib):
    for st in (-19, -20):
        assert attn.status_string(st) != "unknown status"


def test_binding_refuses_tensors_off_the_gpu():
    cache = tuple(torch.zeros((1, 1, 16, w), dtype=torch.uint8) for w in (32, 4, 32, 4))
    k = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.attn_kv4_write(cache, k, k)
    with pytest.raises(ValueError):
        attn.attn_kv4_read(cache, 2)
    with pytest.raises(ValueError):
        attn.attn_decode_kv4(k, cache, scale=1.0)
    with pytest.raises(ValueError):
        attn.attn_decode_kv4(k, cache, scale=1.0, mask_kind="diagonal")
    with pytest.raises(ValueError):
        attn.attn_decode_kv4(k, cache, scale=1.0, keep_first=3)


def test_kv4_cache_rounds_the_capacity_up():
    c = attn.kv4_cache(2, 3, 17, 64, 128, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 3, 32, 32), (2, 3, 32, 4), (2, 3, 32, 64), (2, 3, 32, 8)]
    assert all(t.dtype == torch.uint8 and not t.any() for t in c)
