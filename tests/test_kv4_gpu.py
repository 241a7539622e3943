"""The 4-bit cache on the GPU: what is written is the oracle's rounding byte for byte, what is read
back is exact, and the decode matches the float64 oracle on the values the cache stands for."""

import numpy as np
import pytest
import torch

import attention_tiled_attn_b200 as attn
from oracle import kv4 as orc4

import kv4_util as ku

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda_ready():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from attention_tiled_attn_b200 import build as b
    b.build()
    yield
    assert attn.device_status() == 0


def to_gpu(cache):
    return attn.KV4Cache(*(t.cuda() for t in cache))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(N, H, C, E, Ev, seed=7):
    """A cache of arbitrary bytes, NaN scales among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return attn.KV4Cache(*(torch.randint(0, 256, (N, H, C, w), dtype=torch.uint8, device="cuda", generator=g)
                           for w in (E // 2, E // 16, Ev // 2, Ev // 16)))


def stored_values(codes, scales):
    return orc4.dequantise(codes.cpu().numpy(), scales.cpu().numpy())


def check_stored(codes, scales, x):
    """Cache rows hold the oracle's rounding of x: the same scale bytes and the same values (either zero)."""
    want_c, want_s = orc4.quantise(ku.f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(stored_values(codes, scales), orc4.dequantise(want_c, want_s))


# ------------------------------------------------------------------ writing

def hard_rows(rng, rows, E, dtype):
    """Rows whose blocks hit the roundings' borders: exact ties of scales and elements, zeros, the
    smallest and largest values, infinities and NaN."""
    x = rng.standard_normal((rows, E)) * np.exp(3 * rng.standard_normal((rows, 1)))
    b = x.reshape(-1, 16)
    n = len(b)
    mids = (orc4.SCALES[1:] + orc4.SCALES[:-1]) / 2
    for i in range(0, n, 4):  # largest value exactly 6 x a midpoint of two scales
        b[i] = np.clip(b[i], -1, 1) * 1e-3
        b[i, rng.integers(16)] = 6 * mids[rng.integers(len(mids))]
    em = (orc4.ELEMENTS[1:] + orc4.ELEMENTS[:-1]) / 2
    for i in range(1, n, 4):  # the largest element 6 s, the others midpoints times s
        s = orc4.SCALES[rng.integers(1, 227)]
        b[i] = s * em[rng.integers(0, 7, 16)] * rng.choice([-1, 1], 16)
        b[i, 0] = 6 * s
    special = [0.0, -0.0, 2.0 ** -18 * 6, 2.0 ** -19 * 6, 1e-30, 61440.0, 65504.0, 1e30, np.inf, -np.inf, np.nan]
    for k, v in enumerate(special):
        if 4 * k + 2 < n:
            b[4 * k + 2, rng.integers(16)] = v
            if v == v and abs(v) < 1e-4:
                b[4 * k + 2] = v * rng.uniform(-1, 1, 16)
                b[4 * k + 2, 3] = v
    return torch.as_tensor(b.reshape(rows, E).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,Ev", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_written_bytes_are_the_oracles(E, Ev, dtype):
    rng = np.random.default_rng(E + Ev)
    N, H, L = 2, 3, 37
    k = hard_rows(rng, N * H * L, E, dtype).reshape(N, H, L, E).cuda()
    v = hard_rows(rng, N * H * L, Ev, dtype).reshape(N, H, L, Ev).cuda()
    cache = filled(N, H, 48, E, Ev)
    attn.attn_kv4_write(cache, k, v)
    check_stored(cache.k_codes[:, :, :L], cache.k_scales[:, :, :L], k)
    check_stored(cache.v_codes[:, :, :L], cache.v_scales[:, :, :L], v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_written_bytes_over_many_random_rows(dtype):
    """Two million values of every size: the rounding decisions are exact, so none may differ."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 1, 8192, 128)) * np.exp(2 * rng.standard_normal((1, 1, 8192, 1)))
    k = torch.as_tensor(x.astype(np.float32)).to(dtype).cuda()
    v = torch.as_tensor(np.roll(x, 5, -2).astype(np.float32) * 1.7).to(dtype).cuda()
    cache = attn.kv4_cache(1, 1, 8192, 128)
    attn.attn_kv4_write(cache, k, v)
    check_stored(cache.k_codes, cache.k_scales, k)
    check_stored(cache.v_codes, cache.v_scales, v)


@pytest.mark.parametrize("L", [1, 2, 17, 100])
def test_only_the_given_rows_change(L):
    """Ragged positions and counts, some before, after or across the cache's ends."""
    rng = np.random.default_rng(L)
    N, H, C, E, Ev = 7, 2, 64, 128, 64
    pos = [0, 5, 63, 64, -3, 60, -200]
    count = [L, 0, L, L, L, max(1, L // 2), -1]
    k, v = ku.random_rows(rng, (N, H, L, E)).cuda(), ku.random_rows(rng, (N, H, L, Ev)).cuda()
    cache = filled(N, H, C, E, Ev)
    before = [t.cpu().numpy().copy() for t in cache]
    attn.attn_kv4_write(cache, k, v, pos=ints(pos), count=ints(count))
    kq, vq = orc4.quantise(ku.f64(k)), orc4.quantise(ku.f64(v))
    for got, old, new in zip(cache, before, (*kq, *vq)):
        want = old.copy()
        for n in range(N):
            for l in range(min(L, max(0, count[n]))):
                if 0 <= pos[n] + l < C:
                    want[n, :, pos[n] + l] = new[n, :, l]
        got = got.cpu().numpy()
        touched = np.zeros((N, C), bool)
        for n in range(N):
            for l in range(min(L, max(0, count[n]))):
                if 0 <= pos[n] + l < C:
                    touched[n, pos[n] + l] = True
        rows = np.broadcast_to(touched[:, None, :, None], got.shape)
        assert np.array_equal(got[~rows], want[~rows]), "a byte outside the written rows changed"
        zero = lambda a: np.where((a & 0x0F) == 8, a & 0xF0, a)  # noqa: E731  (either zero)
        if got.shape[-1] >= 32:
            a, b = zero(got[rows]), zero(want[rows])
            a, b = np.where((a & 0xF0) == 0x80, a & 0x0F, a), np.where((b & 0xF0) == 0x80, b & 0x0F, b)
            assert np.array_equal(a, b)
        else:
            assert np.array_equal(got[rows], want[rows])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_repeated_sources(dtype):
    rng = np.random.default_rng(3)
    N, H, L, E, Ev = 3, 2, 19, 64, 128
    both = ku.random_rows(rng, (N, L, 2 * H, E + Ev), dtype).cuda()  # a projection with more than K and V in it
    k, v = both[:, :, :H, :E].transpose(1, 2), both[:, :, H:, E:].transpose(1, 2)
    assert not k.is_contiguous()
    a, b = attn.kv4_cache(N, H, 32, E, Ev), attn.kv4_cache(N, H, 32, E, Ev)
    attn.attn_kv4_write(a, k, v, start=4)
    attn.attn_kv4_write(b, k.contiguous(), v.contiguous(), start=4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    check_stored(a.k_codes[:, :, 4:4 + L], a.k_scales[:, :, 4:4 + L], k)
    # one row for every head and position
    k1, v1 = k[:, :1, :1].expand(N, H, L, E), v[:, :1, :1].expand(N, H, L, Ev)
    attn.attn_kv4_write(a, k1, v1)
    check_stored(a.v_codes[:, :, :L], a.v_scales[:, :, :L], v1)


@pytest.mark.parametrize("E,Ev,dtype", [(128, 128, torch.bfloat16), (64, 128, torch.bfloat16), (128, 64, torch.float32)])
@pytest.mark.parametrize("shift", [0, 1])
def test_many_ragged_rows(E, Ev, dtype, shift):
    """Enough rows for the kernels' wider forms: tiles that end inside a unit, sequences cut by count and by the cache's
    end, sources and outputs aligned to 16 bytes only (shift), and every other byte of the cache as it was."""
    rng = np.random.default_rng(E + shift)
    N, H, L, C = 7, 3, 901, 912
    per16 = 128 // torch.finfo(dtype).bits  # values in 16 bytes
    k, v = (ku.random_rows(rng, (N, H, L, w), dtype).cuda() for w in (E, Ev))
    if shift:
        def shifted(t):
            flat = torch.empty(t.numel() + per16, dtype=t.dtype, device="cuda")
            flat[per16:] = t.reshape(-1)
            return flat[per16:].view(t.shape)
        k, v = shifted(k), shifted(v)
    pos, count = [0, 3, 11, 100, -7, 0, 905], [901, 900, 901, 901, 901, 450, 901]
    cache = filled(N, H, C, E, Ev)
    before = [t.clone() for t in cache]
    attn.attn_kv4_write(cache, k, v, pos=ints(pos), count=ints(count))
    lens = [max(0, min(C, p + c)) for p, c in zip(pos, count)]
    kout, vout = (torch.full((N * H * 905 * w + per16,), 7.0, dtype=dtype, device="cuda")[shift * per16:][:N * H * 905 * w].view(N, H, 905, w)
                  for w in (E, Ev))
    attn.attn_kv4_read(cache, 905, start=5, kv_len=ints(lens), dtype=dtype, k_out=kout, v_out=vout)
    for src, got, codes, scales, old_c, old_s in ((k, kout, *cache[:2], *before[:2]), (v, vout, *cache[2:], *before[2:])):
        for n in range(N):
            a, b = max(0, pos[n]), lens[n]  # cache rows written
            check_stored(codes[n, :, a:b], scales[n, :, a:b], src[n, :, a - pos[n]:b - pos[n]])
            for t, old in ((codes, old_c), (scales, old_s)):
                assert torch.equal(t[n, :, :a], old[n, :, :a]) and torch.equal(t[n, :, b:], old[n, :, b:])
            want = np.zeros((H, 905, got.shape[-1]))
            end = min(910, b)
            if end > 5:
                want[:, :end - 5] = stored_values(codes[n, :, 5:end], scales[n, :, 5:end])
            # what filled() left before the first written row may have scales that no write leaves (infinite values)
            first = max(0, a - 5)
            np.testing.assert_array_equal(ku.f64(got[n, :, first:]), want[:, first:])


# ------------------------------------------------------------------ reading

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,Ev", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_every_byte_reads_back_exactly(E, Ev, dtype):
    """Every pair of a scale byte that a write leaves (and the NaN mark) and an element code."""
    C = 240
    cache = filled(1, 1, C, E, Ev)
    for codes, scales in (cache[:2], cache[2:]):
        scales.copy_((torch.arange(C, dtype=torch.uint8, device="cuda").clamp(max=226)).view(1, 1, C, 1).expand_as(scales))
        scales[:, :, 230] = 255
        codes.copy_((torch.arange(codes.shape[-1] * 16, device="cuda") * 37 % 256).to(torch.uint8).view(1, 1, 16, -1)
                    .repeat(1, 1, C // 16, 1))
    k, v = attn.attn_kv4_read(cache, C, dtype=dtype)
    assert k.dtype == dtype and k.shape == (1, 1, C, E) and v.shape == (1, 1, C, Ev)
    np.testing.assert_array_equal(ku.f64(k), stored_values(*cache[:2]))
    np.testing.assert_array_equal(ku.f64(v), stored_values(*cache[2:]))


@pytest.mark.parametrize("rows", [1, 3, 16, 65])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_ranges(rows, dtype):
    N, H, C, E, Ev = 6, 3, 64, 128, 64
    rng = np.random.default_rng(rows)
    cpu, kval, vval = ku.random_cache(rng, N, H, C, E, Ev)
    cache = to_gpu(cpu)
    lens = [0, 1, 40, 64, 1000, -5]
    pos = [0, 0, 37, 60, -2, 3]
    for t in cache:  # what lies behind a sequence's rows does not matter
        for n in range(N):
            t[n, :, max(0, min(C, lens[n])):] = 255
    for p, start in ((pos, 0), (None, 0), (None, 33), (None, -1), (None, C - 1)):
        k, v = attn.attn_kv4_read(cache, rows, start=start, pos=None if p is None else ints(p), kv_len=ints(lens), dtype=dtype)
        for got, val in ((k, kval), (v, vval)):
            want = np.zeros(got.shape)
            for n in range(N):
                for r in range(rows):
                    j = (p[n] if p is not None else start) + r
                    if 0 <= j < min(C, lens[n]):
                        want[n, :, r] = val[n, :, j]
            np.testing.assert_array_equal(ku.f64(got), want)


def test_read_into_given_outputs():
    cache = filled(2, 1, 16, 64, 64)
    k, v = (torch.full((2, 1, 5, 64), 9.0, dtype=torch.float32, device="cuda") for _ in range(2))
    got = attn.attn_kv4_read(cache, 5, dtype=torch.float32, kv_len=ints([0, 0]), k_out=k, v_out=v)
    assert got[0] is k and got[1] is v and not k.any() and not v.any()
    with pytest.raises(ValueError):
        attn.attn_kv4_read(cache, 6, dtype=torch.float32, k_out=k)


# ------------------------------------------------------------------ attention

def run_decode(N, Hq, H, L, C, E, Ev, lens, *, mode="dot", sink=False, mask="none", window=0, keep=0, seed=0, size=1.0,
               length=None, garbage=True, what=""):
    rng = np.random.default_rng(seed)
    cpu, k, v = ku.random_cache(rng, N, H, C, E, Ev)
    q = ku.bf16(rng.standard_normal((N, Hq, L, E)) * size)
    s = rng.standard_normal(Hq).astype(np.float32) if sink else None
    cache = to_gpu(cpu)
    if garbage:  # bytes behind a sequence's rows, NaN scales among them
        noise = filled(N, H, C, E, Ev)
        for t, o in zip(cache, noise):
            for n in range(N):
                t[n, :, lens[n]:] = o[n, :, lens[n]:]
                if t.shape[-1] <= 8 and lens[n] < C:
                    t[n, :, lens[n]:] = 255
    scale = E ** -0.5
    uniform = all(x == lens[0] for x in lens)
    kw = dict(length=lens[0]) if uniform and lens[0] > 0 and length is None else dict(kv_len=ints(lens), length=length)
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=scale, mode=mode,
                                    sink=None if s is None else torch.from_numpy(s).cuda(), mask_kind=mask,
                                    window=window, keep_first=keep if mask == "streaming" else 0, **kw)
    ref = orc4.attention(ku.f64(q), k, v, lens, scale=scale, mode=mode, sink=None if s is None else s.astype(np.float64),
                         mask_kind=mask, window=window, keep=keep)
    g = Hq // H
    live = [k[n, :, :lens[n]] for n in range(N) if lens[n]]
    logits = 0.0
    for n in range(N):
        if lens[n]:
            kk = np.abs(np.repeat(k[n, :, :lens[n]], g, 0))
            logits = max(logits, float(np.einsum("hle,hse->hls", np.abs(ku.f64(q[n])), kk).max()) * scale)
            if mode == "rbf":
                logits = max(logits, 2 * logits + scale * float((kk * kk).sum(-1).max()))
    ku.compare(out, lse, *ref, v_most=max([float(np.abs(v).max())] if live else [0.0]), scale_of_logits=logits, what=what)
    return out, lse


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 300, 777]


@pytest.mark.parametrize("E,Ev", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("mode", ["dot", "rbf"])
@pytest.mark.parametrize("S", LENGTHS)
def test_decode_lengths(S, mode, E, Ev):
    run_decode(2, 6, 2, 1, -(-S // 16) * 16, E, Ev, [S, S], mode=mode, sink=S % 2 == 0, seed=S)


@pytest.mark.parametrize("group,L", [(1, 1), (2, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (1, 16), (1, 9), (4, 2), (2, 8), (5, 3)])
@pytest.mark.parametrize("mask", ["none", "causal", "window", "streaming"])
def test_decode_query_rows(group, L, mask):
    run_decode(2, 3 * group, 3, L, 320, 128, 128, [301, 77], mask=mask, window=37, keep=5, sink=L % 2 == 0, seed=group)


@pytest.mark.parametrize("mode", ["dot", "rbf"])
@pytest.mark.parametrize("mask,window,keep", [("none", 0, 0), ("causal", 0, 0), ("window", 1, 0), ("window", 100, 0),
                                             ("window", 2**31 - 1, 0), ("streaming", 1, 1), ("streaming", 100, 4),
                                             ("streaming", 64, 65), ("streaming", 130, 500), ("streaming", 7, 2**31 - 1)])
@pytest.mark.parametrize("sink", [False, True])
def test_decode_ragged_lengths(mask, window, keep, sink, mode):
    """Empty sequences, sequences shorter than the query block, and whole ones in one call."""
    lens = [0, 1, 2, 5, 16, 63, 64, 65, 200, 511, 512]
    run_decode(len(lens), 8, 4, 3, 512, 64, 64, lens, mask=mask, window=window, keep=keep, sink=sink, mode=mode,
               seed=window % 97 + keep % 89, length=512)


@pytest.mark.parametrize("E,Ev", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("mode", ["dot", "rbf"])
@pytest.mark.parametrize("group,L", [(4, 1), (9, 1), (4, 4)])
def test_decode_head_widths(group, L, mode, E, Ev):
    """Both row counts of the kernel (up to 8, up to 16 query rows) at every pair of head widths, whole and split units."""
    run_decode(2, 2 * group, 2, L, 1296, E, Ev, [1290, 530], mode=mode, mask="streaming", window=600, keep=130, sink=True, seed=E + Ev + L)


def test_decode_lengths_beyond_the_given_length():
    """kv_len is clamped to [0, length]."""
    rng = np.random.default_rng(21)
    cpu, k, v = ku.random_cache(rng, 4, 2, 96, 64, 64)
    q = ku.bf16(rng.standard_normal((4, 4, 1, 64)))
    out, lse = attn.attn_decode_kv4(q.cuda(), to_gpu(cpu), scale=0.125, length=70, kv_len=ints([70, 1000, -3, 2**31 - 1]))
    ref = orc4.attention(ku.f64(q), k, v, [70, 70, 0, 70], scale=0.125)
    ku.compare(out, lse, *ref, v_most=float(np.abs(v).max()), scale_of_logits=16.0)


def test_decode_slices_of_a_cache():
    """Part of a cache's batch (its rows are contiguous), and no lse."""
    rng = np.random.default_rng(22)
    cpu, k, v = ku.random_cache(rng, 5, 2, 80, 128, 64)
    cache = attn.KV4Cache(*(t[1:4] for t in to_gpu(cpu)))
    q = ku.bf16(rng.standard_normal((3, 4, 1, 128)))
    lens = [80, 3, 41]
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=0.09, kv_len=ints(lens))
    ref = orc4.attention(ku.f64(q), k[1:4], v[1:4], lens, scale=0.09)
    ku.compare(out, lse, *ref, v_most=float(np.abs(v).max()), scale_of_logits=16.0)
    qg, ws, out2, kv_len = q.cuda(), attn.kv4_workspace(), torch.empty_like(out), ints(lens)
    st = attn.attn_decode_kv4_raw(qg.data_ptr(), *(t.data_ptr() for t in cache), out2.data_ptr(), None, 3, 4, 2, 1, 80, 80, 128, 64,
                                  0.09, 0, None, 0, 0, 0, kv_len.data_ptr(), ws.data_ptr(), ws.nbytes,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(out, out2)


def test_decode_all_sequences_empty():
    run_decode(3, 4, 2, 1, 16, 64, 64, [0, 0, 0], length=16)
    run_decode(3, 4, 2, 1, 16, 128, 128, [0, 0, 0], length=16, sink=True)


def test_decode_many_sequences():
    """More sequences than a CTA has threads, and more units than the grid has CTAs."""
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 40, 700).tolist()
    run_decode(700, 2, 1, 1, 48, 64, 64, lens, length=40, mask="causal")


def test_decode_one_long_sequence():
    """One unit split over many CTAs."""
    run_decode(1, 4, 1, 1, 20016, 128, 128, [20001], sink=True)
    run_decode(1, 16, 1, 1, 20016, 64, 64, [19990], mask="streaming", window=9000, keep=70)


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_decode_flat_and_sharp_softmax(size):
    run_decode(2, 8, 2, 1, 1008, 128, 128, [1000, 999], size=size, mask="causal")


def test_decode_large_and_small_queries():
    """Query elements over the whole bf16 range within a row: the operand's 16-bit form keeps them."""
    rng = np.random.default_rng(2)
    cpu, k, v = ku.random_cache(rng, 1, 1, 112, 64, 64)
    q = rng.standard_normal((1, 4, 1, 64))
    q[0, 0] *= 1e-30
    q[0, 1] *= 1e4
    q[0, 2] *= np.exp(rng.uniform(-30, 0, 64))
    q[0, 3] = 0.0
    qb = ku.bf16(q)
    scale = 1e-3
    out, lse = attn.attn_decode_kv4(qb.cuda(), to_gpu(cpu), scale=scale)
    ref = orc4.attention(ku.f64(qb), k, v, [112], scale=scale)
    logits = float(np.einsum("hle,se->hls", np.abs(ku.f64(qb))[0], np.abs(k[0, 0])).max()) * scale
    ku.compare(out, lse, *ref, v_most=float(np.abs(v).max()), scale_of_logits=logits)


def test_hidden_keys_take_no_part_whatever_they_hold():
    """A block of NaN in K and V of keys that some rows see and others do not: only those that see it are NaN."""
    rng = np.random.default_rng(4)
    N, Hq, H, L, C, E, Ev, n = 1, 4, 2, 4, 160, 128, 128, 150
    cpu, k, v = ku.random_cache(rng, N, H, C, E, Ev)
    cache = to_gpu(cpu)
    q = ku.bf16(rng.standard_normal((N, Hq, L, E)))
    cache.v_scales[0, 0, n - 2, 3] = 255  # seen by the last two rows only, in value dimensions 48 to 63
    cache.k_scales[0, 1, n - 1, 0] = 255  # seen by the last row only
    cache.v_scales[0, 1, 10, 0] = 255     # outside every row's window
    cache.v_scales[0, 1, n - 4 - 49, 7] = 255  # seen by the first row only
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=E ** -0.5, length=n, mask_kind="window", window=50)
    ref, ref_lse = orc4.attention(ku.f64(q), k, v, [n], scale=E ** -0.5, mask_kind="window", window=50)
    bad = np.zeros((N, Hq, L, Ev), bool)
    bad[0, :2, 2:, 48:64] = True
    bad[0, 2:, 3, :] = True
    bad[0, 2:, 0, 112:] = True
    got = ku.f64(out)
    assert np.array_equal(np.isnan(got), bad)
    assert np.array_equal(np.isnan(ku.f64(lse)), np.arange(L)[None, None] * np.ones((1, Hq, 1)) + (np.arange(Hq) < 2)[None, :, None] * 10 == 3)
    tol = ku.REL_OUT * np.abs(ref) + 1e-2
    assert np.all(np.abs(got - ref)[~bad] <= tol[~bad])


def test_a_nan_key_that_every_row_sees():
    rng = np.random.default_rng(6)
    cpu, _, _ = ku.random_cache(rng, 1, 1, 256, 64, 64)
    cache = to_gpu(cpu)
    cache.v_scales[0, 0, 77, 1] = 255
    q = ku.bf16(rng.standard_normal((1, 2, 1, 64))).cuda()
    out, lse = attn.attn_decode_kv4(q, cache, scale=0.1)
    assert torch.isnan(out[..., 16:32]).all() and not torch.isnan(out[..., :16]).any() and torch.isfinite(lse).all()


# ------------------------------------------------------------------ together, and as a program uses them

def test_generation_with_the_cache():
    """A ragged prompt, then steps of one token: each step's output is the oracle's on all rows so far, the
    rows behind each sequence keep their bytes, and the read rows give the same through attn_fwd_padded."""
    rng = np.random.default_rng(8)
    N, Hq, H, E, Ev, C = 3, 8, 2, 64, 64, 128
    lens = [40, 1, 65]
    kp, vp = ku.random_rows(rng, (N, H, 65, E)), ku.random_rows(rng, (N, H, 65, Ev))
    cache = filled(N, H, C, E, Ev)
    behind = [t.clone() for t in cache]
    attn.attn_kv4_write(cache, kp.cuda(), vp.cuda(), count=ints(lens))
    kh, vh = np.zeros((N, H, C, E)), np.zeros((N, H, C, Ev))
    for n in range(N):
        kh[n, :, :lens[n]] = orc4.dequantise(*orc4.quantise(ku.f64(kp[n, :, :lens[n]])))
        vh[n, :, :lens[n]] = orc4.dequantise(*orc4.quantise(ku.f64(vp[n, :, :lens[n]])))
    for step in range(4):
        q = ku.bf16(rng.standard_normal((N, Hq, 1, E)))
        k1, v1 = ku.random_rows(rng, (N, H, 1, E)), ku.random_rows(rng, (N, H, 1, Ev))
        attn.attn_kv4_write(cache, k1.cuda(), v1.cuda(), pos=ints(lens))
        for n in range(N):
            kh[n, :, lens[n]:lens[n] + 1] = orc4.dequantise(*orc4.quantise(ku.f64(k1[n])))
            vh[n, :, lens[n]:lens[n] + 1] = orc4.dequantise(*orc4.quantise(ku.f64(v1[n])))
            lens[n] += 1
        out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=0.125, length=max(lens), kv_len=ints(lens), mask_kind="causal")
        ref = orc4.attention(ku.f64(q), kh, vh, lens, scale=0.125)
        ku.compare(out, lse, *ref, v_most=float(np.abs(vh).max()), scale_of_logits=8.0, what=f"step {step}")
    for t, old in zip(cache, behind):
        for n in range(N):
            assert torch.equal(t[n, :, lens[n]:], old[n, :, lens[n]:])
    # the cached rows as bf16 through the forward with key padding: the same attention
    S = max(lens)
    k, v = attn.attn_kv4_read(cache, S, kv_len=ints(lens))
    np.testing.assert_array_equal(ku.f64(k), np.where(np.arange(S)[None, None, :, None] < np.array(lens)[:, None, None, None], kh[:, :, :S], 0))
    out2, lse2 = attn.attn_fwd(q.cuda(), k, v, scale=0.125, kv_end=ints(lens))
    assert (lse2 - lse).abs().max() < 1e-4
    # two bf16 results of one value: a rounding each, and the forward's bf16 probabilities (2^-8 of max|v|)
    assert np.all(np.abs(ku.f64(out) - ku.f64(out2)) <= 2 * ku.REL_OUT * np.abs(ku.f64(out)) + (2.0 ** -8 + 2.0 ** -10) * np.abs(vh).max())


def make_call(rng, N=2, Hq=8, H=2, S=1500, E=128, Ev=128):
    cpu, k, v = ku.random_cache(rng, N, H, -(-S // 16) * 16, E, Ev)
    q = ku.bf16(rng.standard_normal((N, Hq, 1, E)))
    return q.cuda(), to_gpu(cpu), (ku.f64(q), k, v, [S] * N)


def check_call(out, lse, ref_args, scale):
    ref = orc4.attention(*ref_args, scale=scale)
    ku.compare(out, lse, *ref, v_most=float(np.abs(ref_args[2]).max()), scale_of_logits=16.0)


def test_the_same_call_twice_gives_the_same_bits():
    rng = np.random.default_rng(12)
    q, cache, _ = make_call(rng, S=5000)
    a = [attn.attn_decode_kv4(q, cache, scale=0.09, length=5000) for _ in range(4)]
    for out, lse in a[1:]:
        assert torch.equal(out, a[0][0]) and torch.equal(lse, a[0][1])


def test_calls_on_two_streams_overlap():
    """Each stream has a workspace of its own: calls in flight together do not mix."""
    rng = np.random.default_rng(13)
    calls = [make_call(rng, S=3000) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            q, cache, _ = calls[i]
            got[i].append(attn.attn_decode_kv4(q, cache, scale=0.09, length=3000, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i][:2] + got[i][-2:]:
            check_call(out, lse, calls[i][2], 0.09)
        assert all(torch.equal(o, got[i][0][0]) for o, _ in got[i])


def test_a_whole_step_on_a_stream_that_is_not_current():
    rng = np.random.default_rng(31)
    cpu, kh, vh = ku.random_cache(rng, 2, 2, 208, 64, 64)
    cache = to_gpu(cpu)
    q = ku.bf16(rng.standard_normal((2, 4, 1, 64)))
    k1, v1 = ku.random_rows(rng, (2, 2, 1, 64)), ku.random_rows(rng, (2, 2, 1, 64))
    args = q.cuda(), k1.cuda(), v1.cuda(), ints([200, 17])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn.attn_kv4_write(cache, args[1], args[2], pos=ints([199, 16]), stream=side)
    out, lse = attn.attn_decode_kv4(args[0], cache, scale=0.125, length=200, kv_len=args[3], stream=side)
    kb, vb = attn.attn_kv4_read(cache, 200, kv_len=args[3], stream=side)
    side.synchronize()
    for n, p in enumerate((199, 16)):
        kh[n, :, p], vh[n, :, p] = (orc4.dequantise(*orc4.quantise(ku.f64(x[n, :, 0]))) for x in (k1, v1))
    ref = orc4.attention(ku.f64(q), kh, vh, [200, 17], scale=0.125)
    ku.compare(out, lse, *ref, v_most=float(np.abs(vh).max()), scale_of_logits=16.0)
    np.testing.assert_array_equal(ku.f64(kb[1, :, :17]), kh[1, :, :17])
    assert not vb[1, :, 17:].any()


def test_many_steps_without_waiting_for_the_gpu():
    """Steps enqueued one after another, each reading what the one before it and the torch operations between them wrote:
    the rows, the lengths (advanced on the device) and the queries, all in buffers that are used again."""
    rng = np.random.default_rng(33)
    N, Hq, H, E, steps = 2, 4, 2, 64, 60
    start = [100, 3]
    cpu, kh, vh = ku.random_cache(rng, N, H, 176, E, E)
    cache = to_gpu(cpu)
    qs = ku.bf16(rng.standard_normal((steps, N, Hq, 1, E)))
    ks, vs = ku.random_rows(rng, (steps, N, H, 1, E)), ku.random_rows(rng, (steps, N, H, 1, E))
    qg, kg, vg = qs.cuda(), ks.cuda(), vs.cuda()
    q, k, v, lens, pos = torch.empty_like(qg[0]), torch.empty_like(kg[0]), torch.empty_like(vg[0]), ints(start), ints(start)
    outs, backs = [], []
    torch.cuda.synchronize()
    for i in range(steps):
        q.copy_(qg[i])
        k.copy_(kg[i])
        v.copy_(vg[i])
        attn.attn_kv4_write(cache, k, v, pos=pos)
        lens.add_(1)
        outs.append(attn.attn_decode_kv4(q, cache, scale=0.125, length=176, kv_len=lens, mask_kind="causal"))
        backs.append(attn.attn_kv4_read(cache, 1, pos=pos, kv_len=lens, dtype=torch.float32))
        pos.add_(1)
    torch.cuda.synchronize()
    for i in range(steps):
        n_now = [s + i + 1 for s in start]
        new_k, new_v = (orc4.dequantise(*orc4.quantise(ku.f64(x[i]))) for x in (ks, vs))
        for n in range(N):
            kh[n, :, n_now[n] - 1:n_now[n]], vh[n, :, n_now[n] - 1:n_now[n]] = new_k[n], new_v[n]
        np.testing.assert_array_equal(ku.f64(backs[i][0]), new_k)
        np.testing.assert_array_equal(ku.f64(backs[i][1]), new_v)
        ref = orc4.attention(ku.f64(qs[i]), kh, vh, n_now, scale=0.125)
        ku.compare(*outs[i], *ref, v_most=float(np.abs(vh).max()), scale_of_logits=16.0, what=f"step {i}")


def test_a_query_row_that_is_not_finite():
    """Only its own row is lost."""
    rng = np.random.default_rng(32)
    cpu, k, v = ku.random_cache(rng, 1, 1, 304, 128, 128)
    q = ku.bf16(rng.standard_normal((1, 6, 1, 128)))
    bad = q.clone()
    bad[0, 1, 0, 5] = float("nan")
    bad[0, 4, 0, 7] = float("inf")
    out, lse = attn.attn_decode_kv4(bad.cuda(), to_gpu(cpu), scale=0.09, length=300)
    ref, ref_lse = orc4.attention(ku.f64(q), k, v, [300], scale=0.09)
    ok = [0, 2, 3, 5]
    ku.compare(out[:, ok], lse[:, ok], ref[:, ok], ref_lse[:, ok], v_most=float(np.abs(v).max()), scale_of_logits=16.0)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 4]).all()


def test_captured_step_replays_on_new_inputs():
    """One step (append, attend) captured, replayed after its inputs and lengths changed, beside eager calls."""
    rng = np.random.default_rng(14)
    q, cache, ref = make_call(rng, N=2, S=700)
    k1, v1 = (ku.random_rows(rng, (2, 2, 1, 128)).cuda() for _ in range(2))
    lens, pos = ints([600, 33]), ints([599, 32])

    def step():
        attn.attn_kv4_write(cache, k1, v1, pos=pos)
        return attn.attn_decode_kv4(q, cache, scale=0.09, length=704, kv_len=lens, mask_kind="causal")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    for turn in range(3):
        n = [650 + turn, 40 + turn]
        q.copy_(ku.bf16(rng.standard_normal(q.shape)))
        k1.copy_(ku.random_rows(rng, k1.shape))
        v1.copy_(ku.random_rows(rng, v1.shape))
        lens.copy_(ints(n))
        pos.copy_(ints([x - 1 for x in n]))
        for g, _ in graphs:
            g.replay()
        eager = step()
        torch.cuda.synchronize()
        k, v = stored_values(*cache[:2]), stored_values(*cache[2:])
        want = orc4.attention(ku.f64(q), k, v, n, scale=0.09)
        for out, lse in (graphs[0][1], graphs[1][1], eager):
            ku.compare(out, lse, *want, v_most=float(np.abs(v).max()), scale_of_logits=16.0, what=f"turn {turn}")
    # both graphs at once on two streams
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], eager[0]) and torch.equal(graphs[1][1][0], eager[0])


def test_workspace_of_the_callers_own():
    rng = np.random.default_rng(15)
    ws = attn.kv4_workspace()
    for S in (2000, 64, 5000):
        q, cache, ref = make_call(rng, S=S)
        out, lse = torch.empty((2, 8, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 8, 1), device="cuda")
        got = attn.attn_decode_kv4(q, cache, scale=0.09, length=S, workspace=ws, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        check_call(out, lse, ref, 0.09)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_decode_kv4(q, cache, scale=0.09, workspace=ws[:1024])
    assert e.value.status == -20


def test_offsets_past_32_bits():
    """Rows whose byte offsets in the cache pass 2^32: written, read back and attended to."""
    rng = np.random.default_rng(16)
    C, E = 16 * 4_200_000, 128  # 67.2 million rows of 64 bytes
    cache = attn.KV4Cache(*(torch.empty((1, 1, C, w), dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)))
    L = 100
    k, v = ku.random_rows(rng, (1, 1, L, E)), ku.random_rows(rng, (1, 1, L, E))
    attn.attn_kv4_write(cache, k.cuda(), v.cuda(), start=C - L)
    kb, vb = attn.attn_kv4_read(cache, L, start=C - L)
    kq, vq = (orc4.dequantise(*orc4.quantise(ku.f64(x))) for x in (k, v))
    np.testing.assert_array_equal(ku.f64(kb), kq)
    np.testing.assert_array_equal(ku.f64(vb), vq)
    q = ku.bf16(rng.standard_normal((1, 2, 2, E)))
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=0.1, mask_kind="window", window=L - 1)
    ref = orc4.attention(ku.f64(q), kq, vq, [L], scale=0.1, mask_kind="window", window=L - 1)
    ku.compare(out, lse, *ref, v_most=float(np.abs(vq).max()), scale_of_logits=16.0)
    # and with kept first keys: the chunks between them and the window are not read
    kf, vf = ku.random_rows(rng, (1, 1, 3, E)), ku.random_rows(rng, (1, 1, 3, E))
    attn.attn_kv4_write(cache, kf.cuda(), vf.cuda())
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=0.1, mask_kind="streaming", window=L - 1, keep_first=3)
    kq, vq = (np.concatenate([orc4.dequantise(*orc4.quantise(ku.f64(x))), y], 2) for x, y in ((kf, kq), (vf, vq)))
    ref = orc4.attention(ku.f64(q), kq, vq, [L + 3], scale=0.1, mask_kind="streaming", window=L - 1, keep=3)
    ku.compare(out, lse, *ref, v_most=float(np.abs(vq).max()), scale_of_logits=16.0)


def test_a_prompt_piece_attends_through_the_read_rows():
    """Prompt pieces longer than a decode call: each piece is written, the rows so far come back in bf16 and go through
    the causal forward."""
    rng = np.random.default_rng(23)
    N, Hq, H, E, C = 2, 4, 2, 64, 224
    cache = attn.kv4_cache(N, H, C, E)
    k, v = ku.random_rows(rng, (N, H, 200, E)), ku.random_rows(rng, (N, H, 200, E))
    kq, vq = (orc4.dequantise(*orc4.quantise(ku.f64(x))) for x in (k, v))
    done = 0
    for piece in (130, 70):
        q = ku.bf16(rng.standard_normal((N, Hq, piece, E)))
        attn.attn_kv4_write(cache, k[:, :, done:done + piece].cuda(), v[:, :, done:done + piece].cuda(), start=done)
        done += piece
        kb, vb = attn.attn_kv4_read(cache, done)
        out, lse = attn.attn_fwd(q.cuda(), kb, vb, scale=0.125, mask_kind="causal")
        ref, ref_lse = orc4.attention(ku.f64(q), kq, vq, [done] * N, scale=0.125, mask_kind="causal")
        err = np.linalg.norm(ku.f64(out) - ref) / np.linalg.norm(ref)
        # two bf16 roundings (P and the output), each at most 2^-8 of its value and on average well under half of that
        assert err <= 2.0 ** -8 and np.abs(ku.f64(lse) - ref_lse).max() <= 1e-3


def test_binding_refusals():
    cache = attn.kv4_cache(2, 2, 32, 64)
    k = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: attn.attn_kv4_write(cache, k.half(), k.half()),
        lambda: attn.attn_kv4_write(cache, k, k.float()),
        lambda: attn.attn_kv4_write(cache, k[..., :32], k),
        lambda: attn.attn_kv4_write(cache, k.cpu(), k),
        lambda: attn.attn_kv4_write(cache, k[:1], k[:1]),
        lambda: attn.attn_kv4_write(cache, k, k, pos=ints([0])),
        lambda: attn.attn_kv4_write(cache, k, k, pos=torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: attn.attn_kv4_write(cache, k, k, count=torch.zeros(2, dtype=torch.int32)),
        lambda: attn.attn_kv4_write(cache, k, k, start=2**31),
        lambda: attn.attn_kv4_write(cache, k.transpose(2, 3).contiguous().transpose(2, 3), k),
        lambda: attn.attn_kv4_write(cache[:2] + (cache[2][..., :16], cache[3]), k, k),
        lambda: attn.attn_kv4_read(cache, 3, dtype=torch.float16),
        lambda: attn.attn_kv4_read(cache, 3, kv_len=ints([1, 2, 3])),
        lambda: attn.attn_decode_kv4(q.float(), cache, scale=1.0),
        lambda: attn.attn_decode_kv4(q[:1], cache, scale=1.0),
        lambda: attn.attn_decode_kv4(q.repeat(1, 1, 1, 2)[..., ::2], cache, scale=1.0),
        lambda: attn.attn_decode_kv4(q, cache, scale=1.0, kv_len=ints([1])),
        lambda: attn.attn_decode_kv4(q, cache, scale=1.0, sink=torch.zeros(3, device="cuda")),
        lambda: attn.attn_decode_kv4(q, cache, scale=1.0, mask_kind="window", window=2**40),
        lambda: attn.attn_decode_kv4(q, cache, scale=1.0, out=torch.zeros((2, 4, 1, 64), device="cuda")),
        lambda: attn.attn_decode_kv4(q, cache, scale=1.0, workspace=torch.zeros(10)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    for f, status in (
            (lambda: attn.attn_kv4_write(cache, k[:, :, :0], k[:, :, :0]), -2),
            (lambda: attn.attn_kv4_read(cache, 0), -2),
            (lambda: attn.attn_decode_kv4(q, cache, scale=1.0, length=33), -19),
            (lambda: attn.attn_decode_kv4(q, cache, scale=1.0, length=0), -2),
            (lambda: attn.attn_decode_kv4(q, cache, scale=1.0, mode="sink"), -9),
            (lambda: attn.attn_decode_kv4(q.repeat(1, 9, 1, 1), cache, scale=1.0), -17)):
        with pytest.raises(attn.AttnError) as e:
            f()
        assert e.value.status == status
