"""The 4-bit decode where every CTA has many chunks and several units: each stage of its ring is used many times, whole
units lie between parts at both ends of a CTA's share.  Every row is compared with a plain float64 computation on the GPU,
one unit of each case with the CPU oracle.

The values are not negative, and a key of chunk c (128 keys) has one in the value dimensions d = c (mod Ev) only: output d
is then the weight of the chunks d, d + Ev, ... times their values, so that a chunk that is missing, repeated or another
one's shows in full, and the tolerance is relative to the output itself."""

import numpy as np
import pytest
import torch

import attention_tiled_attn_b200 as attn
from oracle import kv4 as orc4

import kv4_util as ku

pytestmark = pytest.mark.gpu

CHUNK = 128


@pytest.fixture(scope="module", autouse=True)
def _cuda_ready():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from attention_tiled_attn_b200 import build as b
    b.build()
    yield
    assert attn.device_status() == 0


def coded_cache(g, N, H, C, E, Ev):
    """Arbitrary K elements under scales between 2^-3 and 1; V as described above."""
    def of(lo, hi, w):
        return torch.randint(lo, hi, (N, H, C, w), dtype=torch.uint8, device="cuda", generator=g)
    cache = attn.KV4Cache(of(0, 256, E // 2), of(96, 121, E // 16), of(1, 8, Ev // 2), of(96, 121, Ev // 16))
    dim = torch.arange(C, device="cuda") // CHUNK % Ev
    here = torch.arange(Ev // 2, device="cuda") == (dim // 2)[:, None]
    cache.v_codes.copy_(torch.where(here, cache.v_codes << (4 * (dim % 2))[:, None].to(torch.uint8), torch.zeros_like(cache.v_codes)))
    return cache


def values64(codes, scales):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    x = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    s = torch.tensor(orc4.SCALES, device="cuda")[scales.long()]
    return x * s.repeat_interleave(16, -1)


def reference(q, cache, lens, scale, mode, sink, mask, window, keep):
    """(out, lse, the logits' size), float64."""
    N, Hq, L, E = q.shape
    H, Ev = cache.k_codes.shape[1], 2 * cache.v_codes.shape[3]
    out = torch.zeros((N, Hq, L, Ev), dtype=torch.float64, device="cuda")
    lse = torch.full((N, Hq, L), float("-inf"), dtype=torch.float64, device="cuda")
    size = 0.0
    for n, S in enumerate(lens):
        if S == 0:
            if sink is not None:
                lse[n] = sink.double()[:, None]
            continue
        k, v = (values64(c[n, :, :S], s[n, :, :S]) for c, s in (cache[:2], cache[2:]))
        x = q[n].double().reshape(H, Hq // H * L, E)
        z, most = scale * x @ k.mT, scale * x.abs() @ k.abs().mT
        if mode == "rbf":
            norms = scale * k.square().sum(-1)[:, None]
            z, most = 2 * z - norms, 2 * most + norms
        size = max(size, most.max().item())
        j, at = torch.arange(S, device="cuda"), (torch.arange(L, device="cuda") + S - L)[:, None]
        seen = torch.ones((L, S), dtype=torch.bool, device="cuda") if mask == "none" else j <= at
        if mask in ("window", "streaming"):
            seen &= (at - j < window) | ((j < keep) if mask == "streaming" else torch.zeros_like(j, dtype=torch.bool))
        z = z.reshape(H, Hq // H, L, S).masked_fill(~seen, float("-inf")).reshape(Hq, L, S)
        total = torch.logsumexp(z, -1)
        if sink is not None:
            total = torch.logaddexp(total, sink.double()[:, None])
        lse[n] = total
        p = torch.exp(z - total[..., None]).nan_to_num(0.0)  # rows without a key
        out[n] = (p.reshape(H, -1, S) @ v).reshape(Hq, L, Ev)
    return out, lse, size


def run(N, Hq, H, L, S, E, Ev, *, lens=None, mode="dot", sink=False, mask="none", window=0, keep=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = coded_cache(g, N, H, -(-S // 16) * 16, E, Ev)
    q = (0.4 * torch.randn(N, Hq, L, E, device="cuda", generator=g)).bfloat16()
    s = torch.randn(Hq, device="cuda", generator=g) if sink else None
    scale = E ** -0.5 * (0.3 if mode == "rbf" else 1.0)
    out, lse = attn.attn_decode_kv4(q, cache, scale=scale, length=S, kv_len=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    mode=mode, sink=s, mask_kind=mask, window=window, keep_first=keep)
    lens = [S] * N if lens is None else lens
    ref, ref_lse, size = reference(q, cache, lens, scale, mode, s, mask, window, keep)
    # Roundings: the output to bf16 (2^-8), each probability to fp16 (2^-11 of it, or 2^-32 of the largest one's where it is
    # below 2^-21 of that), logits (2^-18 of their size and 4, twice: numerator and denominator), and at most S / 32 + 64
    # additions in a row, each by 2^-23.
    adds = (S / 32 + 64) * 2.0 ** -23
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18 * (4 + size) + adds) * ref.abs() + CHUNK * 6 * 2.0 ** -32
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"out off by {(err / tol).max().item():.2f} of the tolerance at {(err / tol).flatten().argmax().item()}"
    dead = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), dead)
    lerr = (lse.double() - ref_lse)[~dead].abs()
    ltol = 2.0 ** -20 * (8 + ref_lse[~dead].abs() + size) + adds
    assert (lerr <= ltol).all(), f"lse off by {(lerr / ltol).max().item():.2f} of the tolerance"
    # the plain computation itself: one unit against the CPU oracle
    n, h = N // 2, H // 2
    heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
    k, v = (orc4.dequantise(c[n:n + 1, h:h + 1].cpu().numpy(), t[n:n + 1, h:h + 1].cpu().numpy()) for c, t in (cache[:2], cache[2:]))
    want, want_lse = orc4.attention(ku.f64(q[n:n + 1, heads]), k, v, [lens[n]], scale=scale, mode=mode,
                                    sink=None if s is None else ku.f64(s)[heads], mask_kind=mask, window=window, keep=keep)
    np.testing.assert_allclose(ku.f64(ref[n:n + 1, heads]), want, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(ku.f64(ref_lse[n:n + 1, heads]), want_lse, rtol=1e-10)


def ragged(N, most, seed, least=1):
    x = np.random.default_rng(seed).integers(least, most + 1, N).tolist()
    x[0] = most
    return x


@pytest.mark.parametrize("E,Ev", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows", [4, 16])
@pytest.mark.parametrize("mode", ["dot", "rbf"])
def test_every_form_of_the_kernel(mode, rows, E, Ev):
    """24 sequences of 16001 rows and fewer, 4 heads: about 60 chunks and unit costs a CTA, for rings of 8 to 16 stages."""
    run(24, 4 * min(rows, 8), 4, rows // min(rows, 8), 16001, E, Ev, lens=ragged(24, 16001, E + Ev), mode=mode, sink=True, mask="causal", seed=rows)


def test_long_contexts_in_a_batch():
    run(16, 32, 8, 1, 16384, 128, 128, sink=True, seed=1)


def test_a_ragged_served_batch():
    run(32, 32, 8, 1, 4096, 128, 128, lens=ragged(32, 4096, 2), sink=True, seed=2)


def test_long_windows():
    run(12, 24, 6, 2, 20000, 128, 64, lens=ragged(12, 20000, 3, 9000), mask="window", window=9001, seed=3)
    run(12, 24, 6, 4, 20000, 64, 64, lens=ragged(12, 20000, 4), mask="streaming", window=7000, keep=1500, sink=True, seed=4)


def test_more_sequences_than_threads():
    """The lengths are summed in more than one round; empty sequences between long ones."""
    lens = ragged(500, 2500, 5)
    lens[7] = lens[300] = lens[499] = 0
    run(500, 4, 2, 1, 2500, 64, 128, lens=lens, mask="causal", seed=5)


def test_one_cta_with_whole_units_between_two_parts():
    """About 7 units a CTA."""
    run(128, 8, 8, 1, 1300, 128, 128, lens=ragged(128, 1300, 6, 700), seed=6)
