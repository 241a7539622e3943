"""The 4-bit cache's decode where the logits are large: finite ones give a softmax as small ones do."""

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


def check_one_hot(out, lse, z, v, group, shift=0.0):
    """z (H, R, S) logits in float64, v (H, S, Ev).  An fp32 logit is off by at most 2^-18 of the largest sum of products
    (128 of them, each rounded to 2^-24); where the best key leads by more than that and 40, every other key's weight is
    below e^-40 of it and the output is its value row, which bf16 holds exactly; the lse is its logit."""
    H, R, S = z.shape
    order = np.argsort(z, -1)
    best = order[..., -1]
    top = np.take_along_axis(z, best[..., None], -1)[..., 0]
    second = np.take_along_axis(z, order[..., -2:-1], -1)[..., 0]
    size = np.abs(z).max(-1) + shift
    clear = top - second > 40 + 2.0 ** -17 * size
    assert clear.mean() > 0.6, "the inputs are to have a clear best key in most rows"
    out, lse = ku.f64(out).reshape(H, R, -1), ku.f64(lse).reshape(H, R)
    for h in range(H):
        want = v[h][best[h]]
        assert np.array_equal(out[h][clear[h]], want[clear[h]])
    assert np.all(np.abs(lse - top) <= 2.0 ** -18 * size + 1e-3 + np.log(S))
    assert np.all(np.abs(lse - top)[clear] <= 2.0 ** -18 * size[clear] + 1e-5)


@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("S", [100, 5000])
@pytest.mark.parametrize("size", [1e6, 1e8, 1e9, 1e12, 1e20, 1e30])
def test_large_queries(size, S, group):
    """Logits far past the fp32 numbers that are whole: up to 1e32, in whole units and in units split over CTAs."""
    rng = np.random.default_rng(int(np.log10(size)) + S)
    H, E = 2, 128
    cpu, k, v = ku.random_cache(rng, 1, H, -(-S // 16) * 16, E, E)
    q = ku.bf16(rng.standard_normal((1, group * H, 1, E)) * size)
    out, lse = attn.attn_decode_kv4(q.cuda(), to_gpu(cpu), scale=0.5, length=S)
    z = 0.5 * np.einsum("hre,hse->hrs", ku.f64(q).reshape(H, group, E), k[0, :, :S])
    check_one_hot(out, lse, z, v[0, :, :S], group)


@pytest.mark.parametrize("S", [100, 5000])
@pytest.mark.parametrize("factor", [1.0, 512.0, 4096.0])
def test_large_distances(S, factor):
    """The distance score with large keys, each query one of them: 2 <q, k> and ||k||^2 are up to 1e12, and the nearest
    key is the query's own."""
    rng = np.random.default_rng(S)
    H, E, group = 2, 128, 4
    k = ku.f64(ku.bf16(rng.standard_normal((1, H, -(-S // 16) * 16, E)) * factor))
    kc, ks = orc4.quantise(k)
    vc, vs = orc4.quantise(rng.standard_normal(k.shape))
    kh, vh = orc4.dequantise(kc, ks)[0], orc4.dequantise(vc, vs)[0]
    own = rng.integers(0, S, (H, group))
    q = ku.bf16(np.stack([kh[h][own[h]] for h in range(H)]).reshape(1, H * group, 1, E))
    cache = attn.KV4Cache(*(torch.from_numpy(t).cuda() for t in (kc, ks, vc, vs)))
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=1.0, length=S, mode="rbf")
    dots = np.einsum("hre,hse->hrs", ku.f64(q).reshape(H, group, E), kh[:, :S])
    norms = (kh[:, :S] ** 2).sum(-1)[:, None]
    check_one_hot(out, lse, 2 * dots - norms, vh[:, :S], group, shift=2 * np.abs(dots).max() + norms.max())


@pytest.mark.parametrize("size", [1.0, 1e8, 1e30])
def test_equal_keys_share_the_weight(size):
    """The best key twice, in different chunks of a unit split over CTAs: both have the same logit, so each half of the
    weight, however large the logit is."""
    rng = np.random.default_rng(3)
    S, E = 5008, 128
    cpu, k, v = ku.random_cache(rng, 1, 1, S, E, E)
    q = ku.bf16(rng.standard_normal((1, 2, 1, E)) * 30 * size)
    z = np.einsum("re,se->rs", ku.f64(q)[0, :, 0], k[0, 0])
    best = z.argmax(-1)
    other = [(int(b) + 2500) % S for b in best]
    for b, o in zip(best, other):
        for t in cpu[:2]:
            t[0, 0, o] = t[0, 0, b]
    k = orc4.dequantise(cpu[0].numpy(), cpu[1].numpy())
    z = np.einsum("re,se->rs", ku.f64(q)[0, :, 0], k[0, 0])
    out, _ = attn.attn_decode_kv4(q.cuda(), to_gpu(cpu), scale=1.0)
    for r in range(2):
        top = np.flatnonzero(z[r] == z[r].max())
        assert sorted(top) == sorted((best[r], other[r]))
        rest = np.delete(z[r], top).max()
        assert z[r].max() - rest > 40 + 2.0 ** -17 * np.abs(z[r]).max()
        mean = v[0, 0, top].mean(0)
        # a rounding to bf16, and the weight's of 1/2 to 2^-18
        assert np.all(np.abs(ku.f64(out)[0, r, 0] - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -16 * np.abs(v[0, 0, top]).max())


def test_logits_past_fp32_are_not_passed_over():
    """A row whose logits overflow fp32, to either side, does not come back as one that sees no key."""
    rng = np.random.default_rng(4)
    cpu, _, _ = ku.random_cache(rng, 1, 1, 304, 128, 128)
    for t in (cpu[0], cpu[2]):
        t &= 0x77  # no signs
    q = ku.bf16(np.abs(rng.standard_normal((1, 4, 1, 128))) * 1e37)
    q[0, 2:] *= -1
    out, lse = attn.attn_decode_kv4(q.cuda(), to_gpu(cpu), scale=10.0, length=300)
    assert torch.isnan(out).all() and not torch.isneginf(lse).any()
