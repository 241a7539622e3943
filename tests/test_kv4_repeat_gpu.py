"""Equal calls of the 4-bit cache's decode give equal bits, whenever their parts happen to run."""

import pytest
import torch

import attention_tiled_attn_b200 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda_ready():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from attention_tiled_attn_b200 import build as b
    b.build()
    yield
    assert attn.device_status() == 0


def random_cache(g, N, H, C, E, Ev):
    """Arbitrary elements under scales between 2^-3 and 1."""
    def of(lo, hi, w):
        return torch.randint(lo, hi, (N, H, C, w), dtype=torch.uint8, device="cuda", generator=g)
    return attn.KV4Cache(of(0, 256, E // 2), of(96, 121, E // 16), of(0, 256, Ev // 2), of(96, 121, Ev // 16))


def bits(got):
    out, lse = got
    return out.view(torch.int16).clone(), lse.view(torch.int32).clone()


# In each case many units are cut in two between neighbouring CTAs, and some in three.
CASES = {
    "8 query rows": dict(N=16, Hq=32, H=8, L=1, S=2100, E=128, Ev=128, ragged=False, sink=True),
    "16 query rows": dict(N=32, Hq=16, H=4, L=4, S=2600, E=128, Ev=64, ragged=False, sink=False),
    "ragged": dict(N=32, Hq=32, H=8, L=1, S=4096, E=128, Ev=128, ragged=True, sink=True),
    "narrow": dict(N=24, Hq=16, H=4, L=2, S=3000, E=64, Ev=64, ragged=True, sink=False),
}


@pytest.mark.parametrize("name", CASES)
def test_equal_bits_however_many_sms_are_busy(name):
    """Another stream holds some of the SMs, so that part of the decode's CTAs starts a millisecond after the others: a
    unit's parts are then ready in another order than on a free GPU."""
    c = CASES[name]
    N, Hq, H, L, S, E, Ev = (c[x] for x in ("N", "Hq", "H", "L", "S", "E", "Ev"))
    g = torch.Generator(device="cuda").manual_seed(len(name))
    cache = random_cache(g, N, H, -(-S // 16) * 16, E, Ev)
    q = (0.3 * torch.randn(N, Hq, L, E, device="cuda", generator=g)).bfloat16()
    kv_len = torch.randint(1, S + 1, (N,), dtype=torch.int32, device="cuda", generator=g) if c["ragged"] else None
    sink = torch.randn(Hq, device="cuda", generator=g) if c["sink"] else None

    def call():
        return bits(attn.attn_decode_kv4(q, cache, scale=E ** -0.5, length=S, kv_len=kv_len, sink=sink))

    want = call()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    side = torch.cuda.Stream()
    # the fp32 forward runs one CTA per head here, each through all of its keys
    held = [torch.randn(1, sms, rows, 64, device="cuda", generator=g) for rows in (1, 12000, 12000)]
    differ = []
    for busy in range(1, sms, 7):
        blocks = [t[:, :busy].contiguous() for t in held]
        torch.cuda.synchronize()
        kept = attn.attn_fwd(*blocks, scale=0.125, stream=side)  # its outputs are in use until the stream is done
        got = call()
        torch.cuda.synchronize()
        del kept
        if not all(torch.equal(a, b) for a, b in zip(got, want)):
            differ.append(busy)
    assert not differ, f"other bits with {differ} SMs busy"


def test_equal_bits_on_many_streams_and_in_graphs():
    """Calls of different shapes on four streams at once, half of them in replayed graphs: each gives the bits that it
    gives alone."""
    calls, want = [], []
    for i, name in enumerate(CASES):
        c = CASES[name]
        g = torch.Generator(device="cuda").manual_seed(50 + i)
        cache = random_cache(g, c["N"], c["H"], -(-c["S"] // 16) * 16, c["E"], c["Ev"])
        q = (0.3 * torch.randn(c["N"], c["Hq"], c["L"], c["E"], device="cuda", generator=g)).bfloat16()
        kv_len = torch.randint(0, c["S"] + 1, (c["N"],), dtype=torch.int32, device="cuda", generator=g)
        calls.append(lambda q=q, cache=cache, kv_len=kv_len, c=c, **kw: attn.attn_decode_kv4(
            q, cache, scale=c["E"] ** -0.5, length=c["S"], kv_len=kv_len, mask_kind="causal", **kw))
        want.append(bits(calls[-1]()))
    graphs = []
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        graphs.append((graph, got))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for turn in range(12):
        eager = []
        for i in range(len(calls)):
            j = (i + turn) % len(calls)  # the call on stream i; the next stream replays the graph of another one
            if (i + turn // 4) % 2:
                with torch.cuda.stream(streams[i]):
                    graphs[j][0].replay()
            else:
                eager.append((j, calls[j](stream=streams[i])))
        torch.cuda.synchronize()
        for j, got in eager:
            assert all(torch.equal(a, b) for a, b in zip(bits(got), want[j])), f"turn {turn}, case {j}"
    for graph, got in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for (_, got), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(bits(got), w))
