"""Measured cases of the 4-bit key/value cache: writing rows into it, reading rows back, attention over it.

A cache row of E values is held as E / 16 blocks of 16.  A block keeps one unsigned 8-bit scale s (5 exponent bits of
bias 15, 3 mantissa bits: the nearest to max|x| / 6, ties to even, at most 10240) and 16 elements of 4 bits (a sign and
one of 0, .5, 1, 1.5, 2, 3, 4, 6: the nearest to |x| / s, ties to even).  Element 2i of a row is the low half of byte i.
A block with a NaN has the scale byte 255, which reads back as NaN.

With ``own`` false ``run`` computes in elementary torch operations, in 32 bits; with ``own`` true it calls the package.
"""

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 16
MAX_ROWS = 16  # query rows of one KV head in a decode call
LARGEST = 16 * 8 * 131072  # cached rows (batch x KV heads x length) of the largest case


def listed():
    return [
        # one short conversation, one token: only the latency counts
        dict(name="decode one 130", op="decode", N=1, Hq=32, H=8, L=1, S=130, E=128, Ev=128, mask="none"),
        # a served batch in the middle of its answers, every sequence of its own length, with sink logits
        dict(name="decode batch ragged 4k", op="decode", N=32, Hq=32, H=8, L=1, S=4096, E=128, Ev=128, mask="none", sink=True, ragged=True),
        # one user's very long context with few KV heads: the key axis alone has to fill the machine
        dict(name="decode few heads 128k", op="decode", N=1, Hq=16, H=2, L=1, S=131072, E=128, Ev=128, mask="causal"),
        # the largest: long contexts in a batch, with sink logits
        dict(name="decode batch 128k", op="decode", N=16, Hq=32, H=8, L=1, S=131072, E=128, Ev=128, mask="none", sink=True),
        # four proposed tokens checked at once under the streaming mask (4 kept keys, a 4096-key window), 64-wide heads
        dict(name="decode streaming L4", op="decode", N=8, Hq=32, H=8, L=4, S=16383, E=64, Ev=64, mask="streaming", window=4096, keep=4, ragged=True),
        # the distance score without grouped heads, an odd length
        dict(name="decode rbf 4100", op="decode", N=8, Hq=12, H=12, L=1, S=4100, E=64, Ev=64, mask="none", mode="rbf"),
        # one new token of each sequence of a batch, at its own position, and those rows again
        dict(name="append one", op="write_read", N=32, H=8, L=1, C=4096, E=128, Ev=128, dtype="bf16", ragged=True),
        # a batch of prompts straight out of the projection (strided), and their rows for the prompt's own attention
        dict(name="prompt 8k", op="write_read", N=4, H=8, L=8192, C=8192, E=128, Ev=128, dtype="bf16", fused=True),
        # ragged pieces of prompts in 32 bits, head widths that differ, an odd length
        dict(name="piece ragged fp32", op="write_read", N=5, H=3, L=777, C=2048, E=64, Ev=128, dtype="fp32", ragged=True),
        # a long cache read back for the attention of a following prompt piece
        dict(name="read 128k", op="read", N=1, H=8, start=0, rows=131072, C=131072, E=128, Ev=128, dtype="bf16"),
        # part of a ragged batch's rows from an odd start
        dict(name="read ragged part", op="read", N=7, H=5, start=333, rows=1999, C=4096, E=64, Ev=64, dtype="bf16", ragged=True),
        # one generation step of a batch: append each sequence's new token, then attend to all it has
        dict(name="step batch ragged 8k", op="step", N=32, Hq=32, H=8, L=1, S=8000, E=128, Ev=128, mask="causal", ragged=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["decode", "decode", "decode", "step", "write_read", "read"])
    E, Ev = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64)])
    H, N = rng.choice([1, 2, 3, 4, 5, 8, 12]), log(1, 64)
    if op in ("decode", "step"):
        L = rng.choice([1, 1, 1, 2, 4])
        group = rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * L <= MAX_ROWS])
        S = max(L, log(1, min(131072, LARGEST // (4 * N * H))))
        mask = rng.choice(["none", "causal", "window", "streaming"])
        return dict(op=op, N=N, Hq=H * group, H=H, L=L, S=S, E=E, Ev=Ev, mask=mask, window=log(1, 8192), keep=rng.randint(1, 100),
                    sink=rng.random() < 0.5, mode=rng.choice(["dot", "dot", "rbf"]), ragged=rng.random() < 0.7)
    C = 16 * log(1, min(8192, LARGEST // (16 * 16 * N * H)))
    n = rng.randint(1, C)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "read":
        return dict(op=op, N=N, H=H, start=rng.randint(0, C - n), rows=n, C=C, E=E, Ev=Ev, dtype=dtype, ragged=rng.random() < 0.5)
    return dict(op=op, N=N, H=H, L=n, C=C, E=E, Ev=Ev, dtype=dtype, ragged=rng.random() < 0.5, fused=rng.random() < 0.5)


def spread(case, most, salt):
    """One whole number in [1, most] for each sequence, the first of them `most` where there are several."""
    if not case.get("ragged"):
        return [most] * case["N"]
    return [most if n == 0 and case["N"] > 1 else 1 + (n * 2654435761 + salt * 40503 + 977) % 1000003 % most for n in range(case["N"])]


def lengths(case):
    """Cached rows of each sequence (those appended by a step among them)."""
    if case["op"] in ("decode", "step"):
        return [max(x, case["L"]) for x in spread(case, case["S"], 1)]
    return spread(case, case["C"], 2)


def capacity(case):
    return case["C"] if "C" in case else -(-case["S"] // BLOCK) * BLOCK


def visible(case):
    """Cached rows that some query of each sequence sees."""
    seen = []
    for n in lengths(case):
        first = max(0, n - case["L"] - case["window"] + 1) if case["mask"] in ("window", "streaming") else 0
        kept = min(case["keep"], first) if case["mask"] == "streaming" else 0
        seen.append(n - first + kept)
    return seen


def work(case):
    N, H, E, Ev = case["N"], case["H"], case["E"], case["Ev"]
    cached = (E + Ev) * 9 // 16  # bytes of one row: half a byte a value, one scale byte for 16
    if case["op"] in ("decode", "step"):
        rows, calls = sum(visible(case)) * H, N * case["Hq"] * case["L"]
        total = rows * cached + calls * (2 * E + 2 * Ev + 4)
        if case["op"] == "step":
            total += N * H * case["L"] * ((E + Ev) * 2 + cached + (E + Ev) * 2)
        return {"bytes": total, "flops": 2 * (E + Ev) * rows * (case["Hq"] // H) * case["L"]}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "read":
        held = sum(max(0, min(n - case["start"], case["rows"])) for n in lengths(case)) * H
        return {"bytes": held * cached + N * H * case["rows"] * (E + Ev) * size, "flops": held * (E + Ev)}
    new = sum(spread(case, case["L"], 3)) * H
    return {"bytes": new * (cached + (E + Ev) * size) + new * cached + N * H * case["L"] * (E + Ev) * size, "flops": 4 * new * (E + Ev)}


def scale_values(byte):
    """The values that scale bytes stand for: 5 exponent and 3 mantissa bits are the upper bits of a 16-bit float."""
    return (byte.to(torch.int16) << 7).view(torch.float16).float()


def quantise(x):
    """(codes, scales): the bytes that a cache holds for the rows of x (..., E)."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    nan = x.isnan().any(-1)
    most = x.abs().amax(-1)
    y = most / torch.full_like(most, 6.0)  # two tensors: a true division
    bits = y.view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (112 << 3)
    byte = torch.where(y < 2.0**-14, torch.round(y * 2.0**17).to(torch.int32), normal).clamp(max=226)
    s = torch.where(nan, torch.zeros_like(y), scale_values(byte)).unsqueeze(-1)
    a = x.abs() / s
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code = torch.where(s > 0, code | ((x < 0).to(torch.uint8) << 3), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(nan, torch.full_like(byte, 255), byte).to(torch.uint8)


def dequantise(codes, scales):
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    x = table[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, BLOCK)) * scale_values(scales).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, H, E, Ev, C = case["N"], case["H"], case["E"], case["Ev"], capacity(case)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    # a cache as earlier writes left it: head dimensions of different sizes, a few of them much larger than the rest
    cache = tuple(torch.empty(N, H, C, w, dtype=torch.uint8, device="cuda") for w in (E // 2, E // BLOCK, Ev // 2, Ev // BLOCK))
    spread_k, spread_v = (torch.exp(0.7 * normal(H, 1, w)) for w in (E, Ev))
    for n in range(N):
        cache[0][n], cache[1][n] = quantise((normal(H, C, E) * spread_k).bfloat16())
        cache[2][n], cache[3][n] = quantise((normal(H, C, Ev) * spread_v).bfloat16())
    s = {"case": case, "cache": cache}

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if case["op"] in ("decode", "step"):
        L, Hq = case["L"], case["Hq"]
        # queries whose logits have a standard deviation of about 1.5
        per_head = (spread_k.square().sum(-1).sqrt() / E**0.5).repeat_interleave(Hq // H, 0).reshape(1, Hq, 1, 1)
        s["q"] = (normal(N, Hq, L, E) * 1.5 / per_head).bfloat16()
        s["scale"] = E**-0.5
        s["sink"] = normal(Hq) if case.get("sink") else None
        s["kv_len"] = whole(lengths(case)) if case.get("ragged") else None
        s["length"] = case["S"]
    if case["op"] in ("write_read", "step"):
        L = case["L"]
        dtype = DTYPES[case.get("dtype", "bf16")]
        if case.get("fused"):
            both = torch.cat((normal(N, L, H, E) * spread_k.transpose(0, 1), normal(N, L, H, Ev) * spread_v.transpose(0, 1)), -1).to(dtype)
            s["k"], s["v"] = both[..., :E].transpose(1, 2), both[..., E:].transpose(1, 2)
        else:
            s["k"], s["v"] = (normal(N, H, L, E) * spread_k).to(dtype), (normal(N, H, L, Ev) * spread_v).to(dtype)
        if case["op"] == "step":
            s["pos"] = whole([n - L for n in lengths(case)])
            s["count"] = None
        elif case.get("ragged"):
            count = spread(case, L, 3)
            pos = [min(a, C - L) for a in spread(case, C, 4)]
            s["pos"], s["count"], s["kv_len"] = whole(pos), whole(count), whole([a + b for a, b in zip(pos, count)])
        else:
            s["pos"] = s["count"] = s["kv_len"] = None
    if case["op"] == "read":
        s["kv_len"] = whole(lengths(case)) if case.get("ragged") else None
    return s


def plain_write(cache, k, v, pos, count):
    N, H, L, _ = k.shape
    C = cache[0].shape[2]
    step = torch.arange(L, device=k.device)
    row = step.expand(N, L) if pos is None else pos.long()[:, None] + step
    ok = (row >= 0) & (row < C)
    if count is not None:
        ok = ok & (step < count[:, None])
    n, l = ok.nonzero(as_tuple=True)
    for held, new in zip(cache, quantise(k) + quantise(v)):
        held[n, :, row[n, l]] = new[n, :, l]


def plain_read(cache, start, pos, rows, kv_len, dtype):
    N, H, C, _ = cache[0].shape
    step = torch.arange(rows, device=cache[0].device)
    row = (start + step).expand(N, rows) if pos is None else pos.long()[:, None] + step
    ok = (row >= 0) & (row < C)
    if kv_len is not None:
        ok = ok & (row < kv_len[:, None])
    at = row.clamp(0, C - 1)
    n = torch.arange(N, device=row.device)[:, None]
    out = []
    for codes, scales in (cache[:2], cache[2:]):
        x = dequantise(codes[n, :, at], scales[n, :, at])  # (N, rows, H, E)
        x = torch.where(ok[:, :, None, None], x, torch.zeros_like(x))
        out.append(x.transpose(1, 2).to(dtype).contiguous())
    return tuple(out)


def mask_of(case, length, S, L):
    """(N, L, S): which cached rows each query sees; `length` (N,) counts the rows of each sequence."""
    j = torch.arange(S, device=length.device)
    i = length[:, None, None] - L + torch.arange(L, device=length.device)[None, :, None]
    ok = (j < length[:, None, None]).expand(-1, L, -1)
    if case["mask"] != "none":
        ok = ok & (j <= i)
    if case["mask"] == "window":
        ok = ok & (i - j < case["window"])
    if case["mask"] == "streaming":
        ok = ok & ((i - j < case["window"]) | (j < case["keep"]))
    return ok


def plain_decode(s, case):
    q = s["q"].float()
    N, Hq, L, E = q.shape
    S, H = s["length"], case["H"]
    kc, ks, vc, vs = (t[:, :, :S] for t in s["cache"])
    k = dequantise(kc, ks)
    z = torch.matmul(q.reshape(N, H, Hq // H * L, E), k.transpose(-1, -2)) * s["scale"]
    if case.get("mode") == "rbf":
        z = 2 * z - s["scale"] * k.square().sum(-1)[:, :, None, :]
    del k
    length = s["kv_len"] if s["kv_len"] is not None else torch.full((N,), S, dtype=torch.int32, device=q.device)
    ok = mask_of(case, length, S, L)
    z = z.reshape(N, Hq, L, S).masked_fill(~ok[:, None], float("-inf"))
    most = z.amax(-1)
    if s["sink"] is not None:
        most = torch.maximum(most, s["sink"][None, :, None])
    shift = torch.where(most == float("-inf"), torch.zeros_like(most), most)
    p = torch.exp(z - shift[..., None])
    total = p.sum(-1)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][None, :, None] - shift)
    o = torch.matmul(p.reshape(N, H, Hq // H * L, S), dequantise(vc, vs)).reshape(N, Hq, L, -1)
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return o.bfloat16(), shift + torch.log(total)


def run(s):
    case, cache = s["case"], s["cache"]
    op = case["op"]
    if own:
        import attention_tiled_attn_b200 as attn

        got = ()
        if op in ("write_read", "step"):
            attn.attn_kv4_write(cache, s["k"], s["v"], pos=s["pos"], count=s["count"])
        if op in ("decode", "step"):
            got = attn.attn_decode_kv4(s["q"], cache, scale=s["scale"], length=s["length"], kv_len=s["kv_len"], mode=case.get("mode", "dot"),
                                       sink=s["sink"], mask_kind=case["mask"], window=case.get("window", 0),
                                       keep_first=case.get("keep", 0) if case["mask"] == "streaming" else 0)
        if op == "read":
            got = attn.attn_kv4_read(cache, case["rows"], start=case["start"], kv_len=s["kv_len"], dtype=DTYPES[case["dtype"]])
        elif op == "write_read" or op == "step":
            got = got + attn.attn_kv4_read(cache, case["L"], pos=s["pos"], kv_len=s["kv_len"], dtype=s["k"].dtype)
        return got
    got = ()
    if op in ("write_read", "step"):
        plain_write(cache, s["k"], s["v"], s["pos"], s["count"])
    if op in ("decode", "step"):
        got = plain_decode(s, case)
    if op == "read":
        got = plain_read(cache, case["start"], None, case["rows"], s["kv_len"], DTYPES[case["dtype"]])
    elif op == "write_read" or op == "step":
        got = got + plain_read(cache, 0, s["pos"], case["L"], s["kv_len"], s["k"].dtype)
    return got


# ---- the definition in 64 bits, apart from the plain form: every rounding is a search among the values it can give ----

def nearest(grid, x):
    """The index of the value of `grid` (ascending) nearest to x, the even index at a tie."""
    middle = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(middle, x, right=False), torch.searchsorted(middle, x, right=True)
    return torch.where(low % 2 == 0, low, high)


def all_scales(device):
    values = [b * 2.0**-17 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 15) for b in range(227)]
    return torch.tensor(values, dtype=torch.float64, device=device)


def exact_rounded(x):
    """What a row x comes back as from the cache."""
    x = x.double().unflatten(-1, (-1, BLOCK)).contiguous()
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    scales = all_scales(x.device)
    most = x.abs().amax(-1)
    s = scales[nearest(scales, (most / torch.full_like(most, 6.0)).contiguous())].unsqueeze(-1)
    m = grid[nearest(grid, (x.abs() / torch.where(s > 0, s, torch.ones_like(s))).contiguous())]
    return (torch.where(x < 0, -m, m) * s).flatten(-2)


def exact_held(codes, scales):
    """The values that cache bytes stand for."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=codes.device)
    half = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.uint8, device=codes.device)
    half[..., 0::2], half[..., 1::2] = codes % 16, codes // 16
    m = grid[(half % 8).long()]
    m = torch.where(half >= 8, -m, m)
    return m * all_scales(codes.device)[scales.long()].repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, cache, N = case["op"], s["cache"], case["N"]
    if op == "read":
        C = case["C"]
        out = []
        for codes, scales in (cache[:2], cache[2:]):
            x = exact_held(codes[:, :, case["start"]:case["start"] + case["rows"]], scales[:, :, case["start"]:case["start"] + case["rows"]])
            for n, length in enumerate(lengths(case) if case.get("ragged") else [C] * N):
                x[n, :, max(0, length - case["start"]):] = 0
            out.append(x)
        return tuple(out)
    back = ()
    if op in ("write_read", "step"):
        back = (exact_rounded(s["k"]), exact_rounded(s["v"]))
        if op == "write_read":
            for n, count in enumerate(spread(case, case["L"], 3)):
                back[0][n, :, count:] = 0
                back[1][n, :, count:] = 0
            return back
    S, H, L, E = case["S"], case["H"], case["L"], case["E"]
    group = case["Hq"] // H
    outs, lses = [], []
    for n in range(N):
        length = lengths(case)[n]
        k, v = (exact_held(codes[n, :, :length], scales[n, :, :length]) for codes, scales in (cache[:2], cache[2:]))
        if op == "step":
            k[:, length - L:], v[:, length - L:] = back[0][n], back[1][n]
        q = s["q"][n].double().reshape(H, group * L, E)
        z = s["scale"] * torch.einsum("hre,hse->hrs", q, k)
        if case.get("mode") == "rbf":
            z = 2 * z - s["scale"] * (k * k).sum(-1)[:, None]
        at = torch.arange(L, device=z.device)[:, None] + length - L
        j = torch.arange(length, device=z.device)[None]
        hidden = torch.zeros(L, length, dtype=torch.bool, device=z.device) if case["mask"] == "none" else j > at
        if case["mask"] in ("window", "streaming"):
            old = at - j >= case["window"]
            hidden = hidden | (old & (j >= case["keep"]) if case["mask"] == "streaming" else old)
        z = z.reshape(H * group, L, length).masked_fill(hidden, float("-inf"))
        if s["sink"] is not None:
            z = torch.cat((z, s["sink"].double()[:, None, None].expand(-1, L, 1)), -1)
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - lse[..., None])[..., :length]
        outs.append(torch.einsum("hrs,hsd->hrd", p.reshape(H, group * L, length), v).reshape(case["Hq"], L, -1))
        lses.append(lse)
    return (torch.stack(outs), torch.stack(lses)) + back
