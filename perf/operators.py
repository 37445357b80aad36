"""Cases, plain forms and exact values of the block-scaled 8-bit cache and of windowed attention.

Three operators of a decode layer call over the paged latent cache (512 latent and 64 rotary columns a
token):

* ``append_q8``: the newest tokens of each request quantized to E4M3 into the paged cache, with one
  power-of-two scale for every ``g`` consecutive tokens;
* ``decode_q8``: absorbed attention over that cache, whole, or through a sliding window beside a few first
  tokens that stay visible (sinks);
* ``decode_window``: absorbed attention over a 16-bit cache through such a window.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, through the
package. ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

R, D = 512, 64  # latent and rotary columns
SCALE = 1.0 / math.sqrt(192.0)
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60  # a scale is a power of two in [2^-60, 2^60]


def listed():
    return [
        # one short chat turn on an idle server: nothing but latency
        dict(name="q8 one short request", op="decode_q8", B=1, H=16, q=1, lo=37, hi=37, bs=16, g=1, dtype="f16", causal=False, window=0, sinks=0),
        # one long document being answered
        dict(name="q8 one long request", op="decode_q8", B=1, H=16, q=1, lo=131072, hi=131072, bs=32, g=32, dtype="f16", causal=False, window=0, sinks=0),
        # a serving batch of 16-head ranks, contexts of all lengths
        dict(name="q8 ragged batch", op="decode_q8", B=32, H=16, q=1, lo=100, hi=16384, bs=32, g=1, dtype="bf16", causal=False, window=0, sinks=0),
        # all heads on one device, long contexts
        dict(name="q8 many heads", op="decode_q8", B=8, H=128, q=1, lo=4096, hi=65536, bs=64, g=64, dtype="bf16", causal=False, window=0, sinks=0),
        # drafts being verified behind long prefixes
        dict(name="q8 verify window", op="decode_q8", B=4, H=16, q=9, lo=40969, hi=81929, bs=32, g=16, dtype="f16", causal=True, window=0, sinks=0),
        # a long-running batch that only keeps a window and the first tokens
        dict(name="q8 sliding window", op="decode_q8", B=48, H=64, q=1, lo=900, hi=40000, bs=64, g=1, dtype="bf16", causal=False, window=4096, sinks=4),
        # a 16-bit cache: one endless stream through a short window
        dict(name="window one stream", op="decode_window", B=1, H=16, q=1, lo=131072, hi=131072, bs=32, g=0, dtype="f16", causal=False, window=1024, sinks=4),
        # a batch of streams on all heads
        dict(name="window many heads", op="decode_window", B=32, H=128, q=1, lo=3000, hi=32768, bs=64, g=0, dtype="bf16", causal=False, window=4096, sinks=64),
        # drafts verified through a window
        dict(name="window verify", op="decode_window", B=16, H=16, q=4, lo=700, hi=20000, bs=32, g=0, dtype="f16", causal=True, window=2000, sinks=5),
        # the cache write of one request's next token
        dict(name="append one token", op="append_q8", B=1, H=0, q=1, lo=1000, hi=1000, bs=32, g=32, dtype="f16", causal=False, window=0, sinks=0),
        # a decode step of a large batch with drafts, landing anywhere in a page
        dict(name="append batch", op="append_q8", B=256, H=0, q=4, lo=3, hi=700, bs=32, g=16, dtype="bf16", causal=False, window=0, sinks=0),
        # the tokens of a prefill chunk
        dict(name="append chunk", op="append_q8", B=8, H=0, q=8192, lo=8192, hi=20001, bs=64, g=1, dtype="bf16", causal=False, window=0, sinks=0),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("decode_q8", "decode_q8", "decode_q8", "decode_window", "decode_window", "append_q8"))
    bs = rng.choice((16, 32, 64))
    c = dict(op=op, H=0, bs=bs, g=0, dtype=rng.choice(("f16", "bf16")), causal=False, window=0, sinks=0)
    if op != "decode_window":
        c["g"] = rng.choice([g for g in (1, 2, 4, 8, 16, 32, 64) if g <= bs])
    if op == "append_q8":
        c["q"] = spread(rng, 1, 4096)
        c["B"] = spread(rng, 1, max(1, 65536 // max(c["q"], 64)))
        c["lo"] = spread(rng, 1, 8192)
        c["hi"] = c["lo"] + spread(rng, 1, 8192)
        return c
    c["H"] = rng.choice((16, 16, 64, 128))
    c["q"] = rng.choice((1, 1, 1, spread(rng, 2, 32)))
    c["causal"] = c["q"] > 1
    if op == "decode_window" or rng.random() < 0.4:
        c["window"] = spread(rng, 1, 16384)
        c["sinks"] = rng.choice((0, 1, 4, spread(rng, 1, 300)))
    tokens = min(131072, int(4e10 / (2176 * c["H"] * c["q"])))  # of the batch together
    c["B"] = spread(rng, 1, 64)
    c["hi"] = spread(rng, 1, max(1, tokens // c["B"]))
    c["lo"] = spread(rng, 1, c["hi"])
    return c


def lengths(case):
    """Context lengths of the requests, the newest tokens among them."""
    r = random.Random(case["lo"] * 1000003 + case["hi"] * 101 + case["B"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[0] = case["hi"]
    return lens


def seen(case, L, i):
    """How many tokens row i of a request of L tokens sees."""
    pos = L - case["q"] + i if case["causal"] else L - 1
    if pos < 0:
        return 0
    if not case["window"]:
        return pos + 1
    low = max(0, pos - case["window"] + 1)
    return pos + 1 - low + min(case["sinks"], low)


def read(case, L):
    """How many tokens of a request any of its rows sees."""
    if not case["window"]:
        return L
    first = L - case["q"] if case["causal"] else L - 1
    low = max(0, first - case["window"] + 1)
    return L - low + min(case["sinks"], low)


def work(case):
    lens, q, H, g = lengths(case), case["q"], case["H"], case["g"]
    if case["op"] == "append_q8":
        tokens = sum(min(q, L) for L in lens)
        return {"bytes": tokens * (3 * (R + D)) + sum(4 * -(-min(q, L) // g) for L in lens), "flops": 2 * tokens * (R + D)}
    a_token = (R + D) + 4 / g if g else 2 * (R + D)
    rows = case["B"] * q * H
    pairs = sum(seen(case, L, i) for L in lens for i in range(q)) * H
    return {"bytes": int(sum(read(case, L) for L in lens) * a_token) + rows * (2 * (R + D) + 2 * R + 4), "flops": 2 * pairs * (R + D + R)}


def pages(case, lens, gen):
    """A block table over a shuffled pool, and the pool's pages; -1 behind each request's last page."""
    bs = case["bs"]
    need = [-(-L // bs) for L in lens]
    nb = sum(need) + max(1, sum(need) // 8)
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")[:, None]
    j = torch.arange(max(need), device="cuda")[None]
    held = j < torch.tensor(need, device="cuda")[:, None]
    return torch.where(held, perm[(at + j).clamp(max=nb - 1)], -1).to(torch.int32).contiguous(), nb


def latents(gen, n, dtype):
    """Latents and rotary keys of n tokens: most tokens near unit size, some far larger or smaller."""
    size = torch.exp2(2.0 * torch.randn(n, 1, generator=gen, device="cuda")).clamp(2.0**-6, 2.0**3)
    c = torch.randn(n, R, generator=gen, device="cuda") * size
    k = torch.randn(n, D, generator=gen, device="cuda") * size
    return c.to(T16[dtype]), k.to(T16[dtype])


def pow2_scale(amax):
    """The least power of two s in the scales' range with amax / s <= 448; NaN where amax is not finite or too large."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    k = torch.where(amax == 0, MIN_EXP, k)
    s = torch.ldexp(torch.ones_like(amax), k.clamp(max=MAX_EXP))
    return torch.where(torch.isfinite(amax) & (k <= MAX_EXP), s, float("nan"))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    lens = lengths(case)
    B, q, H, bs, g, dtype = case["B"], case["q"], case["H"], case["bs"], case["g"], case["dtype"]
    table, nb = pages(case, lens, gen)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    c, k = latents(gen, nb * bs, dtype)
    if g:
        # the pool as earlier writes left it: each block of g tokens on a scale of its own
        c, k = c.float().view(-1, g, R), k.float().view(-1, g, D)
        scales = pow2_scale(torch.maximum(c.abs().amax((1, 2)), k.abs().amax((1, 2))))
        s["ckv"] = (c / scales[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(nb, bs, R)
        s["kpe"] = (k / scales[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(nb, bs, D)
        s["scales"] = scales.view(nb, bs // g)
    else:
        s["ckv"], s["kpe"] = c.view(nb, bs, R), k.view(nb, bs, D)
    del c, k
    if case["op"] == "append_q8":
        c, k = latents(gen, B * q, dtype)
        s["ckv_new"], s["kpe_new"] = c.view(B, q, R), k.view(B, q, D)
        if own:
            from mla_split_kv_gb300 import runtime as rt
            s["cache"] = rt.Q8Cache(s["ckv"], s["kpe"], s["scales"])
        return s
    s["q_abs"] = torch.randn(B, q, H, R, generator=gen, device="cuda").to(T16[dtype])
    s["q_pe"] = torch.randn(B, q, H, D, generator=gen, device="cuda").to(T16[dtype])
    if own:
        from mla_split_kv_gb300 import runtime as rt
        s["out"] = torch.empty(B, q, H, R, dtype=T16[dtype], device="cuda")
        s["lse"] = torch.empty(B, q, H, device="cuda")
        if g:
            s["cache"] = rt.Q8Cache(s["ckv"], s["kpe"], s["scales"])
            s["plan"] = rt.plan_q8(B, H, q, causal=case["causal"], window=case["window"], sinks=case["sinks"])
        else:
            s["plan"] = rt.plan_window(lens, H, q, bs, case["window"], case["sinks"], dtype=dtype, causal=case["causal"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        from mla_split_kv_gb300 import runtime as rt
        if op == "append_q8":
            rt.cache_append_q8(s["cache"], s["ckv_new"], s["kpe_new"], s["table"], s["lens"])
            return cache_values(s)
        if op == "decode_q8":
            rt.decode_q8(s["plan"], s["q_abs"], s["q_pe"], s["cache"], s["table"], s["lens"], SCALE, s["out"], s["lse"])
        else:
            rt.decode_window(s["plan"], s["q_abs"], s["q_pe"], s["ckv"], s["kpe"], s["table"], s["lens"], SCALE, s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    return append_plain(s) if op == "append_q8" else decode_plain(s)


def cache_values(s):
    return {"ckv": s["ckv"].view(torch.float8_e4m3fn), "kpe": s["kpe"].view(torch.float8_e4m3fn), "scales": s["scales"]}


def append_plain(s):
    """The write, by the blocks that each request's new tokens touch: [request, touched block, token of the block]."""
    case = s["case"]
    q, bs, g = case["q"], case["bs"], case["g"]
    first = s["lens"].long() - q  # may be negative: those tokens have no place
    nt = (q - 1) // g + 2
    block = first.clamp(min=0)[:, None] // g + torch.arange(nt, device="cuda")  # logical blocks of g tokens
    t = block[:, :, None] * g + torch.arange(g, device="cuda")
    i = t - first[:, None, None]
    new = (i >= 0) & (i < q)
    old = (i < 0) & new.any(-1, keepdim=True)
    page = s["table"].long().gather(1, (t // bs).clamp(max=s["table"].shape[1] - 1).flatten(1)).view_as(t).clamp(min=0)
    row = page * bs + t % bs
    index = row[:, :, 0] // g
    ckv, kpe, scales = s["ckv"].view(-1, R), s["kpe"].view(-1, D), s["scales"].view(-1)
    at = torch.arange(len(t), device="cuda")[:, None, None].expand_as(i)
    value = torch.cat((s["ckv_new"], s["kpe_new"]), -1)[at, i.clamp(0, q - 1)].float()
    amax = torch.where(new, value.abs().amax(-1), 0).amax(-1)
    keep = old.any(-1)
    before = scales[index]
    fresh = pow2_scale(amax)
    scale = torch.where(keep, torch.maximum(before, fresh), fresh)[:, :, None]
    poisoned = torch.isnan(scale)[..., None]
    quant = torch.where(poisoned, 0, value / scale[..., None])[new].clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    grown = old & (scale > before[:, :, None])
    ratio = (before[:, :, None] / scale).expand_as(grown)[grown][:, None]
    stale = torch.cat((ckv[row[grown]], kpe[row[grown]]), -1).view(torch.float8_e4m3fn).float()
    stale = (stale * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    ckv[row[grown]], kpe[row[grown]] = stale[:, :R], stale[:, R:]
    quant = quant.view(torch.uint8)
    ckv[row[new]], kpe[row[new]] = quant[:, :R], quant[:, R:]
    touched = new.any(-1)
    scales[index[touched]] = scale[..., 0][touched]
    return cache_values(s)


def tokens_read(s):
    """Positions [request, n] that the rows of each request see between them, and which of them are any token's."""
    case = s["case"]
    L = s["lens"].long()
    first = L - (case["q"] if case["causal"] else 1)
    low = (first - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(L)
    sinks = low.clamp(max=case["sinks"])
    n = max(read(case, x) for x in lengths(case))
    u = torch.arange(n, device="cuda")[None]
    t = torch.where(u < sinks[:, None], u, u - sinks[:, None] + low[:, None])
    return t, t < L[:, None]


def attend(s, t, real, ckv, kpe, size, wide):
    """Attention of every row over the positions t, in the type `wide`."""
    case = s["case"]
    q, H = case["q"], case["H"]
    L, qa, qp = s["lens"].long(), s["q_abs"].to(wide).flatten(1, 2), s["q_pe"].to(wide).flatten(1, 2)
    score = (qa @ ckv.mT + qp @ kpe.mT) * SCALE
    if size is not None:
        score, ckv = score * size[:, None], ckv * size[..., None]
    pos = L[:, None] - q + torch.arange(q, device="cuda")[None] if case["causal"] else (L[:, None] - 1).expand(-1, q)
    ok = real[:, None] & (t[:, None] <= pos[..., None])
    if case["window"]:
        ok &= (t[:, None] > pos[..., None] - case["window"]) | (t[:, None] < case["sinks"])
    score = score.unflatten(1, (q, H)).masked_fill(~ok[:, :, None], float("-inf"))
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m.masked_fill(m == float("-inf"), 0))
    l = p.sum(-1, keepdim=True)
    out = (p.flatten(1, 2) @ ckv).unflatten(1, (q, H)) / l.masked_fill(l == 0, 1)
    return {"out": out.to(T16[case["dtype"]]) if wide == torch.float32 else out, "lse": (m + torch.log(l))[..., 0] / math.log(2.0)}


def decode_plain(s):
    case = s["case"]
    bs, g = case["bs"], case["g"]
    t, real = tokens_read(s)
    page = s["table"].long().gather(1, (t // bs).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    row = page * bs + t % bs
    f8 = torch.float8_e4m3fn
    ckv, kpe, size = s["ckv"].view(-1, R)[row], s["kpe"].view(-1, D)[row], None
    if g:
        ckv, kpe, size = ckv.view(f8), kpe.view(f8), s["scales"].view(-1)[row // g]
    return attend(s, t, real, ckv.float(), kpe.float(), size, torch.float32)


def e4m3_table():
    """The 256 values of the format: sign, 4 exponent bits (bias 7), 3 of fraction; S.1111.111 is NaN."""
    b = torch.arange(256, device="cuda")
    e, f = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, f * 2.0**-9, (1 + f / 8) * torch.exp2((e - 7).double()))
    return torch.where((b & 127) == 127, float("nan"), torch.where(b >= 128, -v, v))


def to_e4m3(x):
    """The nearest value of the format in 64 bits, ties to the even fraction, 448 where it is beyond."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0**-30)))
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, torch.where(torch.exp2(e) > x.abs(), e - 1, e)).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    lens, q, bs, g = lengths(case), case["q"], case["bs"], case["g"]
    if case["op"] != "append_q8":
        out, lse, table = [], [], s["table"].long()
        for b, L in enumerate(lens):
            t, real = tokens_read({**s, "lens": s["lens"][b : b + 1]})
            t = t[:, : max(1, read(case, L))]
            row = table[b][t[0] // bs].clamp(min=0) * bs + t[0] % bs
            c, k, size = s["ckv"].view(-1, R)[row], s["kpe"].view(-1, D)[row], None
            if g:
                values = e4m3_table()
                c, k, size = values[c.long()], values[k.long()], s["scales"].view(-1)[row // g].double()[None]
            one = {**s, "lens": s["lens"][b : b + 1], "q_abs": s["q_abs"][b : b + 1], "q_pe": s["q_pe"][b : b + 1]}
            o = attend(one, t, real[:, : t.shape[1]], c.double()[None], k.double()[None], size, torch.float64)
            out.append(o["out"])
            lse.append(o["lse"])
        return {"out": torch.cat(out), "lse": torch.cat(lse)}
    # the write, block after block of each request
    if case["B"] * (q // g + 2) > 20000:
        return exact_fresh(case, s)
    values = e4m3_table()
    ckv, kpe, scales = values[s["ckv"].view(-1, R).long()], values[s["kpe"].view(-1, D).long()], s["scales"].view(-1).double()
    for b, L in enumerate(lens):
        first = max(0, L - q)
        for block in range(first // g, (L - 1) // g + 1):
            t = torch.arange(block * g, min(L, block * g + g), device="cuda")
            row = s["table"][b].long()[t // bs] * bs + t % bs
            i = t - (L - q)
            new, at = row[t >= first], i[t >= first]
            x = torch.cat((s["ckv_new"][b, at], s["kpe_new"][b, at]), -1).double()
            top = float(x.abs().max())
            size = 2.0**MIN_EXP
            while top / size > E4M3_MAX:
                size *= 2
            n = int(row[0]) // g
            if len(new) < len(row):
                size = max(size, float(scales[n]))
                stale = row[t < first]
                if size > float(scales[n]):
                    ckv[stale], kpe[stale] = (to_e4m3(v[stale] * float(scales[n]) / size) for v in (ckv, kpe))
            scales[n] = size
            x = to_e4m3(x / size)
            ckv[new], kpe[new] = x[:, :R], x[:, R:]
    return {"ckv": ckv.view(-1, bs, R), "kpe": kpe.view(-1, bs, D), "scales": scales.view(-1, bs // g)}


def exact_fresh(case, s):
    """exact() of a long write whose tokens each have a scale of their own, by whole requests; None for others."""
    q, bs, g = case["q"], case["bs"], case["g"]
    if g != 1:
        return None
    values = e4m3_table()
    ckv, kpe, scales = values[s["ckv"].view(-1, R).long()], values[s["kpe"].view(-1, D).long()], s["scales"].view(-1).double()
    for b, L in enumerate(lengths(case)):
        t = torch.arange(max(0, L - q), L, device="cuda")
        row = s["table"][b].long()[t // bs] * bs + t % bs
        x = torch.cat((s["ckv_new"][b], s["kpe_new"][b]), -1)[t - (L - q)].double()
        ladder = torch.exp2(torch.arange(MIN_EXP, MAX_EXP + 1, device="cuda").double())
        fits = x.abs().amax(-1)[:, None] / ladder <= E4M3_MAX
        size = ladder[fits.int().argmax(-1)]
        x = to_e4m3(x / size[:, None])
        ckv[row], kpe[row], scales[row] = x[:, :R], x[:, R:], size
    return {"ckv": ckv.view(-1, bs, R), "kpe": kpe.view(-1, bs, D), "scales": scales.view(-1, bs)}
