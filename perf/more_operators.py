"""Cases, plain forms and exact values of the operators around a prompt and a batch with a common prefix.

Five operators over the paged latent cache (512 latent and 64 rotary columns a token):

* ``update_tables``: a step's block tables, slot map and offsets from the requests' lengths and their changes,
  with pages taken from a pool of free ones and given back to it;
* ``append_slots``: the step's new tokens, packed one request after the other, written where the slot map says;
* ``expand_kv``: each head's keys and values (128 columns each) of cached tokens, from their latents;
* ``prefill``: causal attention of packed prompts, or of the newest tokens of longer contexts, over such keys and
  values and the rotary keys that all heads share;
* ``decode_shared``: absorbed attention of a batch whose contexts start with the same tokens, which are read and
  multiplied once for the batch.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, through the
package. ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

R, D, NOPE, VH = 512, 64, 128, 128  # columns: latent, rotary; of a head: keys without rotation, values
SCALE = 1.0 / math.sqrt(192.0)
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode step of a serving batch: every request one token further
        dict(name="tables decode step", op="update_tables", B=256, bs=32, lo=100, hi=8000, new=1, back=0.0, spare=0),
        # a step that takes prompts in, lets decoding requests go on and takes rejected or finished tokens back
        dict(name="tables mixed step", op="update_tables", B=512, bs=64, lo=0, hi=4000, new=2048, back=0.3, spare=4096),
        # the cache write of a small decode step
        dict(name="slots decode step", op="append_slots", T=24, bs=32, dtype="f16", joint=True, pad=8),
        # the cache write of packed prompts
        dict(name="slots packed prompts", op="append_slots", T=65536, bs=64, dtype="bf16", joint=True, pad=500),
        # a few short prompts on a 16-head rank
        dict(name="expand short prompts", op="expand_kv", B=4, lo=30, hi=600, H=16, bs=32, dtype="f16"),
        # one long document, all heads
        dict(name="expand long document", op="expand_kv", B=1, lo=16384, hi=16384, H=128, bs=64, dtype="bf16"),
        # one short question: latency
        dict(name="prefill short prompt", op="prefill", B=1, lo=300, hi=300, before=0, H=16, dtype="f16", joint=True),
        # prompts of all lengths, all heads
        dict(name="prefill ragged prompts", op="prefill", B=6, lo=300, hi=8192, before=0, H=128, dtype="bf16", joint=False),
        # the next chunk of two long documents
        dict(name="prefill behind context", op="prefill", B=2, lo=512, hi=1000, before=40000, H=16, dtype="f16", joint=True),
        # a few chats under one system prompt
        dict(name="shared few requests", op="decode_shared", B=4, H=16, q=1, prefix=2048, lo=1, hi=200, bs=32, dtype="f16", causal=False),
        # a serving batch of 16-head ranks under one long document
        dict(name="shared serving batch", op="decode_shared", B=64, H=16, q=1, prefix=32768, lo=50, hi=2000, bs=32, dtype="bf16", causal=False),
        # all heads, drafts being verified
        dict(name="shared many heads", op="decode_shared", B=24, H=128, q=2, prefix=8192, lo=100, hi=3000, bs=64, dtype="bf16", causal=True),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("update_tables", "append_slots", "expand_kv", "prefill", "prefill", "decode_shared", "decode_shared"))
    c = dict(op=op)
    dtype = rng.choice(("f16", "bf16"))
    if op == "update_tables":
        c["B"], c["bs"] = spread(rng, 1, 2000), rng.choice((16, 32, 64))
        c["lo"] = rng.choice((0, spread(rng, 1, 2000)))
        c["hi"] = c["lo"] + spread(rng, 1, 4000)
        c["new"] = rng.choice((1, 1, spread(rng, 2, max(3, 500000 // c["B"]))))
        c["back"] = rng.choice((0.0, 0.1, 0.5))
        c["spare"] = spread(rng, 1, 5000)
        return c
    if op == "append_slots":
        return dict(op=op, T=spread(rng, 1, 65536), bs=rng.choice((16, 32, 64)), dtype=dtype, joint=rng.random() < 0.5, pad=rng.choice((0, spread(rng, 1, 300))))
    c["H"] = rng.choice((8, 16, 16, 64, 128)) if op != "decode_shared" else rng.choice((16, 16, 64, 128))
    if op == "expand_kv":
        tokens = 2097152 // c["H"]
        c["B"] = spread(rng, 1, 32)
        c["hi"] = spread(rng, 1, max(1, tokens // c["B"]))
        c["lo"] = spread(rng, 1, c["hi"])
        return dict(c, bs=rng.choice((16, 32, 64)), dtype=dtype)
    if op == "prefill":
        pairs = int(6e9 / c["H"] / 4)  # of queries and keys, of the batch together
        c["B"] = spread(rng, 1, 16)
        c["before"] = rng.choice((0, 0, spread(rng, 1, 30000)))
        c["hi"] = spread(rng, 1, min(8192, max(1, pairs // c["B"] // (c["before"] + 1)), max(1, int(math.sqrt(pairs / c["B"])))))
        c["lo"] = spread(rng, 1, c["hi"])
        return dict(c, dtype=dtype, joint=rng.random() < 0.5)
    c["bs"] = rng.choice((16, 32, 64))
    c["q"] = rng.choice((1, 1, 1, spread(rng, 2, 16)))
    c["causal"] = c["q"] > 1
    c["B"] = spread(rng, 2, max(2, 3000 // (c["H"] * c["q"])))
    pairs = int(6e7 / (c["B"] * c["H"] * c["q"]))
    c["prefix"] = max(1, spread(rng, 64, max(65, min(65536, pairs))) // c["bs"]) * c["bs"]
    c["hi"] = max(c["q"], spread(rng, 1, 4000))
    c["lo"] = rng.randint(c["q"], c["hi"])
    return dict(c, dtype=dtype)


def lengths(case):
    """Per request: the tokens it has (update_tables), its cached tokens (expand_kv), its newest tokens (prefill), or
    the tokens it has for itself (decode_shared)."""
    r = random.Random(case["lo"] * 1000003 + case["hi"] * 101 + case["B"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[0] = case["hi"]
    return lens


def changes(case):
    """update_tables: how many tokens each request gets, or (negative) gives back."""
    r = random.Random(case["new"] * 31 + case["B"])
    lens = lengths(case)
    return [-r.randint(0, n) if r.random() < case["back"] else spread(r, 1, case["new"]) for n in lens]


def contexts(case):
    """prefill: the context lengths, the newest tokens among them."""
    r = random.Random(case["before"] + case["B"])
    return [n + (r.randint(case["before"] // 2, case["before"]) if case["before"] else 0) for n in lengths(case)]


def pages(n, bs):
    return -(-n // bs)


def work(case):
    op = case["op"]
    if op == "update_tables":
        lens, new = lengths(case), changes(case)
        moved = sum(abs(pages(a + n, case["bs"]) - pages(a, case["bs"])) for a, n in zip(lens, new))
        grown = sum(n for n in new if n > 0)
        return {"bytes": 4 * (3 * case["B"] + 2 * (case["B"] + 1)) + 8 * moved + 8 * (grown + case["spare"]), "flops": grown + 2 * case["B"]}
    if op == "append_slots":
        return {"bytes": case["T"] * (4 * (R + D) + 8) + 8 * case["pad"], "flops": case["T"]}
    H = case["H"]
    if op == "expand_kv":
        S = sum(lengths(case))
        return {"bytes": 2 * S * (R + 2 * D) + 2 * H * R * (NOPE + VH) + 2 * S * H * (NOPE + VH), "flops": 2 * S * R * H * (NOPE + VH)}
    if op == "prefill":
        new, ctx = lengths(case), contexts(case)
        T, S = sum(new), sum(ctx)
        pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(new, ctx))
        return {"bytes": 2 * T * H * (NOPE + D + VH) + 4 * T * H + 2 * S * (H * (NOPE + VH) + D), "flops": 2 * pairs * H * (NOPE + D + VH)}
    own_lens, q = lengths(case), case["q"]
    rows = case["B"] * q * H
    hidden = q * (q - 1) // 2 * H * case["B"] if case["causal"] else 0
    pairs = rows * case["prefix"] + q * H * sum(own_lens) - hidden
    return {"bytes": 2 * (R + D) * (case["prefix"] + sum(own_lens)) + rows * (2 * (R + D) + 2 * R + 4), "flops": 2 * pairs * (2 * R + D)}


def block_table(lens, bs, gen, spare, shared=0):
    """A block table over a shuffled pool (`shared` first pages are the same in every row; -1 behind each request's
    last page), and the pages that are left over."""
    need = [pages(n, bs) for n in lens]
    nb = shared + sum(need) + spare
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([shared + sum(need[:b]) for b in range(len(need))], device="cuda")[:, None]
    j = torch.arange(max(need), device="cuda")[None]
    held = j < torch.tensor(need, device="cuda")[:, None]
    rows = torch.where(held, perm[(at + j).clamp(max=nb - 1)], -1)
    return torch.cat((perm[:shared].expand(len(lens), shared), rows), 1).contiguous(), perm[shared + sum(need):].clone(), nb


def latents(gen, n, dtype):
    """Latents and rotary keys of n tokens: most tokens near unit size, some larger or smaller."""
    size = torch.exp2(torch.randn(n, 1, generator=gen, device="cuda")).clamp(2.0**-4, 2.0**2)
    c = torch.randn(n, R, generator=gen, device="cuda") * size
    k = torch.randn(n, D, generator=gen, device="cuda") * size
    return c.to(T16[dtype]), k.to(T16[dtype])


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def randn16(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(T16[dtype])


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "update_tables":
        lens, new, bs = lengths(case), changes(case), case["bs"]
        grown = sum(max(0, pages(a + n, bs) - pages(a, bs)) for a, n in zip(lens, new))
        freed = sum(max(0, pages(a, bs) - pages(a + n, bs)) for a, n in zip(lens, new))
        table, free, nb = block_table(lens, bs, gen, grown + 7)
        width = max(pages(a + max(n, 0), bs) for a, n in zip(lens, new)) + 2
        s["table"] = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1).contiguous()
        s["free"] = torch.full((nb,), -1, dtype=torch.int32, device="cuda")  # a stack: `count` pages, the next one last
        s["free"][: len(free)] = free
        s["count"] = torch.tensor([len(free)], dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["T"] = sum(n for n in new if n > 0) + case["spare"]
        assert freed + len(free) <= nb
        if own:
            from mla_split_kv_gb300 import runtime as rt
            s["pool"] = rt.PagePool(s["free"], s["count"], bs)
            s["step"] = rt.alloc_step(case["B"], s["T"])
        return s
    dtype = case["dtype"]
    if op == "append_slots":
        T, bs = case["T"], case["bs"]
        nb = pages(T, bs) + 9
        s["ckv"], s["kpe"] = (x.view(nb, bs, -1) for x in latents(gen, nb * bs, dtype))
        c, k = latents(gen, T + case["pad"], dtype)
        if case["joint"]:  # both of one projection's output
            both = torch.cat((c, k), 1)
            c, k = both[:, :R], both[:, R:]
        s["ckv_new"], s["kpe_new"] = c, k
        first = torch.randint(0, bs, (1,), generator=gen, device="cuda")
        perm = torch.randperm(nb, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda") + first
        s["slots"] = torch.nn.functional.pad(perm[t // bs] * bs + t % bs, (0, case["pad"]), value=-1)
        return s
    H = case["H"]
    if op == "expand_kv":
        lens, bs = lengths(case), case["bs"]
        s["table"], _, nb = block_table(lens, bs, gen, 5)
        s["ckv"], s["kpe"] = (x.view(nb, bs, -1) for x in latents(gen, nb * bs, dtype))
        s["kv_indptr"], s["S"] = offsets(lens), sum(lens)
        s["w_uk"] = (torch.randn(H, NOPE, R, generator=gen, device="cuda") / math.sqrt(R)).to(T16[dtype])
        s["w_uv_t"] = (torch.randn(H, R, VH, generator=gen, device="cuda") / math.sqrt(R)).to(T16[dtype])
        if own:
            s["k"], s["v"] = (torch.empty(s["S"], H, n, dtype=T16[dtype], device="cuda") for n in (NOPE, VH))
            s["k_pe"] = torch.empty(s["S"], D, dtype=T16[dtype], device="cuda")
        return s
    if op == "prefill":
        new, ctx = lengths(case), contexts(case)
        T, S = sum(new), sum(ctx)
        q = randn16(gen, dtype, T, H, NOPE + D)
        s["q_nope"], s["q_pe"] = (q[..., :NOPE], q[..., NOPE:]) if case["joint"] else (q[..., :NOPE].contiguous(), q[..., NOPE:].contiguous())
        s["k"] = randn16(gen, dtype, S, H, NOPE)
        s["v"] = randn16(gen, dtype, S, H, VH)
        s["k_pe"] = randn16(gen, dtype, S, D)
        s["q_indptr"], s["kv_indptr"] = offsets(new), offsets(ctx)
        if own:
            from mla_split_kv_gb300 import runtime as rt
            s["out"] = torch.empty(T, H, VH, dtype=T16[dtype], device="cuda")
            s["lse"] = torch.empty(T, H, device="cuda")
            s["plan"] = rt.plan_prefill(case["B"], H, T)
        return s
    lens, bs, q = lengths(case), case["bs"], case["q"]
    s["table"], _, nb = block_table(lens, bs, gen, 5, case["prefix"] // bs)
    s["ckv"], s["kpe"] = (x.view(nb, bs, -1) for x in latents(gen, nb * bs, dtype))
    total = [case["prefix"] + n for n in lens]
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["q_abs"], s["q_pe"] = randn16(gen, dtype, case["B"], q, H, R), randn16(gen, dtype, case["B"], q, H, D)
    if own:
        from mla_split_kv_gb300 import runtime as rt
        s["out"] = torch.empty(case["B"], q, H, R, dtype=T16[dtype], device="cuda")
        s["lse"] = torch.empty(case["B"], q, H, device="cuda")
        s["plan"] = rt.plan_shared(total, case["prefix"], H, q, bs, dtype=dtype, causal=case["causal"])
    return s


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"update_tables": tables_plain, "append_slots": append_plain, "expand_kv": expand_plain, "prefill": prefill_plain, "decode_shared": shared_plain}[op](s)
    from mla_split_kv_gb300 import runtime as rt
    if op == "update_tables":
        st = s["step"]
        rt.update_tables(s["pool"], s["new"], s["lens"], s["table"], st)
        return dict(lens=st.context_lens, table=s["table"], free=s["free"], count=st.free_count, q_indptr=st.q_indptr, kv_indptr=st.kv_indptr, slots=st.slots, served=st.served)
    if op == "append_slots":
        rt.cache_append_slots(s["ckv"], s["kpe"], s["ckv_new"], s["kpe_new"], s["slots"])
        return dict(ckv=s["ckv"], kpe=s["kpe"])
    if op == "expand_kv":
        rt.expand_kv(s["ckv"], s["kpe"], s["table"], s["kv_indptr"], s["w_uk"], s["w_uv_t"], s["k"], s["v"], s["k_pe"])
        return dict(k=s["k"], v=s["v"], k_pe=s["k_pe"])
    if op == "prefill":
        rt.prefill(s["plan"], s["q_nope"], s["q_pe"], s["k"], s["k_pe"], s["v"], s["q_indptr"], s["kv_indptr"], SCALE, s["out"], s["lse"])
    else:
        rt.decode_shared(s["plan"], s["q_abs"], s["q_pe"], s["ckv"], s["kpe"], s["table"], s["lens"], SCALE, s["out"], s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def tables_plain(s):
    """Pages given back go on the stack first, in the requests' order; growing requests then take theirs from its top,
    in their order, up to the first that does not fit (a page, a place in its row or a slot is missing)."""
    bs, width, T = s["case"]["bs"], s["table"].shape[1], s["T"]
    old, new = s["lens"].long(), torch.maximum(s["new"], -s["lens"]).long()
    held, want = (old + bs - 1) // bs, (old + new + bs - 1) // bs
    back, take = (held - want).clamp(min=0), (want - held).clamp(min=0)
    back_at, take_at, token_at = back.cumsum(0) - back, take.cumsum(0) - take, new.clamp(min=0).cumsum(0)
    j = torch.arange(width, device="cuda")[None]
    lost = (j >= want[:, None]) & (j < held[:, None])
    top = s["count"].long() + back.sum()
    s["free"][(s["count"].long() + back_at[:, None] + j - want[:, None])[lost]] = s["table"][lost]
    misfit = (new > 0) & ((take_at + take > top) | (want > width) | (token_at > T))
    ok = misfit.cumsum(0) == 0
    new = torch.where(ok, new, new.clamp(max=0))
    got = (j >= held[:, None]) & (j < want[:, None]) & ok[:, None]
    s["table"][got] = s["free"][(top - 1 - take_at[:, None] - j + held[:, None])[got]]
    lens, grown = old + new, new.clamp(min=0)
    q_indptr = torch.nn.functional.pad(grown.cumsum(0), (1, 0))
    kv_indptr = torch.nn.functional.pad(lens.cumsum(0), (1, 0))
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(q_indptr, i, right=True) - 1
    real = b < len(lens)
    b = b.clamp(max=len(lens) - 1)
    t = (old[b] + i - q_indptr[b]).clamp(max=width * bs - 1)
    slots = torch.where(real, s["table"][b, t // bs].long() * bs + t % bs, -1)
    served = ok.sum().int()[None]
    i32 = torch.int32
    return dict(lens=lens.to(i32), table=s["table"], free=s["free"], count=(top - torch.where(ok, take, 0).sum()).to(i32), q_indptr=q_indptr.to(i32), kv_indptr=kv_indptr.to(i32), slots=slots, served=served)


def append_plain(s):
    real = s["slots"] >= 0
    at = s["slots"][real]
    s["ckv"].view(-1, R)[at] = s["ckv_new"][real]
    s["kpe"].view(-1, D)[at] = s["kpe_new"][real]
    return dict(ckv=s["ckv"], kpe=s["kpe"])


def packed_rows(s):
    """Cache rows of the requests' tokens, one request after the other."""
    bs, at = s["case"]["bs"], s["kv_indptr"].long()
    i = torch.arange(s["S"], device="cuda")
    b = torch.searchsorted(at, i, right=True) - 1
    t = i - at[b]
    return s["table"][b, t // bs].long() * bs + t % bs


def expand_plain(s):
    row, dtype = packed_rows(s), T16[s["case"]["dtype"]]
    H = s["case"]["H"]
    c = s["ckv"].view(-1, R)[row].float()
    k = (c @ s["w_uk"].float().flatten(0, 1).T).to(dtype).view(-1, H, NOPE)
    v = (c @ s["w_uv_t"].float().transpose(0, 1).flatten(1)).to(dtype).view(-1, H, VH)
    return dict(k=k, v=v, k_pe=s["kpe"].view(-1, D)[row])


def prefill_plain(s):
    """Request by request, as many heads at once as the scores fit in eight gigabytes."""
    case = s["case"]
    H, dtype = case["H"], T16[case["dtype"]]
    new, ctx = lengths(case), contexts(case)
    out = torch.empty(sum(new), H, VH, dtype=dtype, device="cuda")
    lse = torch.empty(sum(new), H, device="cuda")
    q0 = k0 = 0
    for n, c in zip(new, ctx):
        hidden = torch.arange(c, device="cuda")[None] > (torch.arange(n, device="cuda") + (c - n))[:, None]
        step = max(1, 2**31 // (n * c))
        for h in range(0, H, step):
            hs = slice(h, h + step)
            qn, qp = s["q_nope"][q0:q0 + n, hs].float().transpose(0, 1), s["q_pe"][q0:q0 + n, hs].float().transpose(0, 1)
            k, v = s["k"][k0:k0 + c, hs].float().transpose(0, 1), s["v"][k0:k0 + c, hs].float().transpose(0, 1)
            score = (qn @ k.mT + qp @ s["k_pe"][k0:k0 + c].float().T) * SCALE
            score.masked_fill_(hidden, float("-inf"))
            m = score.amax(-1, keepdim=True)
            p = score.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            out[q0:q0 + n, hs] = (p @ v / total).transpose(0, 1).to(dtype)
            lse[q0:q0 + n, hs] = (m + torch.log(total))[..., 0].T / math.log(2.0)
        q0, k0 = q0 + n, k0 + c
    return dict(out=out, lse=lse)


def shared_plain(s):
    """The scores of all rows over the common tokens as one product, those over each request's own beside them."""
    case = s["case"]
    B, q, H, bs, P = case["B"], case["q"], case["H"], case["bs"], case["prefix"]
    ckv, kpe = s["ckv"].view(-1, R), s["kpe"].view(-1, D)
    L = s["lens"].long()
    n = max(lengths(case))
    t = P + torch.arange(n, device="cuda")[None].expand(B, n)
    row = s["table"].long().gather(1, (t // bs).clamp(max=s["table"].shape[1] - 1)).clamp(min=0) * bs + t % bs
    t0 = torch.arange(P, device="cuda")
    first = s["table"][0].long()[t0 // bs] * bs + t0 % bs
    c0, k0, c1, k1 = ckv[first].float(), kpe[first].float(), ckv[row].float(), kpe[row].float()
    qa, qp = s["q_abs"].float().flatten(1, 2), s["q_pe"].float().flatten(1, 2)
    score = torch.cat((qa @ c0.T + qp @ k0.T, qa @ c1.mT + qp @ k1.mT), -1) * SCALE
    pos = L[:, None] - q + torch.arange(q, device="cuda") if case["causal"] else (L[:, None] - 1).expand(B, q)
    every = torch.cat((t0[None].expand(B, P), t), 1)
    score = score.unflatten(1, (q, H)).masked_fill(~(every[:, None] <= pos[..., None])[:, :, None], float("-inf"))
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    p = p.flatten(1, 2)
    out = (p[..., :P] @ c0 + p[..., P:] @ c1).unflatten(1, (q, H)) / total
    return dict(out=out.to(T16[case["dtype"]]), lse=(m + torch.log(total))[..., 0] / math.log(2.0))


def exact(case, seed):
    op = case["op"]
    if op == "prefill" and sum(n * c for n, c in zip(lengths(case), contexts(case))) * case["H"] > 4e10:
        return None
    s = prepare(case, seed)
    return {"update_tables": tables_exact, "append_slots": append_exact, "expand_kv": expand_exact, "prefill": prefill_exact, "decode_shared": shared_exact}[op](s)


def tables_exact(s):
    """The step request by request on the host."""
    case = s["case"]
    bs, T = case["bs"], s["T"]
    table, free = s["table"].tolist(), s["free"].tolist()
    width, lens, count = len(table[0]), list(lengths(case)), int(s["count"])
    new = [max(n, -a) for n, a in zip(changes(case), lens)]
    for b, n in enumerate(new):
        for j in range(pages(lens[b] + n, bs), pages(lens[b], bs)) if n < 0 else ():
            free[count] = table[b][j]
            count += 1
        lens[b] += min(n, 0)
    served, slots, q_indptr = len(lens), [], [0]
    for b, n in enumerate(new):
        before = pages(lens[b], bs)
        take = pages(lens[b] + n, bs) - before if n > 0 else 0
        if n > 0 and served == len(lens) and (take > count or before + take > width or len(slots) + n > T):
            served = b
        if n > 0 and b < served:
            for j in range(take):
                count -= 1
                table[b][before + j] = free[count]
            slots += [table[b][t // bs] * bs + t % bs for t in range(lens[b], lens[b] + n)]
            lens[b] += n
        q_indptr.append(len(slots))
    kv_indptr = [0]
    for n in lens:
        kv_indptr.append(kv_indptr[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(lens=i32(lens), table=i32(table), free=i32(free), count=i32([count]), q_indptr=i32(q_indptr), kv_indptr=i32(kv_indptr),
                slots=torch.tensor(slots + [-1] * (T - len(slots)), device="cuda"), served=i32([served]))


def append_exact(s):
    """The copy, page after page: every row of the cache is some token's, or what it was."""
    bs = s["case"]["bs"]
    rows = s["ckv"].shape[0] * bs
    source = torch.full((rows + 1,), -1, device="cuda")
    source.scatter_(0, torch.where(s["slots"] < 0, rows, s["slots"]), torch.arange(len(s["slots"]), device="cuda"))
    source = source[:rows, None]
    pick = lambda old, new: torch.where(source >= 0, new.double()[source[:, 0].clamp(min=0)], old.flatten(0, 1).double()).view(old.shape)  # noqa: E731
    return dict(ckv=pick(s["ckv"], s["ckv_new"]), kpe=pick(s["kpe"], s["kpe_new"]))


def expand_exact(s):
    bs, lens = s["case"]["bs"], lengths(s["case"])
    c, k_pe = [], []
    for b, n in enumerate(lens):
        ids = s["table"][b, : pages(n, bs)].long()
        c.append(s["ckv"][ids].flatten(0, 1)[:n].double())
        k_pe.append(s["kpe"][ids].flatten(0, 1)[:n].double())
    c = torch.cat(c)
    return dict(k=torch.einsum("tr,hdr->thd", c, s["w_uk"].double()), v=torch.einsum("tr,hrd->thd", c, s["w_uv_t"].double()), k_pe=torch.cat(k_pe))


def prefill_exact(s):
    """By blocks of queries of one request and one head at a time, over no more keys than the block's last query sees."""
    case = s["case"]
    H = case["H"]
    T = int(s["q_indptr"][-1])
    out, lse = torch.zeros(T, H, VH, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n, c in zip(lengths(case), contexts(case)):
        block = min(n, max(64, 2**27 // c))
        for i in range(0, n, block):
            e = min(n, i + block)
            seen = c - n + e
            far = torch.arange(seen, device="cuda") - (c - n + torch.arange(i, e, device="cuda"))[:, None] > 0
            k_pe = s["k_pe"][k0:k0 + seen].double()
            for h in range(H):
                keys = torch.cat((s["k"][k0:k0 + seen, h].double(), k_pe), 1)
                queries = torch.cat((s["q_nope"][q0 + i:q0 + e, h], s["q_pe"][q0 + i:q0 + e, h]), 1).double()
                score = torch.mm(queries, keys.T).mul_(SCALE)
                score[far] = -math.inf
                total = torch.logsumexp(score, 1)
                lse[q0 + i:q0 + e, h] = total / math.log(2.0)
                out[q0 + i:q0 + e, h] = torch.exp(score - total[:, None]) @ s["v"][k0:k0 + seen, h].double()
        q0, k0 = q0 + n, k0 + c
    return dict(out=out, lse=lse)


def shared_exact(s):
    """Request by request, each over the whole of its own context."""
    case = s["case"]
    q, H, bs = case["q"], case["H"], case["bs"]
    out, lse = [], []
    for b, n in enumerate(lengths(case)):
        L = case["prefix"] + n
        ids = s["table"][b, : pages(L, bs)].long()
        c, k = (x[ids].flatten(0, 1)[:L].double() for x in (s["ckv"], s["kpe"]))
        score = SCALE * (torch.einsum("ihr,tr->iht", s["q_abs"][b].double(), c) + torch.einsum("ihr,tr->iht", s["q_pe"][b].double(), k))
        if case["causal"]:
            later = torch.arange(L, device="cuda")[None] > (L - q + torch.arange(q, device="cuda"))[:, None]
            score[later[:, None].expand(q, H, L)] = -math.inf
        total = torch.logsumexp(score, -1)
        lse.append(total / math.log(2.0))
        out.append(torch.einsum("iht,tr->ihr", torch.exp(score - total[..., None]), c))
    return dict(out=torch.stack(out), lse=torch.stack(lse))
