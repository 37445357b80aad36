"""mla_decode_window on the GPU against the f64 oracle: windows, sinks, row counts of every CTA-pair kernel."""
import math

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from mla_split_kv_gb300 import runtime as rt
from oracle import mla_oracle as orc

pytestmark = pytest.mark.gpu
# the bounds stated for every fp32 result of these kernels
MAX_ABS, REL_L2 = 2e-3, 1e-3


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nbuild.build()
    nb.load()
    nb.mla_check_device_errors(None)
    yield
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK, f"device error word {code:#x}"


def make_plan(case, window, sinks, lens=None, **kw):
    return rt.plan_window((case.context_lens if lens is None else lens).tolist(), case.num_heads, case.q_len, case.block_size, window, sinks,
                          dtype=case.dtype, causal=case.causal, **kw)


def decode(case, dc, plan, dtype=torch.float32):
    shape = (case.num_requests, case.q_len, case.num_heads)
    out = torch.full(shape + (512,), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full(shape, float("nan"), device="cuda")
    rt.decode_window(plan, dc.q_abs, dc.q_pe, dc.ckv, dc.kpe, dc.block_table, dc.context_lens, case.scale, out, lse,
                     cache_scale=case.cache_scale)
    return out, lse


def oracle(case, window, sinks, heads):
    out, lse = [], []
    for b in range(case.num_requests):
        L = int(case.context_lens[b])
        rows = orc.physical_rows(case.block_table[b], L, case.block_size)
        c = orc.decode_cache(case.ckv.reshape(-1, 512)[rows], case)
        k = orc.decode_cache(case.kpe.reshape(-1, 64)[rows], case)
        qa, qp = (orc.decode16(x[b][:, heads], orc.query_dtype(case)) for x in (case.q_abs, case.q_pe))
        o, s = orc.attend_rows(qa, qp, c, k, case.scale, case.causal, window, sinks)
        out.append(o)
        lse.append(s)
    return np.stack(out), np.stack(lse)


def check(case, window, sinks, out, lse, heads):
    ref, ref_lse = oracle(case, window, sinks, heads)
    got, got_lse = out.double().cpu().numpy()[:, :, heads], lse.double().cpu().numpy()[:, :, heads]
    dead = np.isneginf(ref_lse)
    assert np.array_equal(dead, np.isneginf(got_lse)) and not got[dead].any()
    if dead.all():
        return
    assert np.abs(got_lse[~dead] - ref_lse[~dead]).max() <= MAX_ABS
    err = np.abs(got[~dead] - ref[~dead]).max()
    rel = np.linalg.norm(got[~dead] - ref[~dead]) / np.linalg.norm(ref[~dead])
    assert err <= MAX_ABS and rel <= REL_L2, (err, rel)


LENS = [0, 1, 40, 333, 2500, 5003]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (33, 0), (64, 1), (200, 70), (1500, 4), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("H,q_len,bs,dtype,causal", [
    (16, 1, 32, "f16", False),    # the paired 16-row kernel
    (16, 1, 16, "bf16", False),
    (16, 1, 64, "e4m3", False),
    (16, 4, 32, "f16", True),     # 64 rows: the 128-row kernel, half of it padding
    (64, 1, 16, "bf16", False),
    (128, 1, 64, "bf16", False),  # a full group
    (16, 9, 32, "bf16", True),    # 144 rows: a second, ragged group
    (16, 32, 64, "f16", True),
    (64, 2, 32, "e4m3", True),
])
def test_decode_window_against_the_oracle(window, sinks, H, q_len, bs, dtype, causal):
    case = gen.make_decode_case(61, LENS, num_heads=H, q_len=q_len, block_size=bs, dtype=dtype, latent_std=0.5, causal=causal)
    dc = rt.upload(case)
    out, lse = decode(case, dc, make_plan(case, window, sinks))
    heads = [0, H - 1] if q_len > 1 else [0, 7, H - 1]
    check(case, window, sinks, out, lse, heads)


@pytest.mark.parametrize("L,H,dtype", [(131072, 16, "f16"), (60000, 128, "bf16")])
@pytest.mark.parametrize("window", [1000, 40000])
def test_decode_window_split_runs(L, H, dtype, window):
    case = gen.make_decode_case(62, [L], num_heads=H, block_size=32, dtype=dtype, latent_std=0.5)
    plan = make_plan(case, window, 4)
    assert plan.plan.num_chunks * plan.plan.clusters_per_chunk > 1 or window < 4096
    out, lse = decode(case, rt.upload(case), plan)
    check(case, window, 4, out, lse, [0, H // 2])


@pytest.mark.parametrize("H,dtype", [(16, "f16"), (128, "bf16")])
def test_a_window_past_the_context_is_mla_decode_bit_for_bit(H, dtype):
    case = gen.make_decode_case(63, [5000, 700, 64], num_heads=H, block_size=32, dtype=dtype)
    dc = rt.upload(case)
    plan = make_plan(case, 5000, 0)
    out, lse = decode(case, dc, plan)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    p = plan.plan
    rt.decode(dc, plan.partials, plan.lse, plan.o_indptr, ref, ref_lse, chunks_dev=plan.chunks, kernel=nb.MLA_KERNEL_TC,
              cluster=p.cluster_ctas, subs=p.clusters_per_chunk, workspace=plan.workspace)
    assert torch.equal(out, ref)
    if dtype == "bf16":
        assert torch.equal(lse, ref_lse)
    else:  # mla_decode sums fp16 probabilities, each off by 2^-11 of itself at most; the windowed call the exact ones
        assert (lse - ref_lse).abs().max() <= math.log2(1 + 2.0 ** -11) + 2.0 ** -18
        check(case, 5000, 0, out, lse, [0, H // 2])


@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 4), (128, 1)])
@pytest.mark.parametrize("P,merge", [(1, 0), (3, 0), (3, 1)])
def test_decode_window_uniform_partitions_and_both_merges(H, q_len, P, merge):
    """No chunk table: the runs split into P; the paired kernel's two ways of merging."""
    case = gen.make_decode_case(64, [2500, 90, 0, 700], num_heads=H, q_len=q_len, block_size=32, dtype="f16", causal=q_len > 1)
    dc = rt.upload(case)
    B = case.num_requests
    part, lse_p = rt.alloc_partials(B * P, q_len, H)
    ws = rt.alloc_decode_workspace(B, B * P, 1, 2, q_len, H)
    d = rt.make_desc(dc, None, nb.MLA_KERNEL_AUTO, 2, workspace=ws, decode_merge=merge)
    out = torch.full((B, q_len, H, 512), float("nan"), device="cuda")
    lse = torch.full((B, q_len, H), float("nan"), device="cuda")
    ind = rt.uniform_indptr(B, P)
    nb.mla_decode_window(dc.q_abs.data_ptr(), dc.q_pe.data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                         dc.block_table.data_ptr(), dc.context_lens.data_ptr(), case.scale, P, part.data_ptr(),
                         lse_p.data_ptr(), ind.data_ptr(), out.data_ptr(), nb.MLA_F32, lse.data_ptr(), 500, 3, d)
    check(case, 500, 3, out, lse, [0, H - 1])


@pytest.mark.parametrize("H,q_len,dtype", [(16, 1, "f16"), (16, 1, "bf16"), (16, 4, "f16"), (16, 8, "bf16"), (64, 1, "f16"), (128, 1, "bf16"),
                                           (16, 1, "e4m3"), (64, 2, "e4m3")])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_decode_window_hides_non_finite_tokens(H, q_len, dtype, value):
    if dtype == "e4m3" and value == np.inf:
        pytest.skip("E4M3 has no infinity")
    causal = q_len > 1
    case = gen.make_decode_case(65, [1500, 333], num_heads=H, q_len=q_len, block_size=64, dtype=dtype, causal=causal)
    window, sinks = 200, 3
    dc = rt.upload(case)
    plan = make_plan(case, window, sinks)
    ref, ref_lse = decode(case, dc, plan)
    bad = np.uint8(0x7F) if dtype == "e4m3" else gen.to_bits(np.array(value), dtype)[()]
    for b in range(2):
        L = int(case.context_lens[b])
        seen = orc.visible_window(L, q_len, 0, causal, window, sinks)
        for t in np.flatnonzero(~seen):  # everything that row 0 does not see, drafts behind it among it
            page = case.block_table[b, t // 64]
            case.ckv[page, t % 64] = bad
            case.kpe[page, t % 64, ::2] = bad
        for t in range(L, -(-L // 64) * 64):
            case.ckv[case.block_table[b, t // 64], t % 64] = bad
    dc = rt.upload(case)
    out, lse = decode(case, dc, plan)
    assert torch.equal(out[:, 0], ref[:, 0]) and torch.equal(lse[:, 0], ref_lse[:, 0])


def test_decode_window_replayed_as_the_contexts_grow():
    """One plan for the longest runs, captured once; the contexts grow through two pages."""
    start, bs, window, sinks = [1000, 31, 0, 501], 32, 300, 5
    case = gen.make_decode_case(66, [L + 80 for L in start], num_heads=16, block_size=bs, dtype="f16")
    dc = rt.upload(case)
    dc.context_lens.copy_(torch.tensor(start, dtype=torch.int32))
    longest = max(nb.mla_window_lens(range(2000, 2000 + bs), 1, bs, False, window, sinks))
    plan = make_plan(case, window, sinks, lens=np.full(4, longest))
    out = torch.empty((4, 1, 16, 512), device="cuda")
    lse = torch.empty((4, 1, 16), device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        dc.context_lens += 1
        rt.decode_window(plan, dc.q_abs, dc.q_pe, dc.ckv, dc.kpe, dc.block_table, dc.context_lens, case.scale, out, lse)
    torch.cuda.synchronize()
    dc.context_lens.copy_(torch.tensor(start, dtype=torch.int32))
    for step in range(1, 72):
        graph.replay()
        torch.cuda.synchronize()
        if step % 5 == 0 or step < 3:
            case.context_lens = np.array([L + step for L in start], np.int32)
            check(case, window, sinks, out, lse, [0, 11])


def test_decode_window_16_bit_output_is_rounded_once():
    case = gen.make_decode_case(67, [3000, 100], num_heads=16, block_size=32, dtype="f16")
    dc = rt.upload(case)
    plan = make_plan(case, 600, 2)
    out, _ = decode(case, dc, plan)
    out16, _ = decode(case, dc, plan, torch.float16)
    assert torch.equal(out16, out.half())


def test_decode_window_refuses_wrong_tensors():
    case = gen.make_decode_case(68, [100], num_heads=16, block_size=32, dtype="f16")
    dc = rt.upload(case)
    plan = make_plan(case, 50, 0)
    out = torch.empty(1, 1, 16, 512, device="cuda")
    args = dict(q_abs=dc.q_abs, q_pe=dc.q_pe, ckv=dc.ckv, kpe=dc.kpe, block_table=dc.block_table, context_lens=dc.context_lens,
                scale=0.1, out=out)
    for bad in (dict(q_abs=dc.q_abs.bfloat16()), dict(ckv=dc.ckv[:, :16]), dict(kpe=dc.kpe[:2]), dict(out=out[:, :, :4]),
                dict(block_table=dc.block_table.long()), dict(context_lens=dc.context_lens.repeat(2))):
        with pytest.raises(ValueError):
            rt.decode_window(plan, **{**args, **bad})


@pytest.mark.parametrize("n", [1, 2, 33, 40])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_merges_of_many_rows_have_the_bits_of_few(n, out_dtype):
    """2048 rows and more are merged by a warp a row, fewer by four: request by request the same bits. Some parts
    have no mass, one request none at all."""
    B, H = 20, 128
    gen_t = torch.Generator(device="cuda").manual_seed(5)
    part = torch.randn(B * n, 1, H, 512, device="cuda", generator=gen_t)
    lse = 4 * torch.randn(B * n, 1, H, device="cuda", generator=gen_t)
    lse[::3, :, ::5] = -float("inf")
    lse[n:2 * n] = -float("inf")
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[out_dtype]

    def merge(lo, hi):
        out, out_lse = torch.empty(hi - lo, 1, H, 512, dtype=dt, device="cuda"), torch.empty(hi - lo, 1, H, device="cuda")
        nb.mla_merge_states(part[lo * n:].data_ptr(), lse[lo * n:].data_ptr(), rt.uniform_indptr(hi - lo, n).data_ptr(),
                            hi - lo, 1, H, out.data_ptr(), rt.CODE_OF[dt], out_lse.data_ptr(), None)
        torch.cuda.synchronize()
        return out, out_lse

    out, out_lse = merge(0, B)
    for b in range(B):
        one, one_lse = merge(b, b + 1)
        assert torch.equal(out[b], one[0]) and torch.equal(out_lse[b], one_lse[0])
    assert not out[1].any() and torch.isneginf(out_lse[1]).all()


@pytest.mark.parametrize("lens,P", [([700] * 20, 3), ([90, 0, 2500, 1] * 5, 1), ([4000] * 9, 2)])
def test_batches_of_16_rows_have_the_bits_of_their_requests(lens, P):
    """Eight requests and more with few entries each are merged by two warps a row, fewer requests by 32: the same
    bits. Uniform partitions, so a request's parts do not depend on its batch."""
    case = gen.make_decode_case(81, lens, num_heads=16, block_size=32, dtype="f16")
    dc = rt.upload(case)

    def run(lo, hi):
        B = hi - lo
        part, lse_p = rt.alloc_partials(B * P, 1, 16)
        ws = rt.alloc_decode_workspace(B, B * P, 1, 4, 1, 16)
        out, lse = torch.full((B, 1, 16, 512), float("nan"), device="cuda"), torch.full((B, 1, 16), float("nan"), device="cuda")
        d = rt.make_desc(dc, None, nb.MLA_KERNEL_TC, 4, workspace=ws)
        d.num_requests = B
        nb.mla_decode(dc.q_abs[lo:].data_ptr(), dc.q_pe[lo:].data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                      dc.block_table[lo:].data_ptr(), dc.context_lens[lo:].data_ptr(), case.scale, P, part.data_ptr(),
                      lse_p.data_ptr(), rt.uniform_indptr(B, P).data_ptr(), out.data_ptr(), nb.MLA_F32, lse.data_ptr(), d)
        torch.cuda.synchronize()
        return out, lse

    out, lse = run(0, len(lens))
    assert not torch.isnan(out).any()
    for b in range(0, len(lens), 3):
        one, one_lse = run(b, b + 1)
        assert torch.equal(out[b], one[0]) and torch.equal(lse[b], one_lse[0])


@pytest.mark.parametrize("H,q_len,dtype", [(16, 1, "f16"), (16, 1, "bf16"), (16, 1, "e4m3"), (64, 1, "f16"), (128, 1, "f16"), (16, 2, "e4m3")])
@pytest.mark.parametrize("lens", [[3, 40, 700], [5] * 12 + [900]])
def test_decode_window_lse_is_that_of_the_exact_probabilities(H, q_len, dtype, lens):
    """Few tokens a row, where a rounding of the greatest probability to fp16 would show: scores are sums of at most
    576 products, exact in fp32 and rounded at most 600 times on the way (2^-23 of the sum of magnitudes each), the
    exponentials and the sum a few units more; bf16 probabilities are kept in two terms (2^-16 of each)."""
    case = gen.make_decode_case(82, lens, num_heads=H, q_len=q_len, block_size=16, dtype=dtype)
    window, sinks = 6, 2
    out, lse = decode(case, rt.upload(case), make_plan(case, window, sinks))
    heads = [0, H - 1]
    _, ref = oracle(case, window, sinks, heads)
    got = lse.double().cpu().numpy()[:, :, heads]
    for b, L in enumerate(lens):
        rows = orc.physical_rows(case.block_table[b], L, 16)
        c = np.abs(orc.decode_cache(case.ckv.reshape(-1, 512)[rows], case))
        k = np.abs(orc.decode_cache(case.kpe.reshape(-1, 64)[rows], case))
        qa, qp = (np.abs(orc.decode16(x[b][:, heads], orc.query_dtype(case))) for x in (case.q_abs, case.q_pe))
        mag = case.scale * (np.einsum("ihr,tr->iht", qa, c) + np.einsum("ihr,tr->iht", qp, k)).max(-1)
        tol = 600 * 2.0 ** -23 * mag / math.log(2) + (2.0 ** -15 if dtype == "bf16" else 2.0 ** -18)
        fin = np.isfinite(ref[b])
        assert np.array_equal(fin, np.isfinite(got[b])) and np.all(np.abs(got[b] - ref[b])[fin] <= tol[fin])
