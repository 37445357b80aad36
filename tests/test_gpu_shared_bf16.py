"""Decode attention of a bf16 batch with a common prefix by the output's type: fp32 outputs keep the bounds that mla_decode's
fp32 results have, 16-bit ones those of weights rounded once."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu
MAX_ABS, REL_L2 = 2e-3, 1e-3  # of fp32 results, as everywhere

CASES = [([65], 64, 16, 1, 64, False, 1.0), ([300, 400], 256, 16, 1, 32, False, 0.5), ([40, 41], 32, 16, 1, 32, False, 1.0),
         ([300, 280, 290], 256, 16, 9, 32, True, 0.5), ([700, 513, 512, 600], 512, 64, 1, 32, False, 1.0), ([2100] * 9, 2048, 64, 2, 16, True, 0.5),
         ([150, 140, 0, 3], 128, 128, 2, 32, True, 1.0), ([64 * 33], 64 * 32, 128, 1, 64, False, 0.5), ([9000 + 50 * i for i in range(20)], 8192, 16, 1, 64, False, 1.0)]


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


def check_fp32(case, out, lse):
    """Scores off by ds as in test_gpu_shared's check. Weights as two bf16 terms: 2^-8 of themselves is what the first
    leaves, and the second leaves 2^-8 of that, 2^-16; else the same roundings. And the bounds of fp32 results."""
    ulp, diff, norm = 2.0 ** -23, 0.0, 0.0
    heads = sorted({0, case.H // 2, case.H - 1})
    for b in range(min(5, len(case.lens))):
        L = case.lens[b]
        row = case.rows_of(b, L)
        c, k = case.ckv.view(-1, 512)[row].double(), case.kpe.view(-1, 64)[row].double()
        seen = torch.full((case.q_len,), L, device="cuda")
        if case.causal:
            seen = (L - case.q_len + torch.arange(case.q_len, device="cuda") + 1).clamp(min=0)
        hidden = torch.arange(L, device="cuda")[None] >= seen[:, None]
        some = seen > 0
        for h in heads:
            q, qp = case.q_abs[b, :, h].double(), case.q_pe[b, :, h].double()
            got, got_lse = out[b, :, h].double(), lse[b, :, h].double()
            assert bool((got[~some] == 0).all()) and bool((got_lse[~some] == -math.inf).all())
            if not bool(some.any()):
                continue
            s = ((q @ c.T + qp @ k.T) * case.scale).masked_fill(hidden, -math.inf)[some]
            mags = abs(case.scale) * (q.abs() @ c.abs().T + qp.abs() @ k.abs().T)[some]
            ds = (576 * ulp * mags + 8 * ulp * s.abs()).masked_fill(hidden[some], 0).amax(1)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            want, size = p @ c, p @ c.abs()
            err = (got[some] - want).abs()
            assert bool((err <= (2.0 ** -16 + 2 * ds + 2.0 ** -19 + 2 * L * ulp)[:, None] * size).all()), (b, h, float(err.max()))
            assert float(err.max()) <= MAX_ABS
            diff += float(err.pow(2).sum())
            norm += float(want.pow(2).sum())
    assert math.sqrt(diff / norm) <= REL_L2, math.sqrt(diff / norm)


@pytest.mark.parametrize("lens,shared,H,q_len,bs,causal,size", CASES)
def test_fp32_outputs(lens, shared, H, q_len, bs, causal, size):
    case = Case(51 + H, lens, shared, H, q_len, bs, "bf16", causal, size=size)
    check_fp32(case, *case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,shared,H,q_len,bs,causal,size", CASES)
def test_16_bit_outputs(lens, shared, H, q_len, bs, causal, size, dtype):
    case = Case(52 + H, lens, shared, H, q_len, bs, dtype, causal, size=size)
    case.check(*case.run(out_dtype=dtype), requests=range(min(5, len(lens))), heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("lens,shared,H,q_len,bs,causal,size", CASES)
def test_fp16_outputs_are_the_fp32_ones_rounded_once(lens, shared, H, q_len, bs, causal, size):
    """They hold more than bf16 weights rounded once would leave them."""
    case = Case(56 + H, lens, shared, H, q_len, bs, "bf16", causal, size=size)
    plan = case.plan()
    out, lse = case.run(plan)
    half, half_lse = case.run(plan, "f16")
    assert torch.equal(half, out.half()) and torch.equal(half_lse, lse)


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_scores_that_rise(out_dtype):
    """Keys that grow along the tokens: the running maximum moves all the time, and weights reach far above 1."""
    case = Case(53, [900, 800, 1500], 640, 16, 2, 32, "bf16", True)
    for b, n in enumerate(case.lens):
        row = case.rows_of(b, n)[case.shared if b else 0:]
        case.ckv.view(-1, 512)[row] *= (torch.arange(len(row), device="cuda") / 400)[:, None].to(case.dtype)
    out, lse = case.run(out_dtype=out_dtype)
    if out_dtype == "f32":
        check_fp32(case, out, lse)
    else:
        case.check(out, lse)


def test_hidden_and_infinite_tokens_beside_16_bit_outputs():
    """What tests of fp32 outputs show of tokens that are not finite, of the other outputs."""
    case = Case(54, [300, 290], 256, 16, 4, 16, "bf16", True)
    want, want_lse = case.run(out_dtype="bf16")
    row = case.rows_of(0, 300)[298]  # seen by the rows 2 and 3 of request 0
    case.ckv.view(-1, 512)[row, 7] = float("nan")
    out, lse = case.run(out_dtype="bf16")
    assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(lse[0, :2], want_lse[0, :2])
    assert bool(out[0, 2:].isnan().all()) and torch.equal(out[1], want[1])
    case.ckv.view(-1, 512)[row, 7] = float("inf")
    case.q_abs[..., 7] = -case.q_abs[..., 7].abs().clamp(min=0.01)
    out, lse = case.run(out_dtype="bf16")
    column = torch.arange(512, device="cuda") == 7
    assert torch.equal(out[0, 2:].isnan(), column.expand(2, 16, 512)) and bool(torch.isfinite(lse).all())
    assert bool(torch.isfinite(out[0, :2]).all()) and bool(torch.isfinite(out[1]).all())


def test_the_same_bits_every_time_and_in_a_graph():
    case = Case(55, [3000 + 111 * i for i in range(12)], 2048, 64, 1, 64, "bf16")
    plan = case.plan()
    for out_dtype in ("f32", "bf16"):
        out, lse = case.run(plan, out_dtype)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            again, again_lse = case.run(plan, out_dtype)
        for _ in range(4):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, again) and torch.equal(lse, again_lse)
