"""mla_decode_window with each score exchange that a caller may choose (more than 16 rows), and the LSE of each way."""
import math

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from mla_split_kv_gb300 import runtime as rt
from oracle import mla_oracle as orc
from tests.test_gpu_window import check, oracle

pytestmark = pytest.mark.gpu
F16, NONE, F32 = nb.MLA_SCORE_EXCHANGE_F16, nb.MLA_SCORE_EXCHANGE_NONE, nb.MLA_SCORE_EXCHANGE_F32


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


def decode(case, dc, window, sinks, exchange=0, P=3, merge=0):
    """Uniform partitions of the visible runs, the exchange as the descriptor has it."""
    B, q_len, H = case.num_requests, case.q_len, case.num_heads
    part, lse_p = rt.alloc_partials(B * P, q_len, H)
    ws = rt.alloc_decode_workspace(B, B * P, 1, 2, q_len, H)
    d = rt.make_desc(dc, None, nb.MLA_KERNEL_AUTO, 2, workspace=ws, decode_merge=merge, score_exchange=exchange)
    out = torch.full((B, q_len, H, 512), float("nan"), device="cuda")
    lse = torch.full((B, q_len, H), float("nan"), device="cuda")
    ind = rt.uniform_indptr(B, P)
    nb.mla_decode_window(dc.q_abs.data_ptr(), dc.q_pe.data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                         dc.block_table.data_ptr(), dc.context_lens.data_ptr(), case.scale, P, part.data_ptr(),
                         lse_p.data_ptr(), ind.data_ptr(), out.data_ptr(), nb.MLA_F32, lse.data_ptr(), window, sinks, d)
    return out, lse


WAYS = [(dtype, x) for dtype in ("f16", "bf16") for x in (F16, NONE, F32)] + [("e4m3", F16), ("e4m3", F32)]


@pytest.mark.parametrize("dtype,exchange", WAYS)
@pytest.mark.parametrize("window,sinks", [(33, 0), (200, 70), (1500, 4)])
@pytest.mark.parametrize("H,q_len", [(64, 1), (16, 9), (128, 1)])
def test_windows_under_every_exchange(H, q_len, window, sinks, dtype, exchange):
    case = gen.make_decode_case(61, [0, 1, 333, 2500, 5003], num_heads=H, q_len=q_len, block_size=32, dtype=dtype,
                                latent_std=0.5, causal=q_len > 1)
    out, lse = decode(case, rt.upload(case), window, sinks, exchange)
    check(case, window, sinks, out, lse, [0, H - 1])


@pytest.mark.parametrize("dtype,exchange", WAYS)
def test_hidden_tokens_reach_no_row_under_any_exchange(dtype, exchange):
    window, sinks, q_len = 200, 3, 5
    case = gen.make_decode_case(65, [1500, 333], num_heads=16, q_len=q_len, block_size=64, dtype=dtype, causal=True)
    ref, ref_lse = decode(case, rt.upload(case), window, sinks, exchange)
    bad = np.uint8(0x7F) if dtype == "e4m3" else gen.to_bits(np.array(np.nan), dtype)[()]
    for b in range(2):
        L = int(case.context_lens[b])
        for t in np.flatnonzero(~orc.visible_window(L, q_len, 0, True, window, sinks)):
            page = case.block_table[b, t // 64]
            case.ckv[page, t % 64] = bad
            case.kpe[page, t % 64, ::2] = bad
    out, lse = decode(case, rt.upload(case), window, sinks, exchange)
    assert torch.equal(out[:, 0], ref[:, 0]) and torch.equal(lse[:, 0], ref_lse[:, 0])


def lse_error(case, lse, window, sinks):
    """The LSE's error over what the exact probabilities' may be off: scores of at most 576 products, exact in fp32 and
    rounded at most 600 times on the way (2^-23 of the sum of magnitudes each), the exponentials and the sum a few
    units more; bf16 probabilities are kept in two terms (2^-16 of each). Also the magnitudes, in log2 units."""
    heads = [0, case.num_heads - 1]
    _, ref = oracle(case, window, sinks, heads)
    got = lse.double().cpu().numpy()[:, :, heads]
    mags = []
    for b in range(case.num_requests):
        rows = orc.physical_rows(case.block_table[b], int(case.context_lens[b]), case.block_size)
        c = np.abs(orc.decode_cache(case.ckv.reshape(-1, 512)[rows], case))
        k = np.abs(orc.decode_cache(case.kpe.reshape(-1, 64)[rows], case))
        qa, qp = (np.abs(orc.decode16(x[b][:, heads], orc.query_dtype(case))) for x in (case.q_abs, case.q_pe))
        mags.append((np.einsum("ihr,tr->iht", qa, c) + np.einsum("ihr,tr->iht", qp, k)).max(-1))
    mag = case.scale * np.stack(mags) / math.log(2)
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(got))
    tol = 600 * 2.0 ** -23 * mag + (2.0 ** -15 if case.dtype == "bf16" else 2.0 ** -18)
    return np.abs(got - ref)[fin], tol[fin], mag[fin]


@pytest.mark.parametrize("dtype,exchange", WAYS)
def test_the_lse_is_that_of_the_exact_probabilities_under_every_exchange(dtype, exchange):
    """An fp16 exchange rounds each half's part of a score to 2^-11 of it at most, together 2^-11 of the magnitudes."""
    case = gen.make_decode_case(82, [3, 40, 700], num_heads=64, block_size=16, dtype=dtype)
    _, lse = decode(case, rt.upload(case), 6, 2, exchange, P=1)
    err, tol, mag = lse_error(case, lse, 6, 2)
    assert np.all(err <= tol + (2.0 ** -11 * mag if exchange == F16 else 0.0))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
def test_the_ticket_way_s_lse_is_that_of_the_rounded_probabilities(dtype):
    """16 rows in one launch: fp16 probabilities (also those beside E4M3 caches) are each off by 2^-11 of themselves at
    most, and the LSE is that of their sum."""
    case = gen.make_decode_case(83, [3, 40, 700], num_heads=16, block_size=16, dtype=dtype)
    _, lse = decode(case, rt.upload(case), 6, 2, P=1, merge=nb.MLA_DECODE_MERGE_TICKETS)
    err, tol, _ = lse_error(case, lse, 6, 2)
    assert np.all(err <= tol + (0.0 if dtype == "bf16" else -math.log2(1 - 2.0 ** -11)))
