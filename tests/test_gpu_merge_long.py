"""Batches of 16 rows in which a few requests have many parts: the same bits as each request by itself, in about the
time of a batch without the rest."""
import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from mla_split_kv_gb300 import runtime as rt

pytestmark = pytest.mark.gpu


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


class Batch:
    """Requests of `parts[b]` chunks of `tokens` tokens each (0: no token, one empty chunk)."""

    def __init__(self, parts, tokens=32, dtype="f16"):
        self.parts, self.tokens, self.dtype = parts, tokens, dtype
        self.case = gen.make_decode_case(51, [n * tokens for n in parts], num_heads=16, block_size=32, dtype=dtype)
        self.dc = rt.upload(self.case)

    def call(self, lo, hi, merge=0, tables_ready=False):
        """The buffers of a call on requests [lo, hi), and what makes it."""
        B, dc = hi - lo, self.dc
        rows, indptr = [], [0]
        for b in range(B):
            n = self.parts[lo + b]
            for k in range(max(1, n)):
                rows.append((b, k * self.tokens, (k + 1) * self.tokens if n else 0, len(rows)))
            indptr.append(len(rows))
        part, lse_p = rt.alloc_partials(len(rows), 1, 16)
        ws = rt.alloc_decode_workspace(B, len(rows), 1, 2, 1, 16)
        ws.view(torch.uint8).fill_(0xFF if merge == 0 else 0)
        out, lse = torch.full((B, 1, 16, 512), float("nan"), device="cuda"), torch.full((B, 1, 16), float("nan"), device="cuda")
        chunks, ind = rt.chunks_to_device(rows), torch.tensor(indptr, dtype=torch.int32, device="cuda")
        keep = (part, lse_p, ws, chunks, ind)

        def go():
            d = rt.make_desc(dc, chunks, nb.MLA_KERNEL_TC, 2, workspace=ws, decode_merge=merge, tables_ready=tables_ready)
            d.num_requests = B
            nb.mla_decode(dc.q_abs[lo:].data_ptr(), dc.q_pe[lo:].data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                          dc.block_table[lo:].data_ptr(), dc.context_lens[lo:].data_ptr(), self.case.scale, 0, part.data_ptr(),
                          lse_p.data_ptr(), ind.data_ptr(), out.data_ptr(), nb.MLA_F32, lse.data_ptr(), d)

        return go, out, lse, keep

    def run(self, lo, hi, **kw):
        go, out, lse, _ = self.call(lo, hi, **kw)
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        return out, lse


@pytest.mark.parametrize("parts", [
    [1, 1, 9, 1, 1, 1, 1, 1],
    [2, 12, 1, 13, 0, 1, 1, 1],
    [1] * 5 + [33] + [1] * 6,
    [64] + [1] * 11,
    [1] * 11 + [97],                                     # more than one round of 96
    [1, 130, 0] + [1] * 13,
    [40, 1, 1, 24, 1, 1, 1, 16] + [1] * 8,               # several
    [20] + [1] * 126 + [14, 33] + [0] * 20 + [25],       # far apart in a large batch
])
@pytest.mark.parametrize("tables_ready", [False, True])
def test_requests_of_many_parts_have_the_bits_of_their_own_call(parts, tables_ready):
    batch = Batch(parts)
    B = len(parts)
    assert B * 16 >= 128 and sum(max(1, n) for n in parts) <= 12 * B
    out, lse = batch.run(0, B, tables_ready=tables_ready)
    for b in range(B):
        if B > 20 and parts[b] <= 1 and b % 9:
            continue
        one, one_lse = batch.run(b, b + 1)
        assert torch.equal(out[b], one[0]) and torch.equal(lse[b], one_lse[0]), b
    assert not torch.isnan(out).any()


def microseconds(batch, hi, calls=20):
    go, _, _, keep = batch.call(0, hi, tables_ready=True)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            go()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(20):
        graph.replay()
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) / calls * 1e3)
    del keep
    return best


def test_a_request_of_many_parts_does_not_slow_its_batch():
    """64 parts beside six and seven requests of one: the eighth request (which takes the batch to 128 rows) changes
    how short requests are merged, not the long one. (Merged as short ones are, its 64 parts were eight rounds of
    loads one behind the other, twice.)"""
    batch = Batch([64] + [1] * 7, tokens=128)
    seven, eight = microseconds(batch, 7), microseconds(batch, 8)
    assert eight <= 1.2 * seven, (seven, eight)


def merge_microseconds(parts, rows=128, calls=20):
    """Device time of a merge of partials over `rows` rows a request, calls back to back."""
    n = sum(parts)
    r = torch.Generator(device="cuda").manual_seed(3)
    part, lse = torch.randn(n, 1, rows, 512, device="cuda", generator=r), torch.randn(n, 1, rows, device="cuda", generator=r)
    ind = torch.tensor(np.concatenate([[0], np.cumsum(parts)]), dtype=torch.int32, device="cuda")
    out, out_lse = torch.empty(len(parts), 1, rows, 512, device="cuda"), torch.empty(len(parts), 1, rows, device="cuda")

    def go():
        nb.mla_merge_states(part.data_ptr(), lse.data_ptr(), ind.data_ptr(), len(parts), 1, rows, out.data_ptr(), nb.MLA_F32,
                            out_lse.data_ptr(), torch.cuda.current_stream().cuda_stream)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            go()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(20):
        graph.replay()
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) / calls * 1e3)
    return best


def test_a_request_of_many_partials_does_not_slow_a_merge_of_many_rows():
    """2048 rows are merged with fewer warps a row than 1920 are; a request of 76 partials among them must not wait
    for that."""
    few, many = merge_microseconds([76] + [2] * 14), merge_microseconds([76] + [2] * 15)
    assert many <= 1.3 * few, (few, many)


@pytest.mark.parametrize("parts", [[76] + [2] * 15, [1, 33, 0, 8, 9, 17, 40, 64, 65] + [3] * 11])
def test_merges_of_many_rows_with_a_long_request_have_the_bits_of_few(parts):
    B, rows, n = len(parts), 128, sum(parts)
    r = torch.Generator(device="cuda").manual_seed(4)
    part, lse = torch.randn(n, 1, rows, 512, device="cuda", generator=r), 4 * torch.randn(n, 1, rows, device="cuda", generator=r)
    lse[::5, :, ::3] = -float("inf")
    at = np.concatenate([[0], np.cumsum(parts)])

    def merge(lo, hi):
        out, out_lse = torch.empty(hi - lo, 1, rows, 512, device="cuda"), torch.empty(hi - lo, 1, rows, device="cuda")
        ind = torch.tensor(at[lo:hi + 1], dtype=torch.int32, device="cuda")
        nb.mla_merge_states(part.data_ptr(), lse.data_ptr(), ind.data_ptr(), hi - lo, 1, rows, out.data_ptr(), nb.MLA_F32,
                            out_lse.data_ptr(), None)
        torch.cuda.synchronize()
        return out, out_lse

    out, out_lse = merge(0, B)
    for b in range(B):
        one, one_lse = merge(b, b + 1)
        assert torch.equal(out[b], one[0]) and torch.equal(out_lse[b], one_lse[0]), b
