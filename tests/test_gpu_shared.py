"""Decode attention of a batch with a common prefix, against the definition in 64 bits."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
TDT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


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


class Case:
    """Contexts lens[b] (the common `shared` tokens among them); what lies in the pool behind a context is NaN."""

    def __init__(self, seed, lens, shared, H=16, q_len=1, bs=32, dtype="f16", causal=False, scale=SCALE, room=0, size=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.shared, self.H, self.q_len, self.bs, self.dt, self.dtype = list(lens), shared, H, q_len, bs, dtype, TDT[dtype]
        self.causal, self.scale, B = causal, scale, len(lens)
        own = [max(0, -(-(n + room) // bs) - shared // bs) for n in lens]
        nblk = shared // bs + sum(own) + 3
        perm = torch.randperm(nblk, device="cuda", generator=g).int()
        self.shared_table = perm[: shared // bs].clone()
        self.table = torch.full((B, shared // bs + max(own)), -1, dtype=torch.int32, device="cuda")
        at = shared // bs
        for b, n in enumerate(own):
            self.table[b, shared // bs:shared // bs + n] = perm[at:at + n]
            at += n
        rand = lambda *s: (torch.randn(*s, device="cuda", generator=g) * size).to(self.dtype)  # noqa: E731
        self.ckv, self.kpe = rand(nblk, bs, 512), rand(nblk, bs, 64)
        self.nan_behind()
        self.q_abs, self.q_pe = rand(B, q_len, H, 512), rand(B, q_len, H, 64)
        self.ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows_of(self, b, n):
        t = torch.arange(n, device="cuda")
        pages = torch.cat((self.shared_table, self.table[b, self.shared // self.bs:])).long()
        return pages[t // self.bs] * self.bs + t % self.bs

    def nan_behind(self):
        """NaN in every row of the pool that is no request's token."""
        used = torch.zeros(self.ckv.shape[0] * self.bs, dtype=torch.bool, device="cuda")
        for b, n in enumerate(self.lens):
            used[self.rows_of(b, n)] = True
        self.ckv.view(-1, 512)[~used] = float("nan")
        self.kpe.view(-1, 64)[~used] = float("nan")

    def plan(self, lens=None):
        return rt.plan_shared(self.lens if lens is None else lens, self.shared, self.H, self.q_len, self.bs, dtype=self.dt, causal=self.causal)

    def run(self, plan=None, out_dtype="f32", **kw):
        shape = (len(self.lens), self.q_len, self.H)
        out = torch.full((*shape, 512), float("nan"), dtype=TDT[out_dtype], device="cuda")
        lse = torch.full(shape, float("nan"), device="cuda")
        rt.decode_shared(plan or self.plan(), self.q_abs, self.q_pe, self.ckv, self.kpe, self.table, self.ctx, self.scale, out, lse,
                         shared_table=self.shared_table, **kw)
        return out, lse

    def check(self, out, lse, requests=None, heads=None):
        """Scores: 576 products, exact in fp32, added with at most 2^-23 of the sum of their magnitudes lost each time,
        and a few roundings on the way into the exponential: off by ds. Weights: a factor exp(ds) in the numerator and
        in the sum, half a step of the cache's type (fp16: at least 2^-25, of weights whose greatest is at least 1), and
        2^-19 for the exponentials, the sums' and the merge's roundings beside the tokens' own. A 16-bit output is
        rounded by half a step once more."""
        half, ulp = torch.finfo(self.dtype).eps / 2, 2.0 ** -23
        for b in range(len(self.lens)) if requests is None else requests:
            L = self.lens[b]
            row = self.rows_of(b, L)
            c, k = self.ckv.view(-1, 512)[row].double(), self.kpe.view(-1, 64)[row].double()
            for h in range(self.H) if heads is None else heads:
                q, qp = self.q_abs[b, :, h].double(), self.q_pe[b, :, h].double()
                s = (q @ c.T + qp @ k.T) * self.scale
                mags = abs(self.scale) * (q.abs() @ c.abs().T + qp.abs() @ k.abs().T)
                seen = torch.full((self.q_len,), L, device="cuda")
                if self.causal:
                    seen = (L - self.q_len + torch.arange(self.q_len, device="cuda") + 1).clamp(min=0)
                hidden = torch.arange(L, device="cuda")[None] >= seen[:, None]
                got, got_lse = out[b, :, h].double(), lse[b, :, h].double()
                empty = seen == 0
                assert bool((got[empty] == 0).all()) and bool((got_lse[empty] == -math.inf).all()), (b, h)
                if bool(empty.all()):
                    continue
                s, mags, hidden, got, got_lse = (x[~empty] for x in (s, mags, hidden, got, got_lse))
                s = s.masked_fill(hidden, -math.inf)
                ds = (576 * ulp * mags + 8 * ulp * s.abs()).masked_fill(hidden, 0).amax(1)
                z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                want, size = p @ c, p @ c.abs()
                tol = (half + 2 * ds + 2.0 ** -19 + 2 * L * ulp)[:, None] * size
                if self.dtype == torch.float16:
                    tol = tol + L * 2.0 ** -25 * c.abs().amax()
                if out.dtype != torch.float32:
                    tol = tol + torch.finfo(out.dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
                err = (got - want).abs()
                assert bool((err <= tol).all()), (b, h, float((err - tol).max()), float(err.max()))
                lse_tol = (ds + L * ulp + 2.0 ** -19) / math.log(2.0) + 4 * ulp * z.abs() / math.log(2.0)
                assert bool(((got_lse - z / math.log(2.0)).abs() <= lse_tol).all()), (b, h)


@pytest.mark.parametrize("lens,shared,H,q_len,bs,dtype,causal", [
    ([65], 64, 16, 1, 64, "f16", False), ([40, 41], 32, 16, 1, 32, "bf16", False), ([100, 64, 300], 64, 16, 1, 16, "f16", False),
    ([700, 513, 512, 600], 512, 64, 1, 32, "bf16", False), ([200, 130], 128, 128, 1, 64, "f16", False), ([2000] * 9, 1600, 16, 1, 32, "bf16", False),
    ([300, 260, 257], 256, 16, 2, 16, "f16", True), ([300, 280, 290], 256, 16, 9, 32, "bf16", True), ([200, 170], 128, 64, 3, 64, "f16", True),
    ([150, 140], 128, 128, 2, 32, "bf16", True), ([400], 320, 16, 32, 16, "f16", True), ([260, 300], 256, 16, 4, 64, "bf16", False),
    ([1024 + 37 * i for i in range(20)], 1024, 16, 1, 64, "f16", False), ([64 * 33], 64 * 32, 128, 1, 64, "bf16", False)])
def test_against_64_bits(lens, shared, H, q_len, bs, dtype, causal):
    case = Case(len(lens) + H + shared, lens, shared, H, q_len, bs, dtype, causal)
    nb.mla_reset_counters()
    out, lse = case.run()
    torch.cuda.synchronize()
    assert nb.mla_get_counters()[nb.CTR_DECODE_SHARED] == 1
    case.check(out, lse, heads=sorted({0, 1, H // 2, H - 1}))


@pytest.mark.parametrize("out_dtype", ["f16", "bf16"])
def test_outputs_of_16_bits(out_dtype):
    case = Case(1, [300, 400], 256, 16, 1, 32, out_dtype)
    case.check(*case.run(out_dtype=out_dtype))


@pytest.mark.parametrize("q_len,causal", [(1, False), (3, True)])
def test_contexts_shorter_than_the_prefix(q_len, causal):
    """Contexts of no tokens, of one, of less than a window, inside the prefix and at its end."""
    case = Case(2, [0, 1, 2, 100, 255, 256, 257, 400, 0], 256, 16, q_len, 16, "bf16", causal)
    out, lse = case.run()
    case.check(out, lse)


def test_all_contexts_empty():
    case = Case(3, [0, 0], 64)
    out, lse = case.run()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_many_requests_and_long_contexts():
    case = Case(4, [8192 + 50 * i for i in range(40)], 8192, 16, 1, 32, "bf16")
    case.check(*case.run(), requests=[0, 7, 8, 39], heads=[0, 15])


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.5])
def test_any_scale(scale):
    case = Case(5, [200, 150], 128, scale=scale, dtype="bf16")
    case.check(*case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores_that_rise(dtype):
    """Keys that grow along the tokens: the running maximum moves all the time."""
    case = Case(6, [900, 800], 640, 16, 1, 32, dtype)
    for b, n in enumerate(case.lens):
        row = case.rows_of(b, n)[case.shared if b else 0:]
        case.ckv.view(-1, 512)[row] *= (torch.arange(len(row), device="cuda") / 120)[:, None].to(case.dtype)
    case.check(*case.run())


def test_large_values():
    """Latents of 2^80 (queries as much smaller) whose scores rise: sums of weights that lag behind the maximum stay finite."""
    case = Case(14, [900, 800], 640, 16, 1, 32, "bf16")
    case.ckv.mul_(2.0 ** 80)
    case.q_abs.mul_(2.0 ** -80)
    for b, n in enumerate(case.lens):
        row = case.rows_of(b, n)[case.shared if b else 0:]
        case.ckv.view(-1, 512)[row] *= (torch.arange(len(row), device="cuda") / 300)[:, None].to(case.dtype)
    out, lse = case.run()
    assert torch.isfinite(out).all()
    case.check(out, lse, heads=[0, 7, 15])


@pytest.mark.parametrize("lens,shared,H,q_len", [([700 + 9 * i for i in range(18)], 512, 128, 1), ([16500], 16384, 16, 1), ([30000, 29000], 28672, 16, 1)])
def test_merges_of_many_rows_and_of_many_parts(lens, shared, H, q_len):
    case = Case(15, lens, shared, H, q_len, 64, "f16")
    case.check(*case.run(), requests=sorted({0, len(lens) - 1}), heads=sorted({0, 5, H - 1}))


def test_hidden_tokens_that_are_not_finite():
    """In a causal window, a token that only the last rows see: the rows before it do not."""
    case = Case(7, [300, 290], 256, 16, 4, 16, "f16", True)
    want, want_lse = case.run()
    row = case.rows_of(0, 300)[298]  # seen by the rows 2 and 3 of request 0
    case.ckv.view(-1, 512)[row, 7] = float("nan")
    out, lse = case.run()
    assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(lse[0, :2], want_lse[0, :2])
    assert bool(out[0, 2:].isnan().all()) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("H,q_len", [(16, 1), (128, 2)])
def test_a_plan_serves_contexts_that_grow_and_shrink(H, q_len):
    case = Case(8, [300, 256, 700], 256, H, q_len, 32, "bf16", q_len > 1, room=2000)
    plan = case.plan()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    out, lse = case.run(plan)
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        rt.decode_shared(plan, case.q_abs, case.q_pe, case.ckv, case.kpe, case.table, case.ctx, case.scale, out, lse,
                         shared_table=case.shared_table, stream=side)
    g = torch.Generator("cuda").manual_seed(9)
    for lens in ([2000, 257, 701], [100, 0, 2300]):
        case.lens = lens
        case.ckv.copy_(torch.randn(case.ckv.shape, device="cuda", generator=g))
        case.kpe.copy_(torch.randn(case.kpe.shape, device="cuda", generator=g))
        case.nan_behind()
        case.ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        case.check(out, lse, heads=[0, H - 1])


def test_the_first_requests_table_row_stands_in_for_the_shared_table():
    case = Case(10, [200, 300], 128)
    want, want_lse = case.run()
    case.table[0, :4] = case.shared_table
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    rt.decode_shared(case.plan(), case.q_abs, case.q_pe, case.ckv, case.kpe, case.table, case.ctx, SCALE, out, lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_the_same_bits_every_time_and_on_another_stream():
    case = Case(11, [3000 + 111 * i for i in range(12)], 2048, 64, 1, 64, "f16")
    plan = case.plan()
    out, lse = case.run(plan)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        again, again_lse = case.run(plan, stream=side)
        side.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_a_page_outside_the_pool_reads_zeros():
    case = Case(12, [200], 128)
    case.ckv.nan_to_num_(0), case.kpe.nan_to_num_(0)
    case.shared_table[1] = 10 ** 6
    out, lse = case.run()
    torch.cuda.synchronize()
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_waits_that_run_out_are_reported():
    case = Case(13, [5000] * 4, 4096)
    try:
        nb.mla_set_wait_timeout_ns(1)
        case.run()
        st, code = nb.mla_check_device_errors(None)
    finally:
        nb.mla_set_wait_timeout_ns(2_000_000_000)
    assert st in (nb.MLA_OK, nb.MLA_ERR_TIMEOUT)
    case.check(*case.run(), requests=[0], heads=[0])
