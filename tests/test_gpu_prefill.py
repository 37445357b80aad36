"""Attention of packed prompts over expanded keys and values, against the definition in 64 bits."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


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
    """Requests of new[b] rows and ctx[b] tokens, packed; `spare` rows of NaN behind the last of them."""

    def __init__(self, seed, new, ctx, H, dtype, causal=True, joint=False, spare=0, scale=SCALE, peaked=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.new, self.ctx, self.H, self.dtype, self.causal, self.scale = new, ctx, H, TDT[dtype], causal, scale
        self.T, self.S = sum(new) + spare, sum(ctx) + spare
        self.q_at, self.kv_at = ([sum(x[:b]) for b in range(len(new) + 1)] for x in (new, ctx))
        self.q_indptr, self.kv_indptr = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.q_at, self.kv_at))

        def rand(n, real, *shape):
            x = torch.randn(n, *shape, device="cuda", generator=g)
            x[real:] = float("nan")
            return x.to(self.dtype)

        q = rand(max(self.T, 1), sum(new), H, 192) * peaked
        self.q_nope, self.q_pe = (q[..., :128], q[..., 128:]) if joint else (q[..., :128].contiguous(), q[..., 128:].contiguous())
        self.k, self.v, self.k_pe = rand(max(self.S, 1), sum(ctx), H, 128), rand(max(self.S, 1), sum(ctx), H, 128), rand(max(self.S, 1), sum(ctx), 64)
        self.plan = rt.plan_prefill(len(new), H, max(self.T, 1))

    def run(self, **kw):
        out = torch.full((max(self.T, 1), self.H, 128), 77.0, dtype=self.dtype, device="cuda")
        lse = torch.full((max(self.T, 1), self.H), 77.0, device="cuda")
        rt.prefill(self.plan, self.q_nope, self.q_pe, self.k, self.k_pe, self.v, self.q_indptr, self.kv_indptr, self.scale, out, lse, causal=self.causal, **kw)
        return out, lse

    def check(self, out, lse, heads=None, rows=None, requests=None):
        """Scores: 192 products, exact in fp32, added with at most 2^-23 of the sum of their magnitudes lost each
        time, and a few roundings of the score itself on its way into the exponential: off by ds. Weights: a factor
        exp(ds) in the numerator and in the sum, 2^-20 for the exponential and the sums' own roundings beside n tokens,
        and half a step of the type (fp16: at least 2^-25, of weights whose greatest is at least 1). The output is
        their average of the values, rounded by half a step once more."""
        half = torch.finfo(self.dtype).eps / 2
        ulp = 2.0 ** -23
        n, t = sum(self.new), sum(self.ctx)
        assert bool((out[n:] == 77).all()) and bool((lse[n:] == 77).all())
        for b in range(len(self.new)) if requests is None else requests:
            L, m = self.ctx[b], self.new[b]
            pick = range(m) if rows is None else sorted({r for r in rows if r < m})
            if not len(pick):
                continue
            at = torch.tensor(list(pick), device="cuda")
            ks = slice(self.kv_at[b], self.kv_at[b] + L)
            pos = torch.arange(L, device="cuda")
            seen = (L - m + at + 1).clamp(0, L) if self.causal else torch.full_like(at, L)
            hidden = pos[None] >= seen[:, None]
            for h in range(self.H) if heads is None else heads:
                q = torch.cat((self.q_nope[self.q_at[b] + at, h], self.q_pe[self.q_at[b] + at, h]), 1).double()
                k = torch.cat((self.k[ks, h], self.k_pe[ks]), 1).double()
                v = self.v[ks, h].double()
                s = (q @ k.T * self.scale).masked_fill(hidden, -math.inf)
                mags = abs(self.scale) * (q.abs() @ k.abs().T)
                ds = ((192 * ulp * mags + 8 * ulp * (s.abs())).masked_fill(hidden, 0).amax(1) if L else torch.zeros(len(at), device="cuda").double())
                got, got_lse = out[self.q_at[b] + at, h].double(), lse[self.q_at[b] + at, h].double()
                empty = seen == 0
                assert bool((got[empty] == 0).all()) and bool((got_lse[empty] == -math.inf).all())
                if bool(empty.all()):
                    continue
                q_ok = ~empty
                s, ds, got, got_lse = s[q_ok], ds[q_ok], got[q_ok], got_lse[q_ok]
                z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                want, size = p @ v, p @ v.abs()
                tol = (half + 2 * ds + 2.0 ** -20 + 2 * L * ulp)[:, None] * size
                if self.dtype == torch.float16:
                    tol = tol + L * 2.0 ** -25 * v.abs().amax()
                tol = tol + half * (want.abs() + tol) + (2.0 ** -25 if self.dtype == torch.float16 else 0)
                err = (got - want).abs()
                assert bool((err <= tol).all()), (b, h, float((err - tol).max()), float(err.max()))
                lse_tol = (ds + L * ulp + 2.0 ** -20) / math.log(2.0) + 4 * ulp * (z.abs() / math.log(2.0))
                assert bool(((got_lse - z / math.log(2.0)).abs() <= lse_tol).all()), (b, h)


CASES = [
    ([1], [1], 1), ([1], [300], 2), ([5], [5], 3), ([127], [127], 1), ([128], [128], 2), ([129], [129], 2), ([256], [256], 1), ([257], [257], 2),
    ([300], [300], 16), ([64], [1000], 4), ([200], [1024], 3), ([1, 1, 1], [1, 128, 129], 2), ([0, 40, 0, 130], [7, 40, 0, 500], 2), ([30] * 20, [30] * 20, 2),
    ([3], [2], 2), ([200], [50], 1), ([0], [0], 1), ([400, 9], [0, 9], 2)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,H", CASES)
def test_small_calls(new, ctx, H, causal, dtype):
    case = Case(len(new) + sum(ctx), new, ctx, H, dtype, causal, joint=H == 2, spare=3)
    out, lse = case.run()
    torch.cuda.synchronize()
    case.check(out, lse)


@pytest.mark.parametrize("new,ctx,H,dtype,causal", [
    ([2000], [2000], 4, "bf16", True), ([1500, 300, 777], [1500, 4000, 777], 3, "f16", True), ([100], [20000], 2, "bf16", True),
    ([600], [9000], 1, "f16", False), ([256] * 70, [256] * 70, 1, "f16", True), ([70, 1300], [20001, 1300], 16, "bf16", True),
    ([513], [30000], 8, "f16", True)])
def test_planned_and_cut_calls(new, ctx, H, dtype, causal):
    case = Case(11 + len(new), new, ctx, H, dtype, causal, joint=True, spare=200)
    nb.mla_reset_counters()
    out, lse = case.run()
    torch.cuda.synchronize()
    assert nb.mla_get_counters()[nb.CTR_PREFILL] == 1
    rows = [0, 1, 127, 128, 255, 256, 300, 511, 512, 513, 776, 1023, 1299, 1499, 1999]
    case.check(out, lse, heads=[0, H - 1], rows=rows, requests=range(min(4, len(new))))


@pytest.mark.parametrize("new,ctx,H,dtype", [
    ([4], [2176], 3, "f16"), ([900, 700], [900, 1276], 5, "bf16"), ([2176], [2176], 2, "bf16"), ([2177], [2177], 2, "f16"), ([1] * 50 + [200], [2] * 50 + [2000], 2, "bf16")])
def test_longest_calls_that_plan_for_themselves(new, ctx, H, dtype):
    case = Case(len(new) + sum(ctx), new, ctx, H, dtype, joint=True)
    out, lse = case.run()
    torch.cuda.synchronize()
    case.check(out, lse, heads=[0, H - 1], rows=[0, 3, 127, 128, 199, 255, 256, 699, 899, 2047, 2048, 2175, 2176], requests=sorted({0, len(new) // 2, len(new) - 1}))


@pytest.mark.parametrize("new,ctx,H,dtype", [
    ([1024], [5000], 24, "bf16"), ([1], [30000], 1, "f16"), ([600, 520, 1], [3000, 2500, 9000], 40, "f16"), ([512] * 6, [512, 900, 4000, 513, 2048, 6000], 16, "bf16"),
    ([1] * 2100 + [300], [20] * 2100 + [9000], 2, "f16"), ([1] * 2050 + [130], [3] * 2050 + [40000], 1, "bf16")])
def test_ways_of_cutting(new, ctx, H, dtype):
    """Equal runs, one run alone, unequal ones, and a long one behind more than the planner weighs ways for."""
    case = Case(len(new) + H, new, ctx, H, dtype, joint=True)
    out, lse = case.run()
    torch.cuda.synchronize()
    B = len(new)
    case.check(out, lse, heads=sorted({0, H // 2, H - 1}), rows=[0, 127, 128, 255, 256, 511, 519, 599, 1023], requests=sorted({0, 1, 7, B // 2, B - 2, B - 1} & set(range(B))))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_any_scale(scale):
    case = Case(21, [150], [200], 2, "bf16", scale=scale)
    case.check(*case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scores_that_rise_and_peak(dtype):
    """Keys that grow along the tokens, so that the running maximum moves by far more than its slack all the time."""
    case = Case(22, [700], [700], 2, dtype, peaked=4.0)
    case.k.mul_((torch.arange(700, device="cuda") / 100)[:, None, None].to(case.dtype))
    case.check(*case.run())


@pytest.mark.parametrize("new,ctx,H", [([300, 5], [300, 700], 3), ([700], [4000], 6), ([1, 1], [40, 1], 2)])
def test_queries_in_other_orders(new, ctx, H):
    """Queries that lie head by head, that are every second row of a tensor, and parts of wider ones."""
    case = Case(24, new, ctx, H, "bf16")
    want = case.run()
    q = torch.cat((case.q_nope, case.q_pe), 2)
    by_head = torch.empty(H, case.T, 192, dtype=q.dtype, device="cuda")
    by_head.copy_(q.transpose(0, 1))
    apart = torch.full((2 * case.T, H, 200), float("nan"), dtype=q.dtype, device="cuda")
    apart[::2, :, :192] = q
    for x in (by_head.transpose(0, 1), apart[::2]):
        case.q_nope, case.q_pe = x[..., :128], x[..., 128:192]
        got = case.run()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    case.check(*got)


@pytest.mark.parametrize("H", [1, 256])
def test_fewest_and_most_heads(H):
    case = Case(25, [130, 2], [200, 2], H, "f16", joint=True)
    case.check(*case.run(), heads=sorted({0, H // 2, H - 1}))


def test_large_values():
    """Values of 2^98 in bf16 under scores that rise: sums of weights that lag behind the maximum stay finite."""
    case = Case(23, [700], [700], 2, "bf16")
    case.k.mul_((torch.arange(700, device="cuda") / 200)[:, None, None].to(case.dtype))
    case.v.mul_(2.0 ** 98)
    out, lse = case.run()
    assert torch.isfinite(out).all()
    case.check(out, lse)


@pytest.mark.parametrize("new,ctx", [([300], [300]), ([300], [1500]), ([130, 600], [130, 2600])])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_tokens_that_are_not_finite_reach_only_rows_that_see_them(what, dtype, new, ctx):
    bad = float(what)
    case = Case(23, new, ctx, 2, dtype, spare=140)
    want, want_lse = case.run()
    b = len(new) - 1
    L, n = ctx[b], new[b]
    at = [L - n + 7, L - n + 128, L - n + 200, L - 1]
    for t, col in zip(at, (0, 33, 127, 64)):
        case.v[case.kv_at[b] + t, 0, col] = bad
    case.v[case.kv_at[b] + at[1], 0, 33] = bad
    out, lse = case.run()
    torch.cuda.synchronize()
    same = out.clone()
    for t, col in zip(at, (0, 33, 127, 64)):
        first = case.q_at[b] + t - (L - n)
        rows = slice(first, case.q_at[b] + n)
        got = out[rows, 0, col].float()
        assert bool((got.isnan() if what == "nan" else got == math.inf).all()), (t, col)
        same[rows, 0, col] = want[rows, 0, col]
    assert torch.equal(same[: sum(new)], want[: sum(new)]) and torch.equal(lse, want_lse)
    # and in the keys: the score of a token that a row does not see does not matter
    case.v = torch.where(torch.isfinite(case.v), case.v, torch.zeros_like(case.v))
    want, want_lse = case.run()
    case.k[case.kv_at[b] + at[2], 1, 5] = float("nan")
    out, lse = case.run()
    first = case.q_at[b] + at[2] - (L - n)
    assert bool(out[first:case.q_at[b] + n, 1].isnan().all()) and bool(lse[first:case.q_at[b] + n, 1].isnan().all())
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first]) and torch.equal(out[first:sum(new), 0], want[first:sum(new), 0])


def test_the_same_bits_every_time_and_on_another_stream():
    case = Case(24, [513, 40, 1000], [20000, 4000, 1000], 16, "bf16")
    out, lse = case.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        again, again_lse = case.run(stream=side)
        side.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("direct", [True, False])
def test_captured_calls_replay_with_other_offsets(direct):
    T, S, H = (600, 900, 4) if direct else (900, 9000, 4)
    shapes = [([100, 200, 300], [100, 500, 300]), ([600, 0, 0], [600, 0, 0]), ([1, 1, 1], [1, 250, 600])]
    if not direct:
        shapes = [([100, 200, 600], [100, 8000, 700]), ([900, 0, 0], [8999, 0, 1]), ([1, 1, 1], [1, 6000, 600])]
    big = Case(25, [T], [S], H, "f16")
    big.plan = rt.plan_prefill(3, H, T)
    qi, ki = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    out, lse = torch.zeros(T, H, 128, dtype=torch.float16, device="cuda"), torch.zeros(T, H, device="cuda")
    call = lambda o, l, **kw: rt.prefill(big.plan, big.q_nope, big.q_pe, big.k, big.k_pe, big.v, qi, ki, SCALE, o, l, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    call(out, lse)
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        call(out, lse, stream=side)
    for new, ctx in shapes:
        at = lambda x: torch.tensor([0, *torch.tensor(x).cumsum(0).tolist()], dtype=torch.int32)  # noqa: E731
        qi.copy_(at(new)), ki.copy_(at(ctx))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        case = Case(25, [T], [S], H, "f16")
        case.new, case.ctx, case.q_at, case.kv_at, case.T, case.S = new, ctx, at(new).tolist(), at(ctx).tolist(), sum(new), sum(ctx)
        case.check(out[: sum(new)], lse[: sum(new)], rows=[0, 1, 99, 128, 199, 256, 599, 899])


def test_offsets_that_pass_the_tensors_are_cut_off():
    case = Case(26, [100], [300], 2, "f16")
    case.q_indptr[1], case.kv_indptr[1] = 140, 10 ** 6
    guard = torch.full((140, 2, 128), 5.0, dtype=torch.float16, device="cuda")
    rt.prefill(case.plan, case.q_nope, case.q_pe, case.k, case.k_pe, case.v, case.q_indptr, case.kv_indptr, SCALE, guard[:100])
    torch.cuda.synchronize()
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2
    assert bool((guard[100:] == 5).all())
    case.check(guard[:100], case.run()[1][:100])
    nb.mla_check_device_errors(None)
