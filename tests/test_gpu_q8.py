"""Block-scaled 8-bit caches on the GPU: the quantizing write bit for bit, and attention over the cache, against
the f64 oracle."""
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


class Q8Case:
    """A batch over a block-scaled pool drawn as bits: bytes by inputs.e4m3_bits, scales powers of two or not."""

    def __init__(self, seed, lens, H=16, q_len=1, bs=32, g=16, dtype="f16", causal=False, window=0, sinks=0, pow2=False):
        rng = np.random.default_rng(seed)
        need = [gen.pages_for(L, bs) for L in lens]
        self.nb = sum(need) + 5
        perm = rng.permutation(self.nb)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.lens, self.H, self.q_len, self.bs, self.g, self.dtype = np.array(lens, np.int32), H, q_len, bs, g, dtype
        self.causal, self.window, self.sinks = causal, window, sinks
        self.ckv, self.kpe = gen.e4m3_bits(rng, (self.nb, bs, 512)), gen.e4m3_bits(rng, (self.nb, bs, 64))
        z = np.exp2(rng.integers(-4, 1, size=(self.nb, bs // g)).astype(np.float64))
        self.scales = (z if pow2 else z * rng.uniform(0.6, 1.4, size=z.shape)).astype(np.float32)
        self.q_abs = gen.to_bits(rng.standard_normal((len(lens), q_len, H, 512)), dtype)
        self.q_pe = gen.to_bits(rng.standard_normal((len(lens), q_len, H, 64)), dtype)

    def upload(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = rt.Q8Cache(dev(self.ckv), dev(self.kpe), dev(self.scales))
        self.qa, self.qp = rt.to_device_16(self.q_abs, self.dtype, "cuda"), rt.to_device_16(self.q_pe, self.dtype, "cuda")
        self.tab, self.ctx = dev(self.table), dev(self.lens)
        return self

    def plan(self):
        return rt.plan_q8(len(self.lens), self.H, self.q_len, self.causal, self.window, self.sinks)

    def decode(self, out_dtype="f32", plan=None, **kw):
        out = torch.full((len(self.lens), self.q_len, self.H, 512), float("nan"), dtype=TDT[out_dtype], device="cuda")
        lse = torch.full((len(self.lens), self.q_len, self.H), float("nan"), device="cuda")
        rt.decode_q8(plan or self.plan(), self.qa, self.qp, self.cache, self.tab, self.ctx, SCALE, out, lse, **kw)
        return out, lse

    def rows(self, b):
        return orc.request_values_q8(self.ckv, self.kpe, self.scales, self.table[b], int(self.lens[b]))

    def check(self, out, lse, heads=None, requests=None):
        """Every sampled row within the error that the arithmetic allows. Scores: products exact in fp32, at most
        576 rounded additions (2^-23 of the sum of magnitudes each, whatever the rounding of the unit), a few
        more for the scales: ds. Probabilities: a factor exp(ds) and two (numerator and sum), and the rounding
        of each weight to a sum of three E4M3 terms, 2^-12 of it. out is their average of the values: at most
        (2^-12 + 2 ds + 2^-18) max|v|; the LSE is off by at most ds / ln 2 and its own rounding."""
        heads = range(self.H) if heads is None else heads
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        half_step = torch.finfo(out.dtype).eps / 2
        for b in range(len(self.lens)) if requests is None else requests:
            c, k = self.rows(b)
            qa, qp = orc.decode16(self.q_abs[b], self.dtype), orc.decode16(self.q_pe[b], self.dtype)
            ref, ref_lse = orc.attend_rows(qa[:, heads], qp[:, heads], c, k, SCALE, self.causal, self.window, self.sinks)
            if len(c) == 0:
                assert not got[b].any() and np.all(np.isneginf(got_lse[b]))
                continue
            for i in range(self.q_len):
                vis = orc.visible_window(len(c), self.q_len, i, self.causal, self.window, self.sinks)
                for n, h in enumerate(heads):
                    if not vis.any():
                        assert not got[b, i, h].any() and np.isneginf(got_lse[b, i, h])
                        continue
                    mag = np.abs(c[vis]) @ np.abs(qa[i, h]) + np.abs(k[vis]) @ np.abs(qp[i, h])
                    ds = 600 * 2.0 ** -23 * SCALE * mag.max()
                    top = np.abs(c[vis]).max(0)
                    err = np.abs(got[b, i, h] - ref[i, n])
                    tol = (2.0 ** -12 + 2 * ds + 2.0 ** -18) * top
                    tol = tol + half_step * (np.abs(ref[i, n]) + tol)
                    assert np.all(err <= tol), (b, i, h, float((err / tol).max()))
                    assert abs(got_lse[b, i, h] - ref_lse[i, n]) <= ds / math.log(2) + 2.0 ** -20 * max(1, abs(ref_lse[i, n])), (b, i, h)
            live = [(i, n, h) for i in range(self.q_len) for n, h in enumerate(heads) if np.isfinite(ref_lse[i, n])]
            if live and out.dtype == torch.float32:
                # over a whole request the errors are random: the relative 2-norm stays under a 16-bit half step
                a = np.stack([got[b, i, h] for i, n, h in live])
                r = np.stack([ref[i, n] for i, n, h in live])
                assert np.linalg.norm(a - r) <= 2.0 ** -11 * np.linalg.norm(r)


# --- the write ----------------------------------------------------------------------


def new_tokens(seed, B, q_len, dtype, spread=3.0):
    rng = np.random.default_rng(seed)
    size = np.exp2(spread * rng.standard_normal((B, q_len, 1)))
    return (gen.to_bits(rng.standard_normal((B, q_len, 512)) * size, dtype),
            gen.to_bits(rng.standard_normal((B, q_len, 64)) * size, dtype))


def append(case, c_bits, k_bits, **kw):
    rt.cache_append_q8(case.cache, rt.to_device_16(c_bits, case.dtype, "cuda"), rt.to_device_16(k_bits, case.dtype, "cuda"),
                       case.tab, case.ctx, **kw)


def same_cache(case, want):
    for got, ref, what in zip((case.cache.ckv, case.cache.kpe, case.cache.scales), want, ("ckv", "kpe", "scales")):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=what == "scales"), what


@pytest.mark.parametrize("bs,g,q_len,dtype", [(16, 1, 1, "f16"), (32, 32, 1, "bf16"), (32, 16, 4, "f16"), (64, 64, 32, "bf16"),
                                              (64, 2, 33, "f16"), (64, 64, 300, "f16"), (16, 8, 7, "bf16"), (64, 1, 129, "bf16")])
def test_append_q8_matches_the_oracle_bit_for_bit(bs, g, q_len, dtype):
    case = Q8Case(1, [0, 1, 2, 31, 33, 64, 700, 1001], q_len=q_len, bs=bs, g=g, dtype=dtype, pow2=True).upload()
    c, k = new_tokens(2, len(case.lens), q_len, dtype)
    want = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens, orc.decode16(c, dtype), orc.decode16(k, dtype))
    nb.mla_reset_counters()
    append(case, c, k)
    assert nb.mla_get_counters()[nb.CTR_WRAP] == 1
    same_cache(case, want)
    append(case, c, k)  # the same tokens again: nothing moves any more
    same_cache(case, want)


def test_append_q8_moves_earlier_bytes_only_when_the_scale_grows():
    case = Q8Case(3, [40, 40, 40], q_len=1, bs=32, g=32, dtype="f16", pow2=True)
    case.scales[:] = 0.25
    case.scales[case.table[2, 1]] = 0.3  # not a power of two: the bytes move by a rounded ratio
    case.upload()
    c, k = np.zeros((3, 1, 512)), np.zeros((3, 1, 64))
    c[:, 0, 0] = [1.0, 448.0, 60000.0]
    c, k = gen.to_f16_bits(c), gen.to_f16_bits(k)
    append(case, c, k)
    s = case.cache.scales.cpu().numpy()
    assert [s[case.table[b, 1], 0] for b in range(3)] == [0.25, 1.0, 256.0]
    for b in range(3):
        page = case.table[b, 1]
        old = orc.decode_e4m3(case.ckv[page, :7]) * (np.float64(np.float32(case.scales[page, 0]) / np.float32(s[page, 0])))
        assert np.array_equal(case.cache.ckv[page, :7].cpu().numpy(), case.ckv[page, :7] if b == 0 else orc.encode_e4m3(np.float32(old).astype(np.float64)))
        assert np.array_equal(case.cache.ckv[page, 8:].cpu().numpy(), case.ckv[page, 8:])  # behind the last token: untouched
    first = [case.table[b, 0] for b in range(3)]
    assert np.array_equal(case.cache.ckv[first].cpu().numpy(), case.ckv[first])


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_append_q8_non_finite_tokens_poison_their_block_alone(value):
    case = Q8Case(4, [40, 40], q_len=3, bs=32, g=2, dtype="bf16", pow2=True).upload()
    c, k = (orc.decode16(x, "bf16") for x in new_tokens(5, 2, 3, "bf16"))
    k[1, 1, 63] = value  # position 38: the block of 38 and 39
    bits = [gen.to_bf16_bits(x) for x in (c, k)]
    want = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens, c, k)
    append(case, *bits)
    same_cache(case, want)
    s = case.cache.scales.cpu().numpy()
    assert np.isnan(s).sum() == 1 and np.isnan(s[case.table[1, 1], 3])
    append(case, *[gen.to_bf16_bits(np.ones_like(x)) for x in (c, k)])  # written again from the block's start
    assert not np.isnan(case.cache.scales.cpu().numpy()).any()


def test_append_q8_extreme_magnitudes():
    lens = [1] * 6
    case = Q8Case(6, lens, q_len=1, bs=16, g=1, dtype="bf16", pow2=True).upload()
    top = [0.0, 1e-38, 2.0 ** -52, 448 * 2.0 ** 60, 480 * 2.0 ** 60, 3e38]
    c, k = np.zeros((6, 1, 512)), np.zeros((6, 1, 64))
    c[:, 0, 5], k[:, 0, 9] = top, -np.array(top)
    bits = [gen.to_bf16_bits(x) for x in (c, k)]
    c, k = (orc.decode16(x, "bf16") for x in bits)
    append(case, *bits)
    same_cache(case, orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens, c, k))


def test_append_q8_bad_pages_are_flagged_and_not_written():
    case = Q8Case(7, [100, 64, 200], q_len=2, bs=32, g=4, dtype="f16", pow2=True)
    want_table = case.table.copy()
    case.table[0, 3] = case.nb + 7
    case.lens[2] = case.table.shape[1] * 32 + 1  # its last token lies behind the table's row
    case.upload()
    c, k = new_tokens(8, 3, 2, "f16")
    append(case, c, k)
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code & 2
    c64, k64 = orc.decode16(c, "f16"), orc.decode16(k, "f16")
    want = orc.cache_append_q8(case.ckv, case.kpe, case.scales, want_table[1:2], case.lens[1:2], c64[1:2], k64[1:2])
    last = want_table[2:3]  # request 2: its first new token is the last position of the row's last page
    want = orc.cache_append_q8(*want, last, np.array([case.lens[2] - 1]), c64[2:3, :1], k64[2:3, :1])
    same_cache(case, want)


# --- attention ----------------------------------------------------------------------


@pytest.mark.parametrize("lens,H,q_len,bs,g,dtype,causal", [
    ([1], 16, 1, 16, 1, "f16", False),
    ([37], 16, 1, 16, 16, "bf16", False),
    ([0, 1, 127, 128, 129, 0, 300, 1], 16, 1, 32, 8, "f16", False),
    ([700, 0, 5000, 64], 16, 1, 64, 64, "bf16", False),
    ([20000], 16, 1, 32, 32, "f16", False),            # one request over all gangs
    ([9000, 3], 128, 1, 64, 1, "bf16", False),
    ([513, 2000, 77], 64, 1, 16, 2, "f16", False),
    ([3, 900, 1, 0, 4100], 16, 9, 32, 16, "f16", True),  # contexts shorter than the window: rows that see nothing
    ([333, 1500], 16, 32, 32, 4, "bf16", True),
    ([100, 40], 64, 3, 64, 32, "f16", True),
    ([640], 16, 4, 32, 1, "bf16", False),               # several rows that all see everything
])
def test_decode_q8_against_the_oracle(lens, H, q_len, bs, g, dtype, causal):
    case = Q8Case(11, lens, H=H, q_len=q_len, bs=bs, g=g, dtype=dtype, causal=causal).upload()
    heads = None if H == 16 and q_len == 1 else sorted({0, 5, H // 2, H - 1})
    nb.mla_reset_counters()
    out, lse = case.decode("f32")
    assert nb.mla_get_counters()[nb.CTR_DECODE_Q8] == 1
    case.check(out, lse, heads)
    out16, lse16 = case.decode(dtype)
    assert torch.equal(out16, out.to(TDT[dtype])) and torch.equal(lse16, lse)  # rounded once; the same bits again


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (129, 33), (1000, 64), (40000, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("lens,H,q_len,bs,dtype,causal", [
    ([0, 1, 15, 128, 1030, 2500], 16, 1, 32, "f16", False),
    ([5, 130, 0, 3000], 16, 7, 64, "bf16", True),
    ([3000, 90], 64, 2, 16, "bf16", True),
])
def test_decode_q8_windows(window, sinks, lens, H, q_len, bs, dtype, causal):
    case = Q8Case(12, lens, H=H, q_len=q_len, bs=bs, g=bs // 4, dtype=dtype, causal=causal, window=window, sinks=sinks).upload()
    out, lse = case.decode("f32")
    case.check(out, lse, None if H == 16 and q_len == 1 else [0, H - 1])


def test_decode_q8_many_short_requests():
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 260, size=700)]
    case = Q8Case(13, lens, bs=16, g=4).upload()
    out, lse = case.decode("f32")
    case.check(out, lse, heads=[3], requests=range(0, 700, 7))
    empty = torch.tensor(lens) == 0
    assert empty.any() and not out.cpu()[empty].any() and torch.isneginf(lse.cpu()[empty]).all()


@pytest.mark.parametrize("where", ["behind", "window", "draft"])
def test_decode_q8_ignores_what_no_row_may_see(where):
    """NaN bytes and scales behind the last token, outside the window, and in tokens that a row may not see yet."""
    kw = dict(behind=dict(lens=[70, 700]), window=dict(lens=[70, 700], window=50, sinks=3),
              draft=dict(lens=[70, 700], q_len=4, causal=True))[where]
    case = Q8Case(14, bs=64, g=1, **kw)
    clean = Q8Case(14, bs=64, g=1, **kw).upload()
    for b, L in enumerate(case.lens):
        L = int(L)
        bad = {"behind": range(L, -(-L // 64) * 64), "window": range(3, L - 50), "draft": range(L - 1, L)}[where]
        for t in bad:
            page = case.table[b, t // 64]
            case.ckv[page, t % 64] = 0x7F
            case.kpe[page, t % 64] = 0xFF
            case.scales[page, t % 64] = (np.nan, np.inf, 0.0)[t % 3] if where != "draft" else np.nan
    case.upload()
    out, lse = case.decode("f32")
    ref, ref_lse = clean.decode("f32")
    if where == "draft":
        assert torch.isnan(out[:, 3]).all() and torch.isnan(lse[:, 3]).all()  # the row that sees it
        out, lse, ref, ref_lse = out[:, :3], lse[:, :3], ref[:, :3], ref_lse[:, :3]
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("L", [40, 5000])
def test_decode_q8_nan_reaches_every_row_that_sees_it(L):
    case = Q8Case(15, [L, L], bs=32, g=8)
    case.scales[case.table[0, 0], 1] = np.nan
    case.upload()
    out, lse = case.decode("f32")
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    case.check(out, lse, requests=[1])
    case.q_abs[0, 0, 3, 7] = gen.to_f16_bits(np.array(np.nan))  # a NaN query: that row alone
    case.scales[case.table[0, 0], 1] = 1.0
    case.upload()
    out, lse = case.decode("f32")
    assert torch.isnan(out[0, 0, 3]).all() and torch.isnan(lse[0, 0, 3])
    others = [h for h in range(16) if h != 3]
    assert torch.isfinite(out[:, :, others]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_q8_wide_ranges(dtype):
    """Scales and queries of very different sizes in one request, and scores that grow token by token."""
    case = Q8Case(16, [600, 2000], bs=32, g=1, dtype=dtype, pow2=True)
    rng = np.random.default_rng(17)
    case.scales[:] = np.exp2(rng.integers(-16, 3, size=case.scales.shape))
    size = np.exp2(rng.integers(-9, 3, size=(2, 1, 16, 1)).astype(np.float64))
    case.q_abs = gen.to_bits(orc.decode16(case.q_abs, dtype) * size, dtype)
    t = np.arange(2000)
    rows = orc.physical_rows(case.table[1], 2000, 32)
    case.scales.reshape(-1)[rows] = np.exp2(-6 + 8 * t / 2000).astype(np.float32)
    case.upload()
    out, lse = case.decode("f32")
    case.check(out, lse)


def test_decode_q8_bad_pages_are_flagged_and_read_as_zeros():
    case = Q8Case(18, [200, 100], bs=32, g=32)
    case.table[0, 2] = case.nb + 3
    case.table[1, 1] = -5
    case.upload()
    out, lse = case.decode("f32")
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code & 2
    # the same as a page of zeros
    page = [i for i in range(case.nb) if i not in case.table][0]
    case.ckv[page], case.kpe[page], case.scales[page] = 0, 0, 1.0
    case.table[0, 2] = case.table[1, 1] = page
    case.upload()
    ref, ref_lse = case.decode("f32")
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_decode_q8_replayed_as_the_contexts_grow():
    """The write and the attention captured once and replayed for every next token; the lengths grow on the
    device. Two graphs share the plan's workspace in turn."""
    case = Q8Case(19, [126, 0, 1000, 63], bs=32, g=32, pow2=True)
    extra = np.setdiff1d(np.arange(case.nb), case.table)[:4]
    table = np.concatenate([case.table, np.full((4, 1), -1, np.int32)], 1)
    for b in range(4):
        table[b, gen.pages_for(int(case.lens[b]), 32)] = extra[b]
    case.table = table
    case.upload()
    plan, plan_w = case.plan(), rt.plan_q8(4, 16, window=40, sinks=2)
    plan_w.workspace = plan.workspace
    steps = 5
    new = [new_tokens(20 + i, 4, 1, "f16", spread=1.0) for i in range(steps)]
    c_in, k_in = (torch.empty(4, 1, n, dtype=torch.float16, device="cuda") for n in (512, 64))
    out, out_w = (torch.empty(4, 1, 16, 512, device="cuda") for _ in range(2))
    lse, lse_w = (torch.empty(4, 1, 16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(side):
        with torch.cuda.graph(graphs[0], stream=side):
            case.ctx += 1
            rt.cache_append_q8(case.cache, c_in, k_in, case.tab, case.ctx)
            rt.decode_q8(plan, case.qa, case.qp, case.cache, case.tab, case.ctx, SCALE, out, lse)
        with torch.cuda.graph(graphs[1], stream=side):
            rt.decode_q8(plan_w, case.qa, case.qp, case.cache, case.tab, case.ctx, SCALE, out_w, lse_w)
    torch.cuda.synchronize()
    for i in range(steps):
        c, k = new[i]
        c_in.copy_(rt.to_device_16(c, "f16", "cuda"))
        k_in.copy_(rt.to_device_16(k, "f16", "cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        case.lens = case.lens + 1
        case.ckv, case.kpe, case.scales = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens,
                                                              orc.decode16(c, "f16"), orc.decode16(k, "f16"))
        same_cache(case, (case.ckv, case.kpe, case.scales))
        case.check(out, lse, heads=[0, 9])
        case.window, case.sinks = 40, 2
        case.check(out_w, lse_w, heads=[0, 9])
        case.window = case.sinks = 0


def test_layer_call_on_a_q8_cache_write_attend_unembed():
    """The next token written, attention, then W_UV^T by mla_merge_unembed on the one partial per request."""
    case = Q8Case(25, [900, 3000], bs=64, g=64, dtype="bf16", pow2=True).upload()
    c, k = new_tokens(26, 2, 1, "bf16", spread=1.0)
    append(case, c, k)
    out, lse = case.decode("f32")
    w_bits = gen.to_bits(np.random.default_rng(27).standard_normal((16, 512, 128)) / math.sqrt(512.0), "bf16")
    w = rt.to_device_16(w_bits, "bf16", "cuda")
    ov = torch.empty((2, 1, 16, 128), device="cuda")
    ind = rt.uniform_indptr(2, 1)
    nb.mla_merge_unembed(out.data_ptr(), lse.data_ptr(), ind.data_ptr(), 2, 1, 16, w.data_ptr(), nb.MLA_BF16, 128,
                         ov.data_ptr(), nb.MLA_F32, None, None)
    case.ckv, case.kpe, case.scales = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens,
                                                          orc.decode16(c, "bf16"), orc.decode16(k, "bf16"))
    case.check(out, lse)
    ref = np.einsum("biHr,Hrv->biHv", out.double().cpu().numpy(), orc.decode16(w_bits, "bf16"))
    assert np.abs(ov.double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()


def test_decode_q8_on_another_stream_and_twice_at_once():
    case = Q8Case(28, [5000, 100, 2000], bs=32, g=16).upload()
    ref, ref_lse = case.decode("f32")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [case.decode("f32", plan=case.plan(), stream=s) for s in streams]
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_decode_q8_refuses_a_short_workspace_and_wrong_shapes():
    case = Q8Case(29, [50], bs=32, g=32).upload()
    plan = case.plan()
    plan.workspace = plan.workspace[:-16]
    with pytest.raises(nb.MlaError) as e:
        case.decode(plan=plan)
    assert e.value.status == nb.MLA_ERR_INVALID_ARG
    plan = case.plan()
    out = torch.empty(1, 1, 16, 512, device="cuda")
    for bad in (dict(q_abs=case.qa[:, :, :8]), dict(q_pe=case.qp.float()), dict(block_table=case.tab.long()),
                dict(context_lens=case.ctx.repeat(2)), dict(out=out[..., :256]), dict(out_lse=out)):
        args = dict(q_abs=case.qa, q_pe=case.qp, cache=case.cache, block_table=case.tab, context_lens=case.ctx, scale=SCALE, out=out)
        with pytest.raises(ValueError):
            rt.decode_q8(plan, **{**args, **bad})


@pytest.mark.parametrize("H,dtype", [(16, "f16"), (16, "bf16"), (64, "f16"), (64, "bf16")])
def test_decode_q8_lengths_around_tiles_and_steps(H, dtype):
    lens = [31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 192, 193, 255, 256, 257, 287, 288, 289, 383, 384, 385]
    case = Q8Case(30, lens, H=H, bs=32, g=8, dtype=dtype).upload()
    out, lse = case.decode("f32")
    case.check(out, lse, heads=[1, H - 1])


@pytest.mark.parametrize("lens,H", [([60000] + [1] * 12, 16),        # rows merged by warps, in more parts than a warp has lanes
                                    ([0, 9000, 0, 30, 0], 16),       # by part lanes, beside requests without a tile
                                    ([200, 0, 40000, 3, 7, 0], 64)])
def test_decode_q8_merges_requests_in_many_parts(lens, H):
    case = Q8Case(31, lens, H=H, bs=64, g=64).upload()
    out, lse = case.decode("f32")
    case.check(out, lse, heads=[0, H - 1])


@pytest.mark.parametrize("H,dtype", [(16, "f16"), (64, "f16"), (64, "bf16")])
def test_decode_q8_one_token_far_above_a_long_even_tail(H, dtype):
    """One token's weight is 2^13 times each of 30000 equal ones, which make most of the sum: their weights are
    rounded alike, so their errors add up. Each is off by 2^-12 of itself or 2^-26 of the greatest one."""
    case = Q8Case(32, [30001], H=H, bs=32, g=1, dtype=dtype, pow2=True)
    q = np.zeros((1, 1, H, 512))
    q[..., 0] = 13.0 * math.log(2.0) / SCALE / 8
    case.q_abs, case.q_pe = gen.to_bits(q, dtype), gen.to_bits(np.zeros((1, 1, H, 64)), dtype)
    case.scales[:] = 1.0
    rows = orc.physical_rows(case.table[0], 30001, 32)
    flat = case.ckv.reshape(-1, 512)
    flat[rows] = flat[rows[1]]            # the tail: one value row
    flat[rows, 0] = orc.encode_e4m3(np.zeros(1))[0]
    flat[rows[777], 0] = orc.encode_e4m3(np.full(1, 8.0))[0]
    case.upload()
    out, lse = case.decode("f32")
    case.check(out, lse, heads=[0, H - 1])


@pytest.mark.parametrize("lens,H,dtype", [([131072], 16, "f16"), ([40000, 9000], 128, "bf16"), ([40000, 9000], 64, "f16")])
def test_decode_q8_bounded_waits_run_out_then_the_plan_is_usable(lens, H, dtype):
    """A limit of a few microseconds, far less than the call takes: every role gives up at its next wait, the call
    comes back with the error, and the next one on the same workspace is right."""
    case = Q8Case(33, lens, H=H, bs=64, g=64, dtype=dtype).upload()
    plan = case.plan()
    plan.workspace.fill_(0xFF)
    try:
        nb.mla_set_wait_timeout_ns(2_000)
        case.decode("f32", plan=plan)
        st, code = nb.mla_check_device_errors(None)
    finally:
        nb.mla_set_wait_timeout_ns(2_000_000_000)
    assert st == nb.MLA_ERR_TIMEOUT and code & 1, (st, code)
    out, lse = case.decode("f32", plan=plan)
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK, code
    case.check(out, lse, heads=[0, H - 1])


def test_q8_calls_refuse_buffers_elsewhere():
    case = Q8Case(34, [50], bs=32, g=32).upload()
    plan = case.plan()
    out = torch.empty(1, 1, 16, 512, device="cuda")
    args = dict(q_abs=case.qa, q_pe=case.qp, cache=case.cache, block_table=case.tab, context_lens=case.ctx, scale=SCALE, out=out)
    cpu_cache = rt.Q8Cache(case.cache.ckv.cpu(), case.cache.kpe.cpu(), case.cache.scales.cpu())
    for name in ("q_abs", "q_pe", "block_table", "context_lens", "out", "cache"):
        with pytest.raises(ValueError):
            rt.decode_q8(plan, **{**args, name: cpu_cache if name == "cache" else args[name].cpu()})
    with pytest.raises(ValueError):
        rt.decode_q8(plan, **{**args, "out": out.double()})
    c, k = (torch.zeros(1, 1, n, dtype=torch.float16, device="cuda") for n in (512, 64))
    for bad in ((cpu_cache, c, k, case.tab, case.ctx), (case.cache, c.cpu(), k, case.tab, case.ctx),
                (case.cache, c, k, case.tab, case.ctx.cpu()), (case.cache, c.double(), k.double(), case.tab, case.ctx)):
        with pytest.raises(ValueError):
            rt.cache_append_q8(*bad)


@pytest.mark.parametrize("g,scale", [(8, 3.0), (8, 0.3), (16, 2.0 ** 100), (2, 1e-30)])
def test_append_q8_beside_tokens_under_a_foreign_scale(g, scale):
    """The block's scale comes from elsewhere, a power of two or not, in range or not: it stays unless the new
    token needs a larger one."""
    case = Q8Case(35, [20, 46], q_len=1, bs=16, g=g, dtype="f16", pow2=True)  # (the last token is not its block's first)
    case.scales[:] = np.float32(scale)
    case.upload()
    c, k = new_tokens(36, 2, 1, "f16", spread=1.0)
    want = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens, orc.decode16(c, "f16"), orc.decode16(k, "f16"))
    append(case, c, k)
    same_cache(case, want)


@pytest.mark.parametrize("H,q_len,dtype", [(128, 32, "f16"), (64, 32, "bf16"), (128, 5, "bf16")])
def test_decode_q8_many_rows(H, q_len, dtype):
    """More row groups than there are SMs, or nearly: one gang, two, or nine."""
    case = Q8Case(40, [300, 0, 31, 900], H=H, q_len=q_len, bs=32, g=16, dtype=dtype, causal=True).upload()
    out, lse = case.decode("f32")
    case.check(out, lse, heads=[0, H - 1])


def test_q8_calls_reach_past_four_gigabytes():
    """Pages whose bytes lie more than 2^32 into the pool, written and read."""
    nblk, bs = 140_000, 64  # 4.6 GB of latent bytes
    case = Q8Case(41, [200, 70], bs=bs, g=8, dtype="bf16", pow2=True)
    small, n = case.table.copy(), case.nb
    case.table = np.where(small >= 0, small + (nblk - n), small).astype(np.int32)
    pool = rt.Q8Cache(torch.empty(nblk, bs, 512, dtype=torch.uint8, device="cuda"),
                      torch.empty(nblk, bs, 64, dtype=torch.uint8, device="cuda"), torch.empty(nblk, bs // 8, device="cuda"))
    for whole, part in zip((pool.ckv, pool.kpe, pool.scales), (case.ckv, case.kpe, case.scales)):
        whole[nblk - n:] = torch.from_numpy(part).cuda()
    case.upload()
    case.cache = pool
    c, k = new_tokens(42, 2, 1, "bf16", spread=1.0)
    append(case, c, k)
    out, lse = case.decode("f32")
    case.table = small
    case.ckv, case.kpe, case.scales = orc.cache_append_q8(case.ckv, case.kpe, case.scales, small, case.lens,
                                                          orc.decode16(c, "bf16"), orc.decode16(k, "bf16"))
    for whole, part in zip((pool.ckv, pool.kpe, pool.scales), (case.ckv, case.kpe, case.scales)):
        assert np.array_equal(whole[nblk - n:].cpu().numpy(), part)
    case.check(out, lse)


COLD = """
import sys
import numpy as np
import tests.test_gpu_q8 as t
from mla_split_kv_gb300 import binding as nb
nb.load()
for H, dtype in ((16, "f16"), (16, "bf16"), (64, "f16"), (64, "bf16")):
    case = t.Q8Case(50, [30001, 0, 4000], H=H, bs=32, g=1, dtype=dtype).upload()
    first, first_lse = case.decode("f32")
    for _ in range(3):
        out, lse = case.decode("f32")
    assert t.torch.equal(first, out) and t.torch.equal(first_lse, lse), (H, dtype)
    case.check(first, first_lse, heads=[3, H - 1], requests=[2])
print("same bits")
"""


def test_decode_q8_first_calls_of_a_process():
    """Cold caches spread the warps of a CTA apart as nothing later does: the first call's bits are the later ones'."""
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", COLD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr
