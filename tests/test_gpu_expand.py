"""Keys and values of every head from cached latents, against the products in 64 bits."""
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

pytestmark = pytest.mark.gpu
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
    def __init__(self, seed, lens, H, bs, dtype, spare_rows=0, spare_pages=3):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.H, self.bs, self.dtype = lens, H, bs, TDT[dtype]
        need = [-(-n // bs) for n in lens]
        nblk = sum(need) + spare_pages
        perm = torch.randperm(nblk, device="cuda", generator=g).int()
        self.table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(self.dtype)  # noqa: E731
        self.ckv, self.kpe = rand(nblk, bs, 512), rand(nblk, bs, 64)
        self.w_uk, self.w_uv_t = rand(H, 128, 512), rand(H, 512, 128)
        self.indptr = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        self.S = sum(lens) + spare_rows
        new = lambda *s: torch.full(s, -77.0, dtype=self.dtype, device="cuda")  # noqa: E731
        self.k, self.v, self.k_pe = new(self.S, H, 128), new(self.S, H, 128), new(self.S, 64)

    def run(self, **kw):
        rt.expand_kv(self.ckv, self.kpe, self.table, self.indptr, self.w_uk, self.w_uv_t, self.k, self.v, self.k_pe, **kw)

    def rows(self, b):
        n = self.lens[b]
        ids = self.table[b, : -(-n // self.bs)].long()
        return self.ckv[ids].flatten(0, 1)[:n], self.kpe[ids].flatten(0, 1)[:n]

    def check(self, requests=None):
        """One rounding to the type (half a step of the value, or of the smallest fp16 numbers) and 512 products, exact
        in fp32, added with at most 2^-23 of the sum of their magnitudes lost each time."""
        half = torch.finfo(self.dtype).eps / 2
        tiny = 2.0 ** -25 if self.dtype == torch.float16 else 0.0
        for b in range(len(self.lens)) if requests is None else requests:
            at = int(self.indptr[b])
            c, k_pe = self.rows(b)
            c = c.double()
            assert torch.equal(self.k_pe[at:at + len(c)], k_pe)
            for got, w in ((self.k, self.w_uk.double().transpose(1, 2)), (self.v, self.w_uv_t.double())):
                want = torch.einsum("tr,hrd->thd", c, w)
                size = torch.einsum("tr,hrd->thd", c.abs(), w.abs())
                err = (got[at:at + len(c)].double() - want).abs()
                assert bool((err <= half * want.abs() + tiny + 512 * 2.0 ** -23 * size * (1 + half)).all()), (b, float(err.max()))


@pytest.mark.parametrize("lens,H,bs,dtype", [
    ([1], 1, 16, "f16"), ([1], 16, 64, "bf16"), ([128], 2, 32, "f16"), ([129], 3, 32, "bf16"), ([256], 16, 64, "f16"),
    ([257], 16, 16, "bf16"), ([700, 0, 31, 64, 513], 16, 32, "f16"), ([0, 0, 40, 0], 5, 16, "bf16"),
    ([2500, 300], 8, 64, "bf16"), ([37] * 90, 7, 16, "f16"), ([1] * 700, 2, 32, "bf16"), ([1000], 128, 64, "f16")])
def test_against_64_bits(lens, H, bs, dtype):
    case = Case(len(lens) * 100 + H, lens, H, bs, dtype, spare_rows=5)
    nb.mla_reset_counters()
    case.run()
    torch.cuda.synchronize()
    assert nb.mla_get_counters()[nb.CTR_PREFILL] == 1
    case.check()
    n = sum(lens)
    assert bool((case.k[n:] == -77).all()) and bool((case.v[n:] == -77).all()) and bool((case.k_pe[n:] == -77).all())


def test_many_tiles_a_pair():
    """Several blocks of a long request, and blocks of others, in one pair's run of tiles; sampled requests."""
    lens = [20000, 1, 0, 300, 5000] + [257] * 20
    case = Case(3, lens, 16, 64, "bf16")
    case.run()
    torch.cuda.synchronize()
    case.check([0, 1, 3, 4, 24])


def test_no_tokens_at_all():
    case = Case(4, [0, 0], 4, 16, "f16", spare_rows=3)
    case.run()
    torch.cuda.synchronize()
    assert bool((case.k == -77).all())


def test_tokens_past_the_outputs_are_left_out():
    case = Case(5, [100, 60], 2, 16, "f16")
    guard = torch.full((200, 2, 128), -5.0, dtype=torch.float16, device="cuda")
    case.S = 130
    case.k, case.v, case.k_pe = guard[:130], case.v[:130], case.k_pe[:130]
    case.run()
    torch.cuda.synchronize()
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2
    assert bool((guard[130:] == -5).all())
    case.lens = [100, 30]
    case.check()


def test_a_page_outside_the_pool_reads_zeros():
    case = Case(6, [40, 33], 2, 16, "bf16")
    case.table[0, 1] = 10 ** 6
    case.run()
    torch.cuda.synchronize()
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2
    assert bool((case.k[16:32] == 0).all()) and bool((case.v[16:32] == 0).all()) and bool((case.k_pe[16:32] == 0).all())
    case.check([1])


def test_a_token_that_is_not_finite_stays_with_its_rows():
    case = Case(7, [300], 4, 32, "bf16")
    page = int(case.table[0, 4])
    case.ckv[page, 3] = float("nan")
    case.run()
    torch.cuda.synchronize()
    t = 4 * 32 + 3
    assert bool(case.k[t].isnan().all()) and bool(case.v[t].isnan().all())
    finite = torch.ones(300, dtype=torch.bool, device="cuda")
    finite[t] = False
    assert bool(torch.isfinite(case.k[finite]).all()) and bool(torch.isfinite(case.v[finite]).all())


def test_captured_calls_on_a_stream_of_their_own():
    case = Case(8, [500, 77], 16, 32, "f16")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    case.run()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        case.run(stream=side)
    want = case.k.clone(), case.v.clone()
    for _ in range(3):
        case.k.zero_(), case.v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(case.k, want[0]) and torch.equal(case.v, want[1])
    case.check()
