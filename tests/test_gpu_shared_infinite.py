"""Infinite latents whose score is -inf, in decode attention of a batch with a common prefix: a weight of 0 times an infinite
value is NaN in that value's column for every row that sees the token, wherever its tile and its piece lie."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from tests.test_gpu_shared import Case

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


COLUMNS = (7, 255, 256, 300, 511)  # of both halves, at their ends


def poison(case, b, token, column):
    """An infinity at this token and column, which every query gives a score of -inf."""
    sign = -1.0 if column % 2 else 1.0
    case.ckv.view(-1, 512)[case.rows_of(b, token + 1)[token], column] = sign * math.inf
    case.q_abs[..., column] = -sign * case.q_abs[..., column].abs().clamp(min=0.01)


def check(case, out, lse):
    """NaN exactly in the columns of infinities that the row sees; else within the bounds of test_gpu_shared's check, of the
    tokens with a finite score, whose formula these are."""
    half, ulp = torch.finfo(case.dtype).eps / 2, 2.0 ** -23
    for b, L in enumerate(case.lens):
        row = case.rows_of(b, L)
        c, k = case.ckv.view(-1, 512)[row].double(), case.kpe.view(-1, 64)[row].double()
        infinite = c.isinf()
        clean = c.masked_fill(infinite, 0)
        for h in range(case.H):
            q, qp = case.q_abs[b, :, h].double(), case.q_pe[b, :, h].double()
            seen = torch.full((case.q_len,), L, device="cuda")
            if case.causal:
                seen = (L - case.q_len + torch.arange(case.q_len, device="cuda") + 1).clamp(min=0)
            behind = torch.arange(L, device="cuda")[None] >= seen[:, None]
            hidden = behind | infinite.any(1)[None]
            s = ((q @ clean.T + qp @ k.T) * case.scale).masked_fill(hidden, -math.inf)
            mags = abs(case.scale) * (q.abs() @ clean.abs().T + qp.abs() @ k.abs().T)
            ds = (576 * ulp * mags + 8 * ulp * s.abs()).masked_fill(hidden, 0).amax(1)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            want, size = p @ clean, p @ clean.abs()
            tol = (half + 2 * ds + 2.0 ** -19 + 2 * L * ulp)[:, None] * size
            if case.dtype == torch.float16:
                tol = tol + L * 2.0 ** -25 * clean.abs().amax()
            got, got_lse = out[b, :, h].double(), lse[b, :, h].double()
            nan = ((~behind).double() @ infinite.double()) > 0
            assert torch.equal(got.isnan(), nan), (b, h, got.isnan().nonzero().tolist(), nan.nonzero().tolist())
            assert bool((((got - want).abs() <= tol) | nan).all()), (b, h)
            lse_tol = (ds + L * ulp + 2.0 ** -19) / math.log(2.0) + 4 * ulp * z.abs() / math.log(2.0)
            assert bool(((got_lse - z / math.log(2.0)).abs() <= lse_tol).all()), (b, h)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,bs", [(16, 32), (64, 16), (128, 64)])
@pytest.mark.parametrize("other", [700, 550, 330, 100])
def test_common_tokens_whatever_the_other_requests_see(other, H, bs, dtype):
    """The tile of token 300 is one that all rows see, or one that another request's rows do not."""
    case = Case(31, [600, other, 700], 512, H, 1, bs, dtype)
    for t, column in zip((300, 301, 0, 511, 383), COLUMNS):
        poison(case, 2, t, column)
    check(case, *case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[513, 600], [512 + 64, 512 + 65], [512 + 128, 512 + 1], [9000, 513]])
def test_own_tokens(lens, dtype):
    """The last token: in a full tile, beside others in a tile, and alone in a piece, whose every score then is -inf."""
    case = Case(32, lens, 512, 16, 1, 32, dtype)
    for b, column in zip(range(2), COLUMNS[2:]):
        poison(case, b, lens[b] - 1, column)
    poison(case, 0, 40, 7)
    check(case, *case.run())


@pytest.mark.parametrize("H,q_len", [(16, 4), (64, 3), (128, 2), (16, 32)])
def test_a_causal_window(H, q_len):
    """Tokens of the window, which its last rows see and its first do not, and common ones that a request that is shorter than
    the prefix does not have."""
    case = Case(33, [300, 290, 250], 256, H, q_len, 16, "bf16", True)
    for b, L in enumerate(case.lens):
        poison(case, b, L - 1, COLUMNS[b])
    poison(case, 0, 300 - q_len, 300)
    poison(case, 0, 252, 511)
    check(case, *case.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shared", [16, 48, 528, 1632])
def test_a_prefix_that_ends_inside_a_tile(shared, dtype):
    """Its last tile is masked although every row sees all of its tokens."""
    case = Case(35, [shared + 90, shared + 200, shared + 64], shared, 64, 2, 16, dtype, True)
    for t, column in zip((shared - 1, shared - 16, shared // 64 * 64 if shared % 64 else shared - 64), COLUMNS):
        poison(case, 0, t, column)
    check(case, *case.run())


def test_pieces_and_units_in_turns():
    """Many units a CTA, some with such a token and some without, in tiles that are masked."""
    case = Case(34, [2048 + 37 * i for i in range(40)], 2048, 16, 1, 16, "bf16")
    for b in range(3, 40, 3):
        poison(case, b, case.lens[b] - 1 - b % 5, COLUMNS[b % 5])
    check(case, *case.run())
