"""mla_cache_append_q8 beside scales that are no powers of two: each new byte is the nearest one, also where a quotient
in fp32 would come to lie on a tie."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from oracle import mla_oracle as orc
from tests.test_gpu_q8 import Q8Case, append, same_cache

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


def quotients_beside_ties(count):
    """Pairs of a 16-bit value x (exact in both types) and an fp32 scale s whose quotient rounds to a tie in fp32
    and is none; a tie lies halfway between two E4M3 values, at an odd number of sixteenths."""
    rng = np.random.default_rng(61)
    found = []
    while len(found) < count:
        tie = float(rng.choice(np.arange(17, 32, 2)) / 16 * 2.0 ** rng.integers(-3, 7))  # at most 31 / 16 * 64
        x = float(rng.integers(128, 256) * 2.0 ** rng.integers(-6, 3))
        s = np.float32(x / tie)
        if Fraction(x) / Fraction(float(s)) != Fraction(tie) and np.float32(x) / s == np.float32(tie):
            found.append((x, float(s)))
    return found


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_new_values_beside_ties(dtype):
    pairs = quotients_beside_ties(96)
    case = Q8Case(62, [18] * len(pairs), bs=16, g=16, dtype=dtype, pow2=True)
    c, k = np.zeros((len(pairs), 1, 512)), np.zeros((len(pairs), 1, 64))
    for b, (x, s) in enumerate(pairs):
        case.scales[case.table[b, 1], 0] = s  # of token 16, which stays; 17 is new
        c[b, 0, ::3], c[b, 0, 1::3], k[b, 0, 5] = x, -x, x
    case.upload()
    bits = [gen.to_bits(v, dtype) for v in (c, k)]
    exact = [orc.decode16(v, dtype) for v in bits]
    assert np.array_equal(exact[0], c)
    want = orc.cache_append_q8(case.ckv, case.kpe, case.scales, case.table, case.lens, *exact)
    # (the case holds what it is for: a rounding to fp32 in between gives other bytes)
    off = [orc.encode_e4m3(np.array([np.float64(np.float32(x) / np.float32(s))]))[0] != orc.encode_e4m3(np.array([x / s]))[0] for x, s in pairs]
    assert sum(off) > 20
    append(case, *bits)
    same_cache(case, want)
