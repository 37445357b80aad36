"""How exactly the block-scaled attention keeps the weights of its value product."""
import math

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from oracle import mla_oracle as orc
from tests.test_gpu_q8 import SCALE, Q8Case

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


@pytest.mark.parametrize("H,q_len,dtype,terms", [(16, 1, "f16", 4), (16, 1, "bf16", 4), (64, 1, "f16", 3), (128, 1, "bf16", 3),
                                                 (16, 5, "bf16", 3)])
def test_a_weight_between_powers_of_two_keeps_its_bits(H, q_len, dtype, terms):
    """Two tokens: one without latent values sets the row's reference, the other lies 0 to 4 powers of two below it
    and alone makes the output. Relative to it: an E4M3 term leaves at most 2^-4, 2^-9, 2^-14 of a value in [1, 2),
    and what the first leaves is held in 11 bits (2^-16), so three terms are off by 2^-14 + 2^-16 and four by
    2^-16. The score is one product of a 16-bit query and 8, exact in fp32, up to 4 in log2 units: at most four
    roundings (scale, log2 e, factor, difference) of 2^-24 * 4 each in the exponent, 2^-20 of the weight, doubled by
    the sum; the exponential, the sums, the quotient and the combination of terms add at most 16 units of 2^-24."""
    case = Q8Case(71, [2], H=H, q_len=q_len, bs=16, g=1, dtype=dtype, pow2=True)
    rng = np.random.default_rng(72)
    rows = orc.physical_rows(case.table[0], 2, 16)
    ckv, kpe = case.ckv.reshape(-1, 512), case.kpe.reshape(-1, 64)
    ckv[rows[0]] = 0
    ckv[rows[1]] = orc.encode_e4m3(rng.integers(1, 16, size=512) * np.exp2(rng.integers(-3, 3, size=512)) * rng.choice([-1.0, 1.0], size=512))
    kpe[rows] = 0
    kpe[rows[0], 0] = orc.encode_e4m3(np.full(1, 8.0))[0]
    case.scales[:] = 1.0
    gap = rng.uniform(0.0, 4.0, size=(1, q_len, H))  # log2 of the ratio of the two weights
    q_pe = np.zeros((1, q_len, H, 64))
    q_pe[..., 0] = gap * math.log(2.0) / SCALE / 8
    case.q_abs, case.q_pe = gen.to_bits(np.zeros((1, q_len, H, 512)), dtype), gen.to_bits(q_pe, dtype)
    case.upload()
    out, lse = case.decode("f32")
    c, k = case.rows(0)
    ref, ref_lse = orc.attend_rows(orc.decode16(case.q_abs[0], dtype), orc.decode16(case.q_pe[0], dtype), c, k, SCALE, False)
    kept = {3: 2.0 ** -14 + 2.0 ** -16, 4: 2.0 ** -16}[terms]
    err = np.abs(out[0].double().cpu().numpy() - ref)
    tol = (kept + 2.0 ** -19 + 16 * 2.0 ** -24) * np.abs(ref)
    assert np.all(err <= tol), float((err / np.abs(ref)).max())
    assert np.abs(lse[0].double().cpu().numpy() - ref_lse).max() <= 2.0 ** -18
