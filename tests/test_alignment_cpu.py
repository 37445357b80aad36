"""Addresses that vector stores need, refused on the host where they are not kept."""
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild

GOOD = 0x10000  # an aligned address that no launch ever sees


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


@pytest.mark.parametrize("off", [4, 8, 16, 48, 80])
def test_partial_outputs_of_the_common_prefix_need_32_bytes(off):
    """A unit's partial outputs go out 32 bytes a store: a workspace at 16 of 32 would put every one of them across."""
    d = nb.mla_shared_desc_t(4, 16, 1, 32, 100, 10, nb.MLA_BF16, 0, 64, nb.MLA_F32, GOOD, GOOD, GOOD, 10, 5, 1, 10, GOOD + off, 2 ** 40, None)
    nb.mla_reset_counters()
    with pytest.raises(nb.MlaError) as e:
        nb.mla_decode_shared(*[GOOD] * 7, 0.1, GOOD, GOOD, d)
    assert e.value.status == nb.MLA_ERR_INVALID_ARG
    ctr = nb.mla_get_counters()
    assert ctr[nb.CTR_REJECTED] == 1 and ctr[nb.CTR_DECODE_SHARED] == 0
