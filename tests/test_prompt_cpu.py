"""Refusals of the prompt's entry points, before anything is launched."""
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild

GOOD = 0x10000  # an aligned address that no launch ever sees


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


def refused(call, status, launches=nb.CTR_PREFILL):
    nb.mla_reset_counters()
    with pytest.raises(nb.MlaError) as e:
        call()
    assert e.value.status == status
    ctr = nb.mla_get_counters()
    assert ctr[nb.CTR_REJECTED] == 1 and ctr[launches] == 0


def expand(args=None, **kw):
    d = nb.mla_expand_desc_t(4, 16, 32, 100, 10, nb.MLA_BF16, 500, None)
    for k, v in kw.items():
        setattr(d, k, v)
    a = [GOOD] * 9
    for i, v in (args or {}).items():
        a[i] = v
    nb.mla_expand_kv(*a, d)


@pytest.mark.parametrize("i", range(9))
def test_expand_needs_every_buffer(i):
    refused(lambda: expand({i: None}), nb.MLA_ERR_INVALID_ARG)
    off = {2: 2, 3: 2, 6: 16, 7: 16}.get(i, 8)
    refused(lambda: expand({i: GOOD + off}), nb.MLA_ERR_INVALID_ARG)


@pytest.mark.parametrize("field,value,status", [
    ("num_requests", 0, 1), ("num_heads", 0, 2), ("num_heads", 257, 2), ("block_size", 8, 2), ("num_blocks", 0, 1),
    ("num_blocks", 2 ** 26, 2), ("max_blocks_per_req", 0, 1), ("dtype", nb.MLA_F32, 2), ("dtype", nb.MLA_E4M3, 2), ("max_tokens", 0, 1)])
def test_expand_refuses(field, value, status):
    refused(lambda: expand(**{field: value}), status)
