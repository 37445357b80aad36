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


def prefill(args=None, strides=None, **kw):
    d = nb.mla_prefill_desc_t(4, 16, nb.MLA_BF16, 1, 500, 900, (2048, 128), (1024, 64), GOOD, 2 ** 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    if strides is not None:
        d.q_nope_stride, d.q_pe_stride = strides
    a = [GOOD] * 7 + [0.1, GOOD, GOOD]
    for i, v in (args or {}).items():
        a[i] = v
    nb.mla_prefill(*a, d)


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5, 6, 8, 9])
def test_prefill_needs_every_buffer(i):
    if i != 9:  # (the LSE may be left out)
        refused(lambda: prefill({i: None}), nb.MLA_ERR_INVALID_ARG)
    off = {5: 2, 6: 2, 8: 16, 9: 2}.get(i, 8)
    refused(lambda: prefill({i: GOOD + off}), nb.MLA_ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=0), 1), (dict(num_requests=8193), 2), (dict(num_heads=0), 2), (dict(num_heads=257), 2),
    (dict(dtype=nb.MLA_F32), 2), (dict(dtype=nb.MLA_E4M3), 2), (dict(causal=2), 1), (dict(max_q_tokens=0), 1),
    (dict(max_kv_tokens=0), 1), (dict(max_kv_tokens=2 ** 31 - 1), 2), (dict(max_q_tokens=2 ** 31 - 1, num_heads=256), 2),
    (dict(strides=((2048, 120), (1024, 64))), 1), (dict(strides=((2048, 132), (1024, 64))), 1), (dict(strides=((64, 128), (1024, 64))), 1),
    (dict(strides=((2048, 128), (1024, 56))), 1), (dict(strides=((2048, 128), (2 ** 39, 64))), 1),
    (dict(args={7: float("nan")}), 1), (dict(args={7: float("inf")}), 1)])
def test_prefill_refuses(kw, status):
    refused(lambda: prefill(**kw), status)


def test_prefill_workspace():
    dev = nb.mla_device_info_t()
    dev.num_sms = 152
    sizes = [nb.mla_prefill_workspace_bytes(dev, 4, 16, T) for T in (1, 500, 100000)]
    assert 0 < sizes[0] <= sizes[1] < sizes[2]
    for bad in ((0, 16, 1), (8193, 16, 1), (1, 0, 1), (1, 257, 1), (1, 1, 0)):
        assert nb.mla_prefill_workspace_bytes(dev, *bad) == 0


def test_descriptors_have_the_headers_layout():
    import ctypes
    d = nb.mla_prefill_desc_t
    assert [getattr(d, n).offset for n, _ in d._fields_] == [0, 4, 8, 12, 16, 20, 24, 40, 56, 64, 72] and ctypes.sizeof(d) == 80
    e = nb.mla_expand_desc_t
    assert [getattr(e, n).offset for n, _ in e._fields_] == [0, 4, 8, 12, 16, 20, 24, 32] and ctypes.sizeof(e) == 40
