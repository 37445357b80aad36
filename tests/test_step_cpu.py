"""Refusals of the step's entry points, before anything is launched."""
import ctypes

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

GOOD = 0x10000  # an aligned address that no launch ever sees


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


def refused(call, status):
    nb.mla_reset_counters()
    with pytest.raises(nb.MlaError) as e:
        call()
    assert e.value.status == status
    ctr = nb.mla_get_counters()
    assert ctr[nb.CTR_REJECTED] == 1 and ctr[nb.CTR_STEP] == 0


def tables(args=None, **kw):
    d = nb.mla_step_desc_t(4, 32, 100, 10, 64, None)
    for k, v in kw.items():
        setattr(d, k, v)
    a = [GOOD] * 11
    for i, v in (args or {}).items():
        a[i] = v
    nb.mla_update_tables(*a, d)


@pytest.mark.parametrize("i", range(11))
def test_tables_need_every_buffer(i):
    refused(lambda: tables({i: None}), nb.MLA_ERR_INVALID_ARG)
    refused(lambda: tables({i: GOOD + (4 if i == 9 else 2)}), nb.MLA_ERR_INVALID_ARG)


@pytest.mark.parametrize("field,value,status", [
    ("num_requests", 0, nb.MLA_ERR_INVALID_ARG), ("num_requests", 8193, nb.MLA_ERR_UNSUPPORTED),
    ("num_blocks", 0, nb.MLA_ERR_INVALID_ARG), ("max_blocks_per_req", 0, nb.MLA_ERR_INVALID_ARG),
    ("capacity", 0, nb.MLA_ERR_INVALID_ARG), ("block_size", 48, nb.MLA_ERR_UNSUPPORTED), ("block_size", 8, nb.MLA_ERR_UNSUPPORTED)])
def test_tables_refuse_shapes(field, value, status):
    refused(lambda: tables(**{field: value}), status)


def append(**kw):
    a = dict(ckv_new=GOOD, ckv_stride=576, kpe_new=GOOD, kpe_stride=576, slots=GOOD, num_tokens=3, block_size=32,
             num_blocks=5, ckv_cache=GOOD, kpe_cache=GOOD, stream=None)
    a.update(kw)
    nb.mla_cache_append_slots(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(ckv_new=None), 1), (dict(kpe_new=None), 1), (dict(slots=None), 1), (dict(ckv_cache=None), 1), (dict(kpe_cache=None), 1),
    (dict(num_tokens=0), 1), (dict(num_tokens=2 ** 31), 1), (dict(num_blocks=0), 1), (dict(block_size=24), 2),
    (dict(ckv_stride=504), 1), (dict(ckv_stride=580), 1), (dict(kpe_stride=56), 1), (dict(kpe_stride=68), 1),
    (dict(ckv_new=GOOD + 8), 1), (dict(kpe_new=GOOD + 8), 1), (dict(slots=GOOD + 4), 1), (dict(ckv_cache=GOOD + 8), 1)])
def test_append_refuses(kw, status):
    refused(lambda: append(**kw), status)


def test_step_descriptor_has_the_headers_layout():
    d = nb.mla_step_desc_t
    assert [getattr(d, n).offset for n, _ in d._fields_] == [0, 4, 8, 12, 16, 24] and ctypes.sizeof(d) == 32


def test_buffers_off_the_gpu_are_refused():
    with pytest.raises(ValueError):
        pool = rt.alloc_pool(4, 32, device="cpu")
        step = rt.alloc_step(2, 8, device="cpu")
        z = torch.zeros(2, dtype=torch.int32)
        rt.update_tables(pool, z, z.clone(), torch.zeros(2, 2, dtype=torch.int32), step)
    with pytest.raises(ValueError):
        t = torch.zeros(2, 16, 512, dtype=torch.float16)
        rt.cache_append_slots(t, t[..., :64].contiguous(), t[0], t[0, :, :64], torch.zeros(16, dtype=torch.int64))
