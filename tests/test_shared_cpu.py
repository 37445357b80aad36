"""The plan of a batch with a common prefix, and the refusals of its entry points, before anything is launched."""
import ctypes

import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild

GOOD = 0x10000  # an aligned address that no launch ever sees


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


def device(sms=152):
    dev = nb.mla_device_info_t()
    dev.num_sms = sms
    return dev


@pytest.mark.parametrize("lens,shared,H,q_len,bs,sms", [
    ([65], 64, 16, 1, 64, 152), ([0], 16, 16, 1, 16, 152), ([10, 0, 3], 512, 128, 3, 32, 152), ([5000] * 40, 4096, 16, 1, 32, 152),
    ([100000, 70000, 66000], 65536, 128, 1, 64, 152), ([2 ** 31 - 1], 2 ** 20, 64, 1, 64, 152), ([700 + 37 * i for i in range(300)], 640, 16, 1, 16, 152),
    ([900, 1000], 512, 64, 5, 32, 7), ([300] * 9, 256, 16, 32, 16, 1), ([300, 300], 256, 16, 9, 16, 200)])
def test_a_plan_covers_every_token_of_every_row_once(lens, shared, H, q_len, bs, sms):
    plan = nb.mla_plan_shared(lens, shared, H, q_len, bs, device(sms))
    B, per = len(lens), q_len * H
    rows, own_groups = B * per, -(-per // 128)
    groups = -(-rows // 128)
    assert plan.cta_indptr[0] == 0 and plan.cta_indptr[-1] == len(plan.units) and len(plan.cta_indptr) - 1 <= sms
    assert all(a <= b for a, b in zip(plan.cta_indptr, plan.cta_indptr[1:]))
    # every slot has one piece, which is two units: a half of the columns each
    by_slot = {}
    for row0, n, request, t0, t1, slot, half in plan.units:
        by_slot.setdefault(slot, []).append((half, row0, n, request, t0, t1))
    assert sorted(by_slot) == list(range(plan.num_slots))
    for units in by_slot.values():
        units.sort()
        assert [u[0] for u in units] == [0, 1] and units[0][1:] == units[1][1:]

    def covers(slots, row0, n, request, t0, end):
        at = t0
        for slot in slots:
            _, r, m, q, a, e = by_slot[slot][0]
            assert (r, m, q, a) == (row0, n, request, at) and e >= a
            assert (e - t0) % 64 == 0 or slot == slots[-1]
            at = e
        assert at == end

    for g in range(groups):
        slots = range(g * plan.shared_parts, (g + 1) * plan.shared_parts)
        covers(slots, g * 128, min(128, rows - g * 128), -1, 0, shared)
    assert len(plan.own_indptr) == B * own_groups + 1
    assert plan.own_indptr[0] == groups * plan.shared_parts and plan.own_indptr[-1] == plan.num_slots
    for b in range(B):
        for g in range(own_groups):
            i = b * own_groups + g
            slots = range(plan.own_indptr[i], plan.own_indptr[i + 1])
            assert len(slots) >= 1  # (the last one takes what the request grows by)
            covers(slots, b * per + g * 128, min(128, per - g * 128), b, shared, 2 ** 31 - 1)


def test_the_busiest_cta_of_a_plan_is_not_far_above_the_average():
    """Equal requests beside a long prefix: no CTA has more than 1.3 times the average of tiles of 64 tokens and six a
    unit, the time of its start and end."""
    plan = nb.mla_plan_shared([20000] * 32, 16384, 128, 1, 64, device())
    load = [sum(-(-(min(t1, 20000) - t0) // 64) + 6 for _, _, _, t0, t1, _, _ in plan.units[a:b])
            for a, b in zip(plan.cta_indptr, plan.cta_indptr[1:])]
    assert len(load) == 152 and max(load) <= 1.3 * sum(load) / len(load)


@pytest.mark.parametrize("lens,shared,H,q_len,bs,status", [
    ([], 64, 16, 1, 16, 1), ([100, -1], 64, 16, 1, 16, 1), ([100], 0, 16, 1, 16, 1), ([100], 72, 16, 1, 16, 1), ([100], 48, 16, 1, 32, 1),
    ([100], 64, 32, 1, 16, 2), ([100], 64, 16, 0, 16, 2), ([100], 64, 16, 33, 16, 2), ([100], 64, 16, 1, 8, 2)])
def test_plans_are_refused(lens, shared, H, q_len, bs, status):
    with pytest.raises(nb.MlaError) as e:
        nb.mla_plan_shared(lens, shared, H, q_len, bs, device())
    assert e.value.status == status


def test_a_plan_that_does_not_fit_says_how_many_units_it_has(lib):
    lens, plan, dev = (ctypes.c_int32 * 2)(500, 600), nb.mla_shared_plan_t(), device()
    units, own, ctas = (nb.mla_shared_unit_t * 1)(), (ctypes.c_int32 * 3)(), (ctypes.c_int32 * 153)()
    plan.shared_tokens, plan.unit_capacity = 256, 1
    for name, x in (("units", units), ("own_indptr", own), ("cta_indptr", ctas)):
        setattr(plan, name, ctypes.cast(x, type(getattr(plan, name))))
    args = (lens, 2, 16, 1, 32, ctypes.byref(dev))
    assert lib.mla_plan_shared(*args, ctypes.byref(plan)) == nb.MLA_ERR_CAPACITY
    assert plan.num_units == len(nb.mla_plan_shared([500, 600], 256, 16, 1, 32, dev).units) > 1 and units[0].rows == 0
    for bad in ((None, *args[1:], ctypes.byref(plan)), (*args[:-1], None, ctypes.byref(plan)), (*args, None)):
        assert lib.mla_plan_shared(*bad) == nb.MLA_ERR_INVALID_ARG
    plan.unit_capacity = plan.num_units  # but no room given
    plan.units = None
    assert lib.mla_plan_shared(*args, ctypes.byref(plan)) == nb.MLA_ERR_INVALID_ARG


def decode(args=None, **kw):
    d = nb.mla_shared_desc_t(4, 16, 1, 32, 100, 10, nb.MLA_BF16, 0, 64, nb.MLA_F32, GOOD, GOOD, GOOD, 10, 5, 1, 10, GOOD, 2 ** 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    a = [GOOD] * 7 + [0.1, GOOD, GOOD]
    for i, v in (args or {}).items():
        a[i] = v
    nb.mla_decode_shared(*a, d)


def refused(call, status):
    nb.mla_reset_counters()
    with pytest.raises(nb.MlaError) as e:
        call()
    assert e.value.status == status
    ctr = nb.mla_get_counters()
    assert ctr[nb.CTR_REJECTED] == 1 and ctr[nb.CTR_DECODE_SHARED] == 0


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5, 6, 8, 9])
def test_decode_needs_every_buffer(i):
    if i != 9:  # (the LSE may be left out)
        refused(lambda: decode({i: None}), nb.MLA_ERR_INVALID_ARG)
    refused(lambda: decode({i: GOOD + (2 if i in (4, 5, 6, 9) else 8)}), nb.MLA_ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=0), 1), (dict(num_requests=2 ** 30), 2), (dict(num_heads=32), 2), (dict(q_len=0), 2), (dict(q_len=33), 2),
    (dict(block_size=8), 2), (dict(num_blocks=0), 1), (dict(num_blocks=2 ** 26), 2), (dict(max_blocks_per_req=0), 1),
    (dict(dtype=nb.MLA_F32), 2), (dict(dtype=nb.MLA_E4M3), 2), (dict(out_dtype=nb.MLA_E4M3), 2), (dict(causal=2), 1),
    (dict(shared_tokens=0), 1), (dict(shared_tokens=72), 1), (dict(units=None), 1), (dict(units=GOOD + 8), 1), (dict(own_indptr=None), 1),
    (dict(own_indptr=GOOD + 2), 1), (dict(cta_indptr=None), 1), (dict(cta_indptr=GOOD + 2), 1), (dict(num_units=0), 1), (dict(num_slots=0), 1),
    (dict(shared_parts=0), 1), (dict(num_ctas=0), 1), (dict(num_ctas=65536), 2), (dict(workspace=None), 1), (dict(workspace=GOOD + 8), 1),
    (dict(workspace_bytes=5 * 128 * 513 * 4 - 1), 1), (dict(args={7: float("nan")}), 1), (dict(args={7: float("-inf")}), 1)])
def test_decode_refuses(kw, status):
    refused(lambda: decode(**kw), status)


def test_workspace():
    assert [nb.mla_decode_shared_workspace_bytes(n) for n in (-1, 0, 1, 7)] == [0, 0, 128 * 513 * 4, 7 * 128 * 513 * 4]


def test_descriptors_have_the_headers_layout():
    def offsets(t):
        return [getattr(t, n).offset for n, _ in t._fields_], ctypes.sizeof(t)

    assert offsets(nb.mla_shared_unit_t) == ([0, 4, 8, 12, 16, 20, 24, 28], 32)
    assert offsets(nb.mla_shared_plan_t) == ([0, 4, 8, 16, 24, 32, 36, 40, 44], 48)
    assert offsets(nb.mla_shared_desc_t) == ([*range(0, 40, 4), 40, 48, 56, 64, 68, 72, 76, 80, 88, 96], 104)
