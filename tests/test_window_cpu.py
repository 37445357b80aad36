"""Windowed attention on the CPU: the visible runs against brute force, plans made from them, refusals."""
import ctypes

import numpy as np
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from oracle import mla_oracle as orc
from tests.test_abi_cpu import desc, fake_gb300

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("q_len,causal", [(1, False), (1, True), (5, True), (5, False), (32, True)])
def test_window_lens_count_the_pages_that_some_row_sees(bs, q_len, causal):
    lens = list(range(0, 4 * bs)) + [1000, 1023, 1024, 4099]
    for W in (1, 2, bs - 1, bs, bs + 1, 200, 2 ** 31 - 1):
        for S in (0, 1, bs, bs + 1, 150, 2 ** 31 - 1):
            got = nb.mla_window_lens(lens, q_len, bs, causal, W, S)
            for L, n in zip(lens, got):
                seen = np.zeros(L, bool)
                for i in range(q_len):
                    seen |= orc.visible_window(L, q_len, i, causal, W, S)
                # the run reads whole pages: from the sinks' up to the first gap, then from the window's first to the end
                first = (L - q_len if causal else L - 1) - W + 1
                low = max(0, first) // bs * bs
                sink_end = min(-(-S // bs) * bs, low)
                assert n == sink_end + L - low, (L, W, S)
                read = np.zeros(L, bool)
                read[:sink_end], read[low:] = True, True
                assert not (seen & ~read).any()


def test_window_lens_of_a_long_context_repeat_with_the_page():
    for bs in (16, 64):
        runs = nb.mla_window_lens(range(5000, 5000 + 3 * bs), 1, bs, False, 700, 4)
        assert runs[:bs] == runs[bs:2 * bs] == runs[2 * bs:]
        assert max(runs) <= bs + 700 + bs and min(runs) >= 700


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), nb.MLA_ERR_INVALID_ARG), (dict(window=-5), nb.MLA_ERR_INVALID_ARG), (dict(sinks=-1), nb.MLA_ERR_INVALID_ARG),
    (dict(B=0), nb.MLA_ERR_INVALID_ARG), (dict(q_len=0), nb.MLA_ERR_UNSUPPORTED), (dict(q_len=33), nb.MLA_ERR_UNSUPPORTED),
    (dict(bs=24), nb.MLA_ERR_UNSUPPORTED), (dict(causal=2), nb.MLA_ERR_INVALID_ARG), (dict(lens=-1), nb.MLA_ERR_INVALID_ARG),
    (dict(), nb.MLA_OK),
])
def test_window_lens_refusals(lib, kw, want):
    a = dict(B=1, q_len=1, bs=32, causal=0, window=10, sinks=0, lens=5)
    a.update(kw)
    lens, out = (ctypes.c_int32 * 1)(a["lens"]), (ctypes.c_int32 * 1)()
    assert lib.mla_window_lens(lens, a["B"], a["q_len"], a["bs"], a["causal"], a["window"], a["sinks"], out) == want
    assert lib.mla_window_lens(None, 1, 1, 32, 0, 10, 0, out) == nb.MLA_ERR_INVALID_ARG
    assert lib.mla_window_lens(lens, 1, 1, 32, 0, 10, 0, None) == nb.MLA_ERR_INVALID_ARG


def call(lib, d, P=2, window=100, sinks=4, ptr=FAKE):
    return lib.mla_decode_window(*([FAKE] * 6), 0.1, P, FAKE, FAKE, FAKE, ptr, nb.MLA_F16, None, window, sinks, d)


@pytest.mark.parametrize("kw,args,want", [
    (dict(), dict(window=0), nb.MLA_ERR_INVALID_ARG), (dict(), dict(window=-1), nb.MLA_ERR_INVALID_ARG),
    (dict(), dict(sinks=-1), nb.MLA_ERR_INVALID_ARG), (dict(kernel=nb.MLA_KERNEL_SIMT), {}, nb.MLA_ERR_UNSUPPORTED),
    (dict(cluster_ctas=1), {}, nb.MLA_ERR_UNSUPPORTED), (dict(num_heads=64, cluster_ctas=4), {}, nb.MLA_ERR_UNSUPPORTED),
    (dict(num_heads=32), {}, nb.MLA_ERR_UNSUPPORTED), (dict(q_len=33), {}, nb.MLA_ERR_UNSUPPORTED),
    (dict(block_size=128), {}, nb.MLA_ERR_UNSUPPORTED), (dict(), dict(P=0), nb.MLA_ERR_INVALID_ARG),
    (dict(), dict(ptr=None), nb.MLA_ERR_INVALID_ARG), (dict(), dict(ptr=FAKE + 8), nb.MLA_ERR_INVALID_ARG),
    (dict(num_heads=16, q_len=1, cluster_ctas=2), {}, nb.MLA_ERR_INVALID_ARG),  # no workspace
])
def test_decode_window_rejects_before_launch(lib, kw, args, want):
    before = nb.mla_get_counters()
    assert call(lib, desc(**{"cluster_ctas": 2, **kw}), **args) == want
    after = nb.mla_get_counters()
    assert after[nb.CTR_REJECTED] == before[nb.CTR_REJECTED] + 1 and after[nb.CTR_PARTIAL_TC] == before[nb.CTR_PARTIAL_TC]


def test_decode_window_rejects_a_null_descriptor(lib):
    assert call(lib, None) == nb.MLA_ERR_INVALID_ARG


def test_a_plan_of_the_runs_covers_them():
    lens = [131072, 5000, 100, 0]
    runs = nb.mla_window_lens(lens, 1, 32, False, 4096, 4)
    plan = nb.mla_plan(runs, 16, 1, 32, fake_gb300())
    for b, n in enumerate(runs):
        chunks = plan.chunks[plan.o_indptr[b]:plan.o_indptr[b + 1]]
        assert chunks[0][1] == 0 and chunks[-1][2] == n


@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 4), (64, 1), (128, 1), (128, 32)])
@pytest.mark.parametrize("lens", [[1], [40], [300], [4200], [131072], [0, 0], [0, 1, 129, 257, 700], [2048] * 16, [4224] * 32,
                                  [100] * 200, [9000] + [1] * 90])
def test_window_partitions_cover_the_runs_in_order(lens, H, q_len):
    """Whatever plan is taken: a request's partitions follow one another from its first token to its last, none of a
    split run is empty, slots are numbered in order, and the pair kernels can run it."""
    bs, dev = 32, fake_gb300()
    plan = rt._window_partitions(lens, H, q_len, bs, "f16", dev)
    assert plan.cluster_ctas >= 2 and (H * q_len <= 16 or plan.cluster_ctas == 2)
    assert plan.o_indptr[0] == 0 and plan.o_indptr[-1] == plan.num_chunks == len(plan.chunks)
    for b, n in enumerate(lens):
        at = 0
        parts = plan.chunks[plan.o_indptr[b]:plan.o_indptr[b + 1]]
        for k, (rb, t0, t1, slot) in enumerate(parts):
            assert rb == b and t0 == at and slot == plan.o_indptr[b] + k
            assert t1 > t0 or (len(parts) == 1 and n == 0)
            at = t1
        assert parts and at == n


@pytest.mark.parametrize("q_len,causal", [(1, False), (5, True)])
def test_a_window_plan_covers_growing_contexts(monkeypatch, q_len, causal):
    """With `grow`, every run up to that many tokens later is covered, whatever the page phase; without, the very
    next one may not be."""
    monkeypatch.setattr(rt, "alloc_partials", lambda *a, **k: (None, None))
    monkeypatch.setattr(rt, "alloc_decode_workspace", lambda *a, **k: None)
    bs, W, S, dev = 32, 300, 5, fake_gb300()
    lens = [0, 1, 290, 310, 1000, 1023, 5000]
    covered = lambda plan: [plan.plan.chunks[plan.plan.o_indptr[b + 1] - 1][2] for b in range(len(lens))]  # noqa: E731
    missed = False
    for grow in (0, 1, 20, 33, 400):
        got = covered(rt.plan_window(lens, 16, q_len, bs, W, S, causal=causal, dev=dev, device="cpu", grow=grow))
        for more in range(grow + 1):
            runs = nb.mla_window_lens([n + more for n in lens], q_len, bs, causal, W, S)
            assert all(n <= c for n, c in zip(runs, got)), (grow, more)
        if grow == 0:
            runs = nb.mla_window_lens([n + 1 for n in lens], q_len, bs, causal, W, S)
            missed = any(n > c for n, c in zip(runs, got))
    assert missed
    with pytest.raises(ValueError):
        rt.plan_window(lens, 16, q_len, bs, W, S, dev=dev, device="cpu", grow=-1)
