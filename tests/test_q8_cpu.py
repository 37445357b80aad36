"""Block-scaled 8-bit caches and windows on the CPU: the oracle's pieces against brute force, the descriptor's
layout, and every refusal of the entry points before any launch."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from oracle import mla_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return nb.load()


# --- the oracle's pieces ------------------------------------------------------------


def test_encode_e4m3_is_the_nearest_pattern():
    values = orc.decode_e4m3(np.arange(256, dtype=np.uint8))
    finite = np.isfinite(values)
    assert np.array_equal(orc.decode_e4m3(orc.encode_e4m3(values[finite])), values[finite])
    x = np.concatenate([np.random.default_rng(1).standard_normal(2000) * 2.0 ** np.arange(-10, 10).repeat(100), [500.0, -1e9, 2.0 ** -10, 3 * 2.0 ** -11]])
    got = orc.decode_e4m3(orc.encode_e4m3(x))
    best = np.abs(np.clip(x, -448, 448)[:, None] - values[finite][None]).min(1)
    assert np.array_equal(np.abs(np.clip(x, -448, 448) - got), best)
    # a tie goes to the even mantissa: 17 lies between 16 (mantissa 0) and 18 (1), 2^-10 between 0 and 2^-9
    assert list(orc.decode_e4m3(orc.encode_e4m3(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])))) == [16, 20, 0, 2.0 ** -8]
    # torch's own conversion of the same values agrees
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(orc.decode_e4m3(orc.encode_e4m3(np.clip(x, -448, 448).astype(np.float32).astype(np.float64))), want)


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.5, 2.0), (0.0, 2.0 ** -60), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                       (1.76, 2.0 ** -7), (math.inf, math.nan), (448 * 2.0 ** 60, 2.0 ** 60), (449 * 2.0 ** 60, math.nan)])
def test_block_scale(amax, want):
    got = orc.block_scale(amax)
    assert got == want or (math.isnan(got) and math.isnan(want))


def test_visible_window_brute_force():
    for n in range(0, 12):
        for q in (1, 3):
            for causal in (False, True):
                for W in (0, 1, 2, 5, 100):
                    for S in (0, 1, 4):
                        if W == 0 and S:
                            continue
                        for i in range(q):
                            got = set(np.flatnonzero(orc.visible_window(n, q, i, causal, W, S)))
                            pos = n - q + i if causal else n - 1
                            want = {t for t in range(n) if (not causal or t <= pos) and (W == 0 or pos - t < W or t < S)}
                            assert got == want


# --- the C ABI ----------------------------------------------------------------------


def test_q8_descriptor_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in nb.mla_q8_desc_t._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"mla_split_kv.h\"\nint main(void) {\n" +
                   "".join(f'  printf("%zu\\n", offsetof(mla_q8_desc_t, {f}));\n' for f in fields) +
                   '  printf("%zu\\n", sizeof(mla_q8_desc_t));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(nb.mla_q8_desc_t, f).offset for f in fields] + [ctypes.sizeof(nb.mla_q8_desc_t)]


def call_append(lib, ckv_new=FAKE, kpe_new=FAKE, dtype=nb.MLA_F16, table=FAKE, lens=FAKE, B=2, q_len=1, bs=32, g=16,
                num_blocks=8, max_blocks=4, ckv=FAKE, kpe=FAKE, scales=FAKE):
    before = nb.mla_get_counters()
    st = lib.mla_cache_append_q8(ckv_new, kpe_new, dtype, table, lens, B, q_len, bs, g, num_blocks, max_blocks, ckv, kpe,
                                 scales, None)
    after = nb.mla_get_counters()
    assert after[nb.CTR_REJECTED] == before[nb.CTR_REJECTED] + 1 and after[nb.CTR_WRAP] == before[nb.CTR_WRAP]
    return st


@pytest.mark.parametrize("kw,want", [
    (dict(ckv_new=None), nb.MLA_ERR_INVALID_ARG), (dict(kpe_new=None), nb.MLA_ERR_INVALID_ARG),
    (dict(table=None), nb.MLA_ERR_INVALID_ARG), (dict(lens=None), nb.MLA_ERR_INVALID_ARG),
    (dict(ckv=None), nb.MLA_ERR_INVALID_ARG), (dict(kpe=None), nb.MLA_ERR_INVALID_ARG),
    (dict(scales=None), nb.MLA_ERR_INVALID_ARG), (dict(ckv_new=FAKE + 8), nb.MLA_ERR_INVALID_ARG),
    (dict(kpe=FAKE + 8), nb.MLA_ERR_INVALID_ARG), (dict(scales=FAKE + 2), nb.MLA_ERR_INVALID_ARG),
    (dict(B=0), nb.MLA_ERR_INVALID_ARG), (dict(q_len=0), nb.MLA_ERR_INVALID_ARG),
    (dict(num_blocks=0), nb.MLA_ERR_INVALID_ARG), (dict(max_blocks=0), nb.MLA_ERR_INVALID_ARG),
    (dict(dtype=nb.MLA_F32), nb.MLA_ERR_UNSUPPORTED), (dict(dtype=nb.MLA_E4M3), nb.MLA_ERR_UNSUPPORTED),
    (dict(bs=48), nb.MLA_ERR_UNSUPPORTED), (dict(g=0), nb.MLA_ERR_INVALID_ARG), (dict(g=3), nb.MLA_ERR_INVALID_ARG),
    (dict(g=64), nb.MLA_ERR_INVALID_ARG), (dict(g=-1), nb.MLA_ERR_INVALID_ARG),
    (dict(B=1 << 20, q_len=1 << 12), nb.MLA_ERR_UNSUPPORTED),
])
def test_append_q8_rejects_before_launch(lib, kw, want):
    assert call_append(lib, **kw) == want


def q8_desc(**kw):
    d = nb.mla_q8_desc_t(2, 16, 1, 32, 8, 4, nb.MLA_F16, 0, 16, 0, 0, nb.MLA_F16, FAKE, 1 << 40, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(num_requests=0), nb.MLA_ERR_INVALID_ARG), (dict(num_requests=65536), nb.MLA_ERR_UNSUPPORTED),
    (dict(num_blocks=0), nb.MLA_ERR_INVALID_ARG), (dict(max_blocks_per_req=0), nb.MLA_ERR_INVALID_ARG),
    (dict(num_heads=32), nb.MLA_ERR_UNSUPPORTED), (dict(q_len=0), nb.MLA_ERR_UNSUPPORTED),
    (dict(q_len=33), nb.MLA_ERR_UNSUPPORTED), (dict(block_size=8), nb.MLA_ERR_UNSUPPORTED),
    (dict(dtype=nb.MLA_E4M3), nb.MLA_ERR_UNSUPPORTED), (dict(dtype=nb.MLA_F32), nb.MLA_ERR_UNSUPPORTED),
    (dict(out_dtype=nb.MLA_E4M3), nb.MLA_ERR_UNSUPPORTED), (dict(causal=2), nb.MLA_ERR_INVALID_ARG),
    (dict(scale_block=24), nb.MLA_ERR_INVALID_ARG), (dict(scale_block=64), nb.MLA_ERR_INVALID_ARG),
    (dict(window=-1), nb.MLA_ERR_INVALID_ARG), (dict(window=5, sinks=-1), nb.MLA_ERR_INVALID_ARG),
    (dict(sinks=4), nb.MLA_ERR_INVALID_ARG), (dict(workspace=None), nb.MLA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 8), nb.MLA_ERR_INVALID_ARG), (dict(num_blocks=1 << 27), nb.MLA_ERR_UNSUPPORTED),
])
def test_decode_q8_rejects_bad_descriptors_before_launch(lib, kw, want):
    before = nb.mla_get_counters()
    st = lib.mla_decode_q8(*([FAKE] * 7), 0.1, FAKE, None, q8_desc(**kw))
    after = nb.mla_get_counters()
    assert st == want and after[nb.CTR_REJECTED] == before[nb.CTR_REJECTED] + 1
    assert after[nb.CTR_DECODE_Q8] == before[nb.CTR_DECODE_Q8]


def test_decode_q8_rejects_null_misaligned_and_a_bad_scale(lib):
    for k in range(9):  # q_abs, q_pe, ckv, kpe, scales, table, lens; then the scale's place is skipped; out
        if k == 7:
            continue
        for bad in (None, FAKE + 1):
            args = [FAKE] * 7 + [0.1, FAKE, None]
            args[k] = bad
            assert lib.mla_decode_q8(*args, q8_desc()) == nb.MLA_ERR_INVALID_ARG, (k, bad)
    assert lib.mla_decode_q8(*([FAKE] * 7), 0.1, FAKE, FAKE + 2, q8_desc()) == nb.MLA_ERR_INVALID_ARG
    assert lib.mla_decode_q8(*([FAKE] * 7), 0.1, FAKE, None, None) == nb.MLA_ERR_INVALID_ARG
    for scale in (math.nan, math.inf, -math.inf):
        assert lib.mla_decode_q8(*([FAKE] * 7), scale, FAKE, None, q8_desc()) == nb.MLA_ERR_INVALID_ARG


def test_decode_q8_workspace_bytes(lib):
    dev = nb.mla_device_info_t()
    dev.num_sms = 152
    for q_len, H in ((1, 16), (4, 16), (1, 128), (32, 128), (9, 64)):
        n = nb.mla_decode_q8_workspace_bytes(dev, q_len, H)
        # at least one open end of every row for each pair of neighbouring gangs, at most two per SM and row of a CTA
        assert n % 16 == 0 and n >= 2 * q_len * H * 514 * 4 and n <= 2 * max(152 * 64, q_len * H + 64) * 514 * 4
    assert nb.mla_decode_q8_workspace_bytes(dev, 0, 16) == 0 and nb.mla_decode_q8_workspace_bytes(dev, 1, 17) == 0
    dev.num_sms = 0
    assert nb.mla_decode_q8_workspace_bytes(dev, 1, 16) == 0


# --- the Python calls ---------------------------------------------------------------


def test_q8_cache_refuses_tensors_of_another_form():
    ckv, kpe = torch.zeros(4, 32, 512, dtype=torch.uint8), torch.zeros(4, 32, 64, dtype=torch.uint8)
    assert rt.Q8Cache(ckv, kpe, torch.ones(4, 2)).scale_block == 16
    for bad in ((ckv[:, :16], kpe, torch.ones(4, 2)), (ckv, kpe[:3], torch.ones(4, 2)), (ckv, kpe, torch.ones(4, 3)),
                (ckv, kpe, torch.ones(4, 2, dtype=torch.float64)), (ckv.float(), kpe, torch.ones(4, 2)),
                (ckv, kpe, torch.ones(2, 4).T), (ckv, kpe, torch.ones(8))):
        with pytest.raises(ValueError):
            rt.Q8Cache(*bad)


def test_q8_calls_refuse_host_tensors():
    cache = rt.Q8Cache(torch.zeros(4, 32, 512, dtype=torch.uint8), torch.zeros(4, 32, 64, dtype=torch.uint8), torch.ones(4, 2))
    tab, ctx = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    new = [torch.zeros(1, 1, n, dtype=torch.float16) for n in (512, 64)]
    with pytest.raises(ValueError):
        rt.cache_append_q8(cache, *new, tab, ctx)
    q = [torch.zeros(1, 1, 16, n, dtype=torch.float16) for n in (512, 64)]
    plan = rt.Q8Plan(1, 16, 1, False, 0, 0, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        rt.decode_q8(plan, *q, cache, tab, ctx, 0.1, torch.zeros(1, 1, 16, 512))
