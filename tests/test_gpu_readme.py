"""The steps that the documentation shows, run as they stand there, step after step."""
import os
import re

import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from tests.test_gpu_expand import Case as ExpandCase
from tests.test_gpu_prefill import Case as PromptCase
from tests.test_gpu_shared import Case as SharedCase
from tests.test_gpu_step import HostStep

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


def blocks():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        section = f.read().split("### Prompts, steps and common prefixes", 1)[1]
    return re.findall(r"```python\n(.*?)```", section, re.S)


def test_a_loop_of_steps_gives_no_page_out_twice():
    setup, one_step, shared_step = blocks()
    g = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    B, H, bs, num_blocks, width = 4, 16, 32, 60, 16
    env = dict(rt=rt, B=B, num_heads=H, num_blocks=num_blocks, capacity=512, max_tokens=512, scale=192.0 ** -0.5)
    exec(setup, env)
    host = HostStep([0] * B, bs, num_blocks, width, np.random.default_rng(0))
    host.free = env["pool"].pages.tolist()
    assert host.free == list(range(num_blocks - 1, -1, -1))
    env["block_table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    env["ckv"], env["kpe"] = rand(num_blocks, bs, 512), rand(num_blocks, bs, 64)
    env["w_uk"], env["w_uv_t"] = rand(H, 128, 512) / 16, rand(H, 512, 128) / 16
    history = [torch.empty(0, 576, dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    for changes in ([100, 40, 1, 0], [1, 33, 200, 7], [1, -50, 1, 90], [64, 1, -202, 1]):
        want = host.step(changes, 512)
        grown, S = [max(n, 0) for n in changes], sum(host.lens)
        T = sum(grown)
        new, q = rand(T, 576), rand(T, H, 192)
        env.update(changes=torch.tensor(changes, dtype=torch.int32, device="cuda"), ckv_new=new[:, :512], kpe_new=new[:, 512:],
                   k_nope=torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda"), v=torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda"),
                   k_pe=torch.empty(S, 64, dtype=torch.bfloat16, device="cuda"), q_nope=q[..., :128], q_pe=q[..., 128:],
                   out=torch.full((T, H, 128), 77.0, dtype=torch.bfloat16, device="cuda"))
        exec(one_step, env)
        torch.cuda.synchronize()
        for b, (n, x) in enumerate(zip(changes, new.split(grown))):
            history[b] = torch.cat((history[b], x)) if n >= 0 else history[b][:n]
        step = env["step"]
        for name, value in want.items():
            assert getattr(step, name).tolist() == [int(x) for x in value], name
        assert env["pool"].count.item() == len(host.free) and env["pool"].pages[:len(host.free)].tolist() == host.free
        for b, x in enumerate(history):
            t = torch.arange(len(x), device="cuda")
            rows = env["block_table"][b].long()[t // bs] * bs + t % bs
            assert torch.equal(env["ckv"].view(-1, 512)[rows], x[:, :512]) and torch.equal(env["kpe"].view(-1, 64)[rows], x[:, 512:])
        e = ExpandCase.__new__(ExpandCase)
        e.lens, e.bs, e.dtype, e.table, e.indptr = host.lens, bs, torch.bfloat16, env["block_table"], step.kv_indptr
        e.ckv, e.kpe, e.w_uk, e.w_uv_t, e.k, e.v, e.k_pe = (env[x] for x in ("ckv", "kpe", "w_uk", "w_uv_t", "k_nope", "v", "k_pe"))
        e.check()
        p = PromptCase.__new__(PromptCase)
        p.new, p.ctx, p.H, p.dtype, p.causal, p.scale = grown, host.lens, H, torch.bfloat16, True, env["scale"]
        p.q_at, p.kv_at = step.q_indptr.tolist(), step.kv_indptr.tolist()
        p.k, p.v, p.k_pe, p.q_nope, p.q_pe = e.k, e.v, e.k_pe, env["q_nope"], env["q_pe"]
        lse = torch.full((T, H), 77.0, device="cuda")
        rt.prefill(env["prompts"], p.q_nope, p.q_pe, p.k, p.k_pe, p.v, step.q_indptr, step.kv_indptr, p.scale, torch.empty_like(env["out"]), lse)
        p.check(env["out"], lse, heads=[0, H - 1])

    # and a batch over a common prefix: the first request's first two pages
    P = 64
    env.update(context_lens_host=[165, 120, 64, 98], shared=P, q_abs=rand(B, 1, H, 512), q_pe=rand(B, 1, H, 64),
               out=torch.empty(B, 1, H, 512, device="cuda"), out_lse=torch.empty(B, 1, H, device="cuda"))
    step.context_lens.copy_(torch.tensor(env["context_lens_host"], dtype=torch.int32))
    env["block_table"].copy_(torch.arange(B * width, device="cuda").view(B, width) % num_blocks)
    exec(shared_step, env)
    torch.cuda.synchronize()
    c = SharedCase.__new__(SharedCase)
    c.lens, c.shared, c.H, c.q_len, c.bs, c.dtype, c.causal, c.scale = env["context_lens_host"], P, H, 1, bs, torch.bfloat16, False, env["scale"]
    c.shared_table, c.table, c.ckv, c.kpe, c.q_abs, c.q_pe = env["block_table"][0, :P // bs], env["block_table"], env["ckv"], env["kpe"], env["q_abs"], env["q_pe"]
    c.check(env["out"], env["out_lse"], heads=[0, H - 1])
