"""Requests from their prompts to their ends: tables, cache writes, prompts and decode steps over one pool of pages."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from tests.test_gpu_expand import Case as ExpandCase
from tests.test_gpu_prefill import Case as PromptCase
from tests.test_gpu_shared import Case as SharedCase

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


class Server:
    """A pool, its requests' tables and what each request's cache rows have to hold."""

    def __init__(self, seed, B, pages, width, H, bs, dtype, capacity):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.B, self.H, self.bs, self.dt, self.dtype = B, H, bs, dtype, TDT[dtype]
        self.pool = rt.alloc_pool(pages, bs)
        self.pool.pages[:] = self.pool.pages[torch.randperm(pages, device="cuda", generator=self.g)]
        self.step = rt.alloc_step(B, capacity)
        self.lens, self.table = self.step.context_lens, torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.step.free_count = self.pool.count  # the step's outputs are the next one's inputs
        self.changes = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ckv = torch.full((pages, bs, 512), float("nan"), dtype=self.dtype, device="cuda")
        self.kpe = torch.full((pages, bs, 64), float("nan"), dtype=self.dtype, device="cuda")
        self.w_uk, self.w_uv_t = self.rand(H, 128, 512) / 16, self.rand(H, 512, 128) / 16
        self.history = [self.rand(0, 576) for _ in range(B)]

    def rand(self, *s):
        return torch.randn(*s, device="cuda", generator=self.g).to(self.dtype)

    def tables(self, changes):
        self.changes.copy_(torch.tensor(changes, dtype=torch.int32))
        rt.update_tables(self.pool, self.changes, self.lens, self.table, self.step)

    def grow(self, changes, tokens=None):
        """`changes` new tokens a request, in the tables and the cache."""
        self.tables(changes)
        tokens = self.rand(sum(changes), 576) if tokens is None else tokens
        rt.cache_append_slots(self.ckv, self.kpe, tokens[:, :512], tokens[:, 512:], self.step.slots)
        self.note(changes, tokens)

    def note(self, changes, tokens):
        for b, x in enumerate(tokens.split(list(changes))):
            self.history[b] = torch.cat((self.history[b], x))

    def check_cache(self):
        assert self.lens.tolist() == [len(x) for x in self.history]
        for b, x in enumerate(self.history):
            t = torch.arange(len(x), device="cuda")
            rows = self.table[b].long()[t // self.bs] * self.bs + t % self.bs
            assert torch.equal(self.ckv.view(-1, 512)[rows], x[:, :512]) and torch.equal(self.kpe.view(-1, 64)[rows], x[:, 512:])

    def prompt(self, new):
        """The newest tokens' attention over everything their requests have, checked from the cache on."""
        ctx = [len(x) for x in self.history]
        e = ExpandCase.__new__(ExpandCase)
        e.lens, e.H, e.bs, e.dtype, e.table, e.indptr, e.ckv, e.kpe, e.w_uk, e.w_uv_t = (
            ctx, self.H, self.bs, self.dtype, self.table, self.step.kv_indptr, self.ckv, self.kpe, self.w_uk, self.w_uv_t)
        S, T = sum(ctx), sum(new)
        e.k, e.v, e.k_pe = (torch.full(s, float("nan"), dtype=self.dtype, device="cuda") for s in ((S, self.H, 128), (S, self.H, 128), (S, 64)))
        e.run()
        q = self.rand(T, self.H, 192)
        p = PromptCase.__new__(PromptCase)
        p.new, p.ctx, p.H, p.dtype, p.causal, p.scale, p.T, p.S = new, ctx, self.H, self.dtype, True, SCALE, T, S
        p.q_at, p.kv_at = ([sum(x[:b]) for b in range(len(new) + 1)] for x in (new, ctx))
        p.q_indptr, p.kv_indptr, p.q_nope, p.q_pe = self.step.q_indptr, self.step.kv_indptr, q[..., :128], q[..., 128:]
        p.k, p.v, p.k_pe, p.plan = e.k, e.v, e.k_pe, rt.plan_prefill(self.B, self.H, T)
        out, lse = p.run()
        torch.cuda.synchronize()
        assert p.q_at == self.step.q_indptr.tolist() and p.kv_at == self.step.kv_indptr.tolist()
        e.check()
        p.check(out, lse, heads=[0, self.H - 1])


@pytest.mark.parametrize("bs,H,dtype", [(16, 16, "bf16"), (32, 64, "f16"), (64, 16, "f16")])
def test_requests_from_prompt_to_end_over_a_common_prefix(bs, H, dtype):
    pages, P, B = 6 + 1600 // bs, 256, 5
    s = Server(bs + H, B, pages, 1024 // bs, H, bs, dtype, capacity=1024)
    s.grow([P, 0, 0, 0, 0])  # the document that all of them are about, in the first request's pages
    s.prompt([P, 0, 0, 0, 0])
    s.table[1:, :P // bs] = s.table[0, :P // bs]
    s.lens[1:] = P
    for b in range(1, B):
        s.history[b] = s.history[0]
    s.grow([70, 1, 0, 33, 300])  # the requests' own prompts
    s.check_cache()
    s.prompt([70, 1, 0, 33, 300])
    s.grow([1, 5, 64, 0, 7])  # one goes on, others' prompts come in pieces
    s.prompt([1, 5, 64, 0, 7])

    # decode steps, captured once: tables, cache, attention
    plan = rt.plan_shared(s.lens.tolist(), P, H, 1, bs, dtype=dtype)
    tokens, q_abs, q_pe = s.rand(B, 576), s.rand(B, 1, H, 512), s.rand(B, 1, H, 64)
    out, lse = torch.empty(B, 1, H, 512, device="cuda"), torch.empty(B, 1, H, device="cuda")
    s.changes.fill_(1)

    def decode():
        rt.update_tables(s.pool, s.changes, s.lens, s.table, s.step)
        rt.cache_append_slots(s.ckv, s.kpe, tokens[:, :512], tokens[:, 512:], s.step.slots)
        rt.decode_shared(plan, q_abs, q_pe, s.ckv, s.kpe, s.table, s.lens, SCALE, out, lse)

    decode()
    s.note([1] * B, tokens)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            decode()
    torch.cuda.current_stream().wait_stream(stream)

    def check():
        c = SharedCase.__new__(SharedCase)
        c.lens, c.shared, c.H, c.q_len, c.bs, c.dtype, c.causal, c.scale = [len(x) for x in s.history], P, H, 1, bs, s.dtype, False, SCALE
        c.shared_table, c.table, c.ckv, c.kpe, c.q_abs, c.q_pe = s.table[0, :P // bs], s.table, s.ckv, s.kpe, q_abs, q_pe
        c.check(out, lse, heads=[0, H - 1])

    torch.cuda.synchronize()
    check()
    for i in range(40):  # across the ends of pages
        tokens.copy_(s.rand(B, 576))
        graph.replay()
        s.note([1] * B, tokens)
        if i % 13 == 0:
            torch.cuda.synchronize()
            check()
    torch.cuda.synchronize()
    check()
    s.check_cache()
    assert s.step.served.item() == B

    # two end: what is their own goes back, then their share of the common pages is let go; others go on meanwhile
    held = [-(-len(x) // bs) for x in s.history]
    free = s.pool.count.item()
    ended = [P - len(s.history[1]), 0, P - len(s.history[4])]
    s.tables([0, ended[0], 2, 0, ended[2]])
    new = s.rand(2, 576)
    rt.cache_append_slots(s.ckv, s.kpe, new[:, :512], new[:, 512:], s.step.slots)
    s.history[1], s.history[4] = s.history[1][:P], s.history[4][:P]
    s.note([0, 0, 2, 0, 0], new)
    s.check_cache()
    s.lens[1], s.lens[4] = 0, 0
    s.history[1], s.history[4] = s.rand(0, 576), s.rand(0, 576)
    own = P // bs
    grown = -(-len(s.history[2]) // bs) - held[2]
    assert s.pool.count.item() == free + held[1] - own + held[4] - own - grown
    stack = s.pool.pages[:s.pool.count.item()].tolist()
    used = {p for b in (0, 2, 3) for p in s.table[b, :-(-len(s.history[b]) // bs)].tolist()}
    assert len(set(stack)) == len(stack) and not used & set(stack) and len(used) + len(stack) == pages
    s.grow([0, 90, 0, 0, 0])  # a new request in an old one's place
    s.prompt([0, 90, 0, 0, 0])


def test_a_plan_serves_fewer_requests_and_rows():
    big = PromptCase(3, [300] * 5, [700] * 5, 4, "bf16")
    small = PromptCase(4, [200, 90], [1500, 90], 4, "bf16", spare=5)
    small.plan = big.plan
    for case in (big, small, big):
        case.check(*case.run(), heads=[0, 3], requests=[0, 1])


def test_two_plans_on_two_streams_at_once():
    a, b = PromptCase(5, [700, 100], [3000, 100], 8, "bf16"), PromptCase(6, [90] * 30, [400] * 30, 8, "f16")
    c = SharedCase(7, [900 + 7 * i for i in range(12)], 512, 64, 1, 32, "bf16")
    d = SharedCase(8, [5000] * 3, 4096, 16, 2, 64, "f16", causal=True)
    plans = {c: c.plan(), d: d.plan()}
    run = lambda case: case.run(plans[case]) if case in plans else case.run()  # noqa: E731
    want = [run(x) for x in (a, b, c, d)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(5):
        for x, stream in zip((a, b, c, d), streams):
            with torch.cuda.stream(stream):
                got.append(run(x))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 4][0]) and torch.equal(lse, want[i % 4][1]), i


@pytest.mark.parametrize("call", ["expand", "prefill", "planned prefill"])
def test_waits_that_run_out_are_reported(call):
    case = ExpandCase(9, [3000], 16, 32, "bf16") if call == "expand" else PromptCase(9, [700], [700 if call == "prefill" else 9000], 8, "bf16")
    case.run()
    torch.cuda.synchronize()
    nb.mla_check_device_errors(None)
    nb.mla_set_wait_timeout_ns(1)
    try:
        for _ in range(50):  # (a wait is found too long when the device's timer has moved on and it still lasts)
            case.run()
            st, code = nb.mla_check_device_errors(None)
            if st != nb.MLA_OK:
                break
    finally:
        nb.mla_set_wait_timeout_ns(2_000_000_000)
    assert st == nb.MLA_ERR_TIMEOUT and code & 1, (st, code)
    got = case.run()  # the next call is whole again
    torch.cuda.synchronize()
    if call == "expand":
        case.check()
    else:
        case.check(*got, heads=[0, 7])
