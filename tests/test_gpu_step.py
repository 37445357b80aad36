"""A step's tables and slots on the GPU against the same step done request by request on the host, and the write of
packed tokens through the slots."""
import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

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


def pages(n, bs):
    return -(-n // bs)


class HostStep:
    """The requests, their pages and the free ones as lists."""

    def __init__(self, lens, bs, num_blocks, width, rng):
        perm = [int(x) for x in rng.permutation(num_blocks)]
        self.bs, self.width, self.lens = bs, width, list(lens)
        self.rows = [[perm.pop() for _ in range(pages(n, bs))] for n in lens]
        self.free = perm

    def table(self):
        return np.array([(r + [-1] * self.width)[: self.width] for r in self.rows], np.int32)

    def step(self, changes, capacity):
        changes = [max(c, -n) for c, n in zip(changes, self.lens)]
        for b, c in enumerate(changes):
            if c < 0:
                keep = pages(self.lens[b] + c, self.bs)
                self.free += self.rows[b][keep:]
                self.rows[b] = self.rows[b][:keep]
                self.lens[b] += c
        slots, q, served = [], [0], None
        for b, c in enumerate(changes):
            if c > 0 and served is None:
                lack = pages(self.lens[b] + c, self.bs) - len(self.rows[b])
                if lack > len(self.free) or len(self.rows[b]) + lack > self.width or len(slots) + c > capacity:
                    served = b
                else:
                    self.rows[b] += [self.free.pop() for _ in range(lack)]
                    slots += [self.rows[b][t // self.bs] * self.bs + t % self.bs for t in range(self.lens[b], self.lens[b] + c)]
                    self.lens[b] += c
            q.append(len(slots))
        kv = np.concatenate(([0], np.cumsum(self.lens)))
        return dict(q_indptr=q, kv_indptr=kv, slots=slots + [-1] * (capacity - len(slots)), served=[len(self.lens) if served is None else served],
                    context_lens=self.lens, free_count=[len(self.free)])


class DeviceStep:
    def __init__(self, host, num_blocks, capacity, in_place):
        dev = lambda a, dt=np.int32: torch.from_numpy(np.array(a, dt)).cuda()  # noqa: E731
        stack = host.free + [-7] * (num_blocks - len(host.free))
        self.pool = rt.PagePool(dev(stack), dev([len(host.free)]), host.bs)
        self.lens, self.table = dev(host.lens), dev(host.table())
        self.out = rt.alloc_step(len(host.lens), capacity)
        self.in_place = in_place
        if in_place:
            self.out.context_lens, self.out.free_count = self.lens, self.pool.count

    def step(self, changes, **kw):
        rt.update_tables(self.pool, torch.tensor(changes, dtype=torch.int32, device="cuda"), self.lens, self.table, self.out, **kw)

    def take_over(self):
        if not self.in_place:
            self.lens.copy_(self.out.context_lens)
            self.pool.count.copy_(self.out.free_count)

    def check(self, host, want):
        for name, value in want.items():
            assert getattr(self.out, name).tolist() == [int(x) for x in value], name
        table = self.table.cpu().numpy()
        for b, row in enumerate(host.rows):
            assert table[b, : len(row)].tolist() == row, b
        assert self.pool.pages[: len(host.free)].tolist() == host.free


def draw_changes(rng, lens, most, back):
    return [int(-rng.integers(0, n + 1)) if rng.random() < back else int(rng.integers(0, most + 1)) for n in lens]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,most,back,capacity", [(1, 16, 1, 0.0, 1), (1, 64, 700, 0.0, 8192), (7, 32, 40, 0.4, 300), (33, 16, 100, 0.5, 20000),
                                                     (300, 64, 1, 0.2, 400), (1500, 32, 20, 0.3, 40000), (8192, 16, 5, 0.5, 9000)])
def test_steps_like_on_the_host(B, bs, most, back, capacity, in_place):
    rng = np.random.default_rng(B * 7 + bs + most)
    lens = rng.integers(0, 300, size=B).tolist()
    nblk, width = 2 * sum(pages(n, bs) for n in lens) + 3 * B, 64
    host = HostStep(lens, bs, nblk, width, rng)
    dev = DeviceStep(host, nblk, capacity, in_place)
    for _ in range(4):
        changes = draw_changes(rng, host.lens, most, back)
        want = host.step(changes, capacity)
        dev.step(changes)
        torch.cuda.synchronize()
        dev.check(host, want)
        dev.take_over()


@pytest.mark.parametrize("why", ["pages", "width", "slots"])
def test_requests_behind_one_that_does_not_fit_stay(why):
    rng = np.random.default_rng(5)
    lens, bs = [30, 0, 64, 17, 100, 3], 16
    nblk, width, capacity = {"pages": (22, 20, 500), "width": (60, 9, 500), "slots": (60, 20, 90)}[why]
    host = HostStep(lens, bs, nblk, width, rng)
    dev = DeviceStep(host, nblk, capacity, False)
    changes = [20, 10, -40, 60, 60, 1]  # the shrinking one's pages count, whatever fails
    want = host.step(changes, capacity)
    dev.step(changes)
    torch.cuda.synchronize()
    dev.check(host, want)
    assert want["served"] == [{"pages": 4, "width": 4, "slots": 4}[why]] and want["q_indptr"][4:] == [90, 90, 90]


@pytest.mark.parametrize("why", ["pages", "width"])
def test_many_places_and_requests_that_do_not_fit(why):
    """More places than one CTA fills: the slots come from a kernel of their own, which must not see what did not fit."""
    rng = np.random.default_rng(6)
    lens, bs, capacity = [30, 0, 6400, 17, 1000, 3, 5000, 0], 16, 30000
    nblk, width = {"pages": (1200, 3000), "width": (6000, 700)}[why]
    host = HostStep(lens, bs, nblk, width, rng)
    dev = DeviceStep(host, nblk, capacity, True)
    for changes in ([9000, 1, -6000, 4000, 0, 900, -1, 0], [1, 0, 1, 1, 1, 1, 1, 5000], [-9030, 3, 3000, 16, -1000, 1, 2, 15000]):
        want = host.step(changes, capacity)
        dev.step(changes)
        torch.cuda.synchronize()
        dev.check(host, want)


def test_pages_given_back_are_taken_in_the_same_step():
    rng = np.random.default_rng(6)
    host = HostStep([160, 0, 160, 5], 16, 21, 30, rng)
    assert len(host.free) == 0
    dev = DeviceStep(host, 21, 400, True)
    changes = [-160, 150, -33, 40]
    want = host.step(changes, 400)
    dev.step(changes)
    torch.cuda.synchronize()
    dev.check(host, want)
    assert want["served"] == [4]


def test_more_given_back_than_there_is():
    rng = np.random.default_rng(7)
    host = HostStep([40, 9], 16, 8, 8, rng)
    dev = DeviceStep(host, 8, 16, False)
    want = host.step([-1000, -9], 16)
    dev.step([-1000, -2 ** 31])
    torch.cuda.synchronize()
    dev.check(host, want)


def test_a_growth_past_the_longest_length_does_not_fit():
    rng = np.random.default_rng(8)
    host = HostStep([40, 9], 64, 8, 8, rng)
    dev = DeviceStep(host, 8, 16, False)
    dev.step([2 ** 31 - 1, 1])
    torch.cuda.synchronize()
    assert dev.out.served.item() == 0 and dev.out.context_lens.tolist() == [40, 9] and dev.out.slots.tolist() == [-1] * 16


def test_captured_steps_replay():
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 200, size=50).tolist()
    host = HostStep(lens, 32, 2000, 40, rng)
    dev = DeviceStep(host, 2000, 64, True)
    changes = torch.ones(50, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        rt.update_tables(dev.pool, changes, dev.lens, dev.table, dev.out)
    for k in range(40):
        want = host.step([1] * 50, 64)
        graph.replay()
        torch.cuda.synchronize()
        dev.check(host, want)


def test_a_page_outside_the_pool_gives_no_slot():
    rng = np.random.default_rng(10)
    host = HostStep([5, 20], 16, 10, 4, rng)
    dev = DeviceStep(host, 10, 8, False)
    dev.table[0, 0] = 10
    dev.step([2, 1])
    torch.cuda.synchronize()
    assert dev.out.slots.tolist()[:3] == [-1, -1, host.rows[1][1] * 16 + 4]
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,bs,joint", [(1, 16, False), (1, 32, True), (37, 64, True), (8193, 32, False), (9000, 16, True)])
def test_packed_tokens_land_in_their_slots(T, bs, joint, dtype):
    g = torch.Generator("cuda").manual_seed(T)
    nblk = pages(T, bs) + 7
    bits = lambda *shape: torch.randint(-2 ** 15, 2 ** 15, shape, dtype=torch.int16, device="cuda", generator=g)  # noqa: E731 (NaN patterns too)
    ckv, kpe = bits(nblk, bs, 512), bits(nblk, bs, 64)
    want_c, want_k = ckv.clone().view(-1, 512), kpe.clone().view(-1, 64)
    if joint:
        both = bits(T, 576 + 8)
        c, k = both[:, :512], both[:, 512:576]
    else:
        c, k = bits(T, 512), bits(T, 64)
    slots = torch.randperm(nblk * bs, device="cuda", generator=g)[:T]
    if T > 1:
        slots[::5] = -1
    real = slots >= 0
    want_c[slots[real]], want_k[slots[real]] = c[real], k[real]
    nb.mla_reset_counters()
    rt.cache_append_slots(ckv.view(dtype), kpe.view(dtype), c.view(dtype), k.view(dtype), slots)
    torch.cuda.synchronize()
    assert nb.mla_get_counters()[nb.CTR_STEP] == 1
    assert torch.equal(ckv.view(-1, 512), want_c) and torch.equal(kpe.view(-1, 64), want_k)


def test_a_slot_past_the_pool_is_not_written():
    ckv, kpe = torch.zeros(3, 16, 512, dtype=torch.float16, device="cuda"), torch.zeros(3, 16, 64, dtype=torch.float16, device="cuda")
    new = torch.ones(2, 576, dtype=torch.float16, device="cuda")
    rt.cache_append_slots(ckv, kpe, new[:, :512], new[:, 512:], torch.tensor([48, 47], device="cuda"))
    torch.cuda.synchronize()
    assert ckv.view(-1, 512).sum(1).tolist() == [0.0] * 47 + [512.0] and kpe.view(-1, 64).sum(1).tolist() == [0.0] * 47 + [64.0]
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_ERR_DEVICE_CHECK and code == 2


def test_a_step_writes_and_the_next_kernel_reads():
    """Tables, then the packed write through their slots, one behind the other on a stream of their own."""
    rng = np.random.default_rng(11)
    lens = [0, 45, 31, 200]
    host = HostStep(lens, 32, 60, 20, rng)
    dev = DeviceStep(host, 60, 600, True)
    want = host.step([300, 1, -5, 77], 600)
    T = 378
    new = torch.randn(T, 576, device="cuda").half()
    ckv, kpe = torch.zeros(60, 32, 512, dtype=torch.float16, device="cuda"), torch.zeros(60, 32, 64, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    changes = torch.tensor([300, 1, -5, 77], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    rt.update_tables(dev.pool, changes, dev.lens, dev.table, dev.out, stream=side)
    rt.cache_append_slots(ckv, kpe, new[:, :512], new[:, 512:], dev.out.slots, stream=side)
    side.synchronize()
    dev.check(host, want)
    at = torch.tensor(want["slots"][:T], device="cuda")
    assert torch.equal(ckv.view(-1, 512)[at], new[:, :512]) and torch.equal(kpe.view(-1, 64)[at], new[:, 512:])
    assert int((ckv.view(-1, 512) != 0).any(1).sum()) == T
