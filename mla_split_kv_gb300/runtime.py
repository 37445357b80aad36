"""Device buffers and one decode layer call through the C ABI.

torch supplies device memory and streams; the binding passes raw pointers;
all computation happens in the CUDA library.
"""
from __future__ import annotations

import dataclasses
import heapq
from typing import Optional, Sequence

import numpy as np
import torch

from . import binding as nb
from .inputs import DecodeCase

TORCH_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def to_device_16(bits: np.ndarray, dtype: str, device) -> torch.Tensor:
    """uint16 bit patterns -> a 16-bit float tensor on `device` (bit-exact)."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(TORCH_DTYPE[dtype])


@dataclasses.dataclass
class DeviceCase:
    q_abs: torch.Tensor
    q_pe: torch.Tensor
    ckv: torch.Tensor
    kpe: torch.Tensor
    block_table: torch.Tensor
    context_lens: torch.Tensor
    case: DecodeCase


def to_device_cache(bits: np.ndarray, dtype: str, device) -> torch.Tensor:
    """Cache patterns -> device: 16-bit floats (bit-exact), or E4M3 bytes as uint8."""
    if dtype == "e4m3":
        return torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint8)).to(device)
    return to_device_16(bits, dtype, device)


def query_dtype(dtype: str) -> str:
    """The queries' 16-bit type beside a cache of `dtype`: fp16 beside E4M3."""
    return "f16" if dtype == "e4m3" else dtype


def upload(case: DecodeCase, device="cuda", ckv: torch.Tensor = None, kpe: torch.Tensor = None) -> DeviceCase:
    """Copy a case to the device. A resident cache (ckv/kpe) can be shared."""
    qdt = query_dtype(case.dtype)
    return DeviceCase(
        q_abs=to_device_16(case.q_abs, qdt, device),
        q_pe=to_device_16(case.q_pe, qdt, device),
        ckv=ckv if ckv is not None else to_device_cache(case.ckv, case.dtype, device),
        kpe=kpe if kpe is not None else to_device_cache(case.kpe, case.dtype, device),
        block_table=torch.from_numpy(np.ascontiguousarray(case.block_table)).to(device),
        context_lens=torch.from_numpy(np.ascontiguousarray(case.context_lens)).to(device),
        case=case,
    )


def chunks_to_device(chunks: Sequence[Sequence[int]], device="cuda") -> torch.Tensor:
    arr = np.asarray(chunks, dtype=np.int32).reshape(-1, 4)
    return torch.from_numpy(arr).to(device)


def make_desc(dc: DeviceCase, chunks_dev: Optional[torch.Tensor], kernel: int, cluster: int,
              stream: Optional[torch.cuda.Stream] = None, subs: int = 1,
              workspace: Optional[torch.Tensor] = None, tables_ready: bool = False,
              decode_merge: int = 0, prefix_ready: bool = False,
              score_exchange: int = 0) -> nb.mla_decode_desc_t:
    c = dc.case
    d = nb.mla_decode_desc_t()
    d.num_requests = c.num_requests
    d.num_heads = c.num_heads
    d.q_len = c.q_len
    d.block_size = c.block_size
    d.num_blocks = int(dc.ckv.shape[0])
    d.max_blocks_per_req = int(dc.block_table.shape[1])
    d.dtype = nb.DTYPE_CODES[c.dtype]
    d.causal = 1 if c.causal else 0
    d.chunks = chunks_dev.data_ptr() if chunks_dev is not None else None
    d.num_chunks = int(chunks_dev.shape[0]) if chunks_dev is not None else 0
    d.cluster_ctas = cluster
    d.kernel = kernel
    s = stream if stream is not None else torch.cuda.current_stream()
    d.stream = s.cuda_stream
    d.clusters_per_chunk = subs
    d.workspace = workspace.data_ptr() if workspace is not None else None
    d.workspace_bytes = workspace.numel() if workspace is not None else 0
    d.tables_ready = 1 if tables_ready else 0
    d.decode_merge = decode_merge
    d.prefix_ready = 1 if prefix_ready else 0
    d.cache_scale = float(c.cache_scale)
    d.score_exchange = score_exchange
    # the descriptor holds raw device pointers: keep their tensors alive as long as it lives
    d._keep = (chunks_dev, workspace)
    return d


def alloc_workspace(num_chunks: int, subs: int, cluster: int, q_len: int, H: int,
                    device="cuda") -> Optional[torch.Tensor]:
    """Zeroed workspace for partitions spread over `subs` clusters of `cluster` CTAs (None when subs <= 1)."""
    n = nb.mla_workspace_bytes(num_chunks, subs, cluster, q_len, H)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def alloc_decode_workspace(B: int, num_chunks: int, subs: int, cluster: int, q_len: int, H: int,
                           device="cuda") -> torch.Tensor:
    """Zeroed workspace of mla_decode on the paired kernel (request tickets and LSE copies of its single-launch
    way, then the chunk tickets and the pair entries)."""
    n = nb.mla_decode_workspace_bytes(B, num_chunks, subs, cluster, q_len, H)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode(dc: DeviceCase, part: torch.Tensor, lse: torch.Tensor, o_indptr_dev: torch.Tensor, out: torch.Tensor,
           out_lse: Optional[torch.Tensor] = None, num_partitions: int = 1, desc: Optional[nb.mla_decode_desc_t] = None,
           **desc_kw) -> torch.Tensor:
    """One decode layer call through mla_decode (its ways on the paired kernel chosen by decode_merge)."""
    d = desc if desc is not None else make_desc(dc, desc_kw.get("chunks_dev"), desc_kw.get("kernel", nb.MLA_KERNEL_AUTO),
                                                desc_kw.get("cluster", 0), desc_kw.get("stream"),
                                                desc_kw.get("subs", 1), desc_kw.get("workspace"),
                                                desc_kw.get("tables_ready", False), desc_kw.get("decode_merge", 0),
                                                desc_kw.get("prefix_ready", False),
                                                desc_kw.get("score_exchange", 0))
    out_code = {torch.float32: nb.MLA_F32, torch.float16: nb.MLA_F16, torch.bfloat16: nb.MLA_BF16}[out.dtype]
    nb.mla_decode(dc.q_abs.data_ptr(), dc.q_pe.data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                  dc.block_table.data_ptr(), dc.context_lens.data_ptr(), float(dc.case.scale), num_partitions,
                  part.data_ptr(), lse.data_ptr(), o_indptr_dev.data_ptr(), out.data_ptr(), out_code,
                  out_lse.data_ptr() if out_lse is not None else None, d)
    return out


def decode_unembed(dc: DeviceCase, part: torch.Tensor, lse: torch.Tensor, o_indptr_dev: torch.Tensor,
                   w_uv_t: torch.Tensor, out_v: torch.Tensor, out_lse: Optional[torch.Tensor] = None,
                   num_partitions: int = 1, desc: Optional[nb.mla_decode_desc_t] = None, **desc_kw) -> torch.Tensor:
    """One decode layer call through mla_decode_unembed: attention, then W_UV^T [H, 512, v_head] per head."""
    d = desc if desc is not None else make_desc(dc, desc_kw.get("chunks_dev"), desc_kw.get("kernel", nb.MLA_KERNEL_AUTO),
                                                desc_kw.get("cluster", 0), desc_kw.get("stream"),
                                                desc_kw.get("subs", 1), desc_kw.get("workspace"),
                                                desc_kw.get("tables_ready", False), desc_kw.get("decode_merge", 0),
                                                desc_kw.get("prefix_ready", False),
                                                desc_kw.get("score_exchange", 0))
    codes = {torch.float32: nb.MLA_F32, torch.float16: nb.MLA_F16, torch.bfloat16: nb.MLA_BF16}
    nb.mla_decode_unembed(dc.q_abs.data_ptr(), dc.q_pe.data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                          dc.block_table.data_ptr(), dc.context_lens.data_ptr(), float(dc.case.scale), num_partitions,
                          part.data_ptr(), lse.data_ptr(), o_indptr_dev.data_ptr(), w_uv_t.data_ptr(),
                          codes[w_uv_t.dtype], int(w_uv_t.shape[-1]), out_v.data_ptr(), codes[out_v.dtype],
                          out_lse.data_ptr() if out_lse is not None else None, d)
    return out_v


def alloc_partials(num_slots: int, q_len: int, H: int, device="cuda"):
    part = torch.empty((num_slots, q_len, H, 512), dtype=torch.float32, device=device)
    lse = torch.empty((num_slots, q_len, H), dtype=torch.float32, device=device)
    return part, lse


def decode_partial(dc: DeviceCase, part: torch.Tensor, lse: torch.Tensor, num_partitions: int = 1,
                   chunks_dev: Optional[torch.Tensor] = None, kernel: int = nb.MLA_KERNEL_AUTO,
                   cluster: int = 0, stream=None, desc: Optional[nb.mla_decode_desc_t] = None, subs: int = 1,
                   workspace: Optional[torch.Tensor] = None, tables_ready: bool = False,
                   score_exchange: int = 0) -> None:
    d = desc if desc is not None else make_desc(dc, chunks_dev, kernel, cluster, stream, subs, workspace,
                                                tables_ready, score_exchange=score_exchange)
    nb.mla_decode_partial(dc.q_abs.data_ptr(), dc.q_pe.data_ptr(), dc.ckv.data_ptr(), dc.kpe.data_ptr(),
                          dc.block_table.data_ptr(), dc.context_lens.data_ptr(), float(dc.case.scale),
                          num_partitions, part.data_ptr(), lse.data_ptr(), d)


def merge_states(part: torch.Tensor, lse: torch.Tensor, o_indptr_dev: torch.Tensor, B: int, q_len: int, H: int,
                 out_dtype: str = "f32", out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                 stream=None):
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[out_dtype]
    if out is None:
        out = torch.empty((B, q_len, H, 512), dtype=tdt, device=part.device)
    s = stream if stream is not None else torch.cuda.current_stream()
    nb.mla_merge_states(part.data_ptr(), lse.data_ptr(), o_indptr_dev.data_ptr(), B, q_len, H, out.data_ptr(),
                        nb.DTYPE_CODES[out_dtype], out_lse.data_ptr() if out_lse is not None else None,
                        s.cuda_stream)
    return out


def uniform_indptr(B: int, P: int, device="cuda") -> torch.Tensor:
    return torch.arange(0, (B + 1) * P, P, dtype=torch.int32, device=device)


@dataclasses.dataclass
class SegmentPlan:
    """Partitions of a verify window over a segmented prefix: each segment planned on its own,
    chunk slots request-major over all segments, so one merge of o_indptr combines them."""
    chunk_tables: list       # per segment, device int32 [n, 4] {b, t0, t1, slot}
    plans: list              # per segment, the planner's Plan
    o_indptr: torch.Tensor   # device [B+1]
    num_slots: int


def plan_segments(seg, dev: nb.mla_device_info_t, max_partitions: int = 0, device="cuda") -> SegmentPlan:
    segs = seg.segments
    B = segs[0].num_requests
    plans = [nb.mla_plan(s.context_lens.tolist(), s.num_heads, s.q_len, s.block_size, dev,
                         max_partitions=max_partitions, dtype=s.dtype) for s in segs]
    # request b's slots: its chunks of segment 0, then of segment 1, ...
    per = [[p.o_indptr[b + 1] - p.o_indptr[b] for b in range(B)] for p in plans]
    indptr = [0]
    for b in range(B):
        indptr.append(indptr[-1] + sum(per[k][b] for k in range(len(segs))))
    tables = []
    for k, p in enumerate(plans):
        rows = []
        for b in range(B):
            base = indptr[b] + sum(per[j][b] for j in range(k))
            for i, (cb, t0, t1, _) in enumerate(p.chunks[p.o_indptr[b]:p.o_indptr[b + 1]]):
                rows.append((cb, t0, t1, base + i))
        tables.append(chunks_to_device(rows, device))
    return SegmentPlan(chunk_tables=tables, plans=plans,
                       o_indptr=torch.tensor(indptr, dtype=torch.int32, device=device), num_slots=indptr[-1])


# ---------------------------------------------------------------------------
# sliding windows
# ---------------------------------------------------------------------------


@dataclasses.dataclass
class WindowPlan:
    """A plan of mla_decode_window for one batch shape, with the buffers its calls use. It serves contexts of any
    length, in the time planned for visible runs no longer than it was made for: each request's last partition takes
    what its run has beyond that. Calls that may overlap in time (other streams) need a plan each."""
    num_requests: int
    num_heads: int
    q_len: int
    block_size: int
    dtype: str
    causal: bool
    window: int
    sinks: int
    plan: nb.Plan
    chunks: torch.Tensor
    o_indptr: torch.Tensor
    partials: torch.Tensor
    lse: torch.Tensor
    workspace: torch.Tensor


# What a partition costs a CTA pair beside its tokens, in tokens: 5 to 8 us of start and end, at the 64-token tile's
# 2.6 us of more than 16 rows and the 128-token tile's 1.75 of 16.
_PART_TOKENS = 250


def _window_partitions(runs: Sequence[int], num_heads: int, q_len: int, block_size: int, dtype: str,
                       dev: nb.mla_device_info_t) -> nb.Plan:
    """A plan of visible runs. mla_plan's own thresholds leave runs below 4096 tokens whole, as long as most windows
    are: the longest partition then sets the time (16 runs of 2048 tokens, 64 rows: 100 us whole, 35 us over all CTA
    pairs). And it fills the device with CTAs rather than with requests: batches of short runs go through large
    clusters in several waves. So plans with more and smaller partitions, none below the 128 tokens that a CTA pair
    needs, and with one cluster size at a time are laid out beside its own, and the one whose busiest pair is done
    first is taken."""
    rows = num_heads * q_len
    groups = -(-rows // 128)

    def busiest_pair(plan: nb.Plan) -> int:
        pairs = plan.clusters_per_chunk * (plan.cluster_ctas // 2)
        servers = max(1, dev.max_clusters[plan.cluster_ctas.bit_length() - 1] // (groups * plan.clusters_per_chunk))
        ends = [0] * min(servers, plan.num_chunks)
        for _, t0, t1, _ in plan.chunks:  # in launch order, each to the pairs that are free first
            heapq.heapreplace(ends, ends[0] + _PART_TOKENS + -(-(t1 - t0) // pairs))
        parts = max(plan.o_indptr[b + 1] - plan.o_indptr[b] for b in range(len(runs)))
        return max(ends) + 2 * parts  # the merge reads a part in about the time of two tokens

    def only(size: int, clusters: int) -> nb.mla_device_info_t:
        d = nb.mla_device_info_t()
        d.num_sms = dev.num_sms
        d.max_clusters[size] = min(dev.max_clusters[size], clusters)
        return d

    best = nb.mla_plan(runs, num_heads, q_len, block_size, dev, dtype=dtype)
    cost = busiest_pair(best) if best.cluster_ctas > 1 else None
    tries = [(dev, n, 128 * n) for n in (2, 4, 8, 16, 32, 64)] + [(dev, 8, 256), (dev, 64, 256)]
    # partitions of about so many tokens, whatever their request's length
    tries += [(only(1, max(len(runs), sum(runs) // tokens) * groups), 64, 256) for tokens in (160, 256, 384)]
    if rows <= 16:
        tries += [(only(size, 1 << 30), 1, 0) for size in (1, 2, 3, 4)]
    for where, most, split_min in tries:
        if not any(where.max_clusters):
            continue
        plan = nb.mla_plan(runs, num_heads, q_len, block_size, where, max_partitions=most, min_partitions=1,
                           split_min_tokens=split_min, dtype=dtype)
        if plan.cluster_ctas > 1 and (cost is None or busiest_pair(plan) < cost):
            best, cost = plan, busiest_pair(plan)
    return best


def _open_ended(plan: nb.Plan) -> list:
    """The plan's chunks, each request's last one up to the end of its run however long that is (the kernels clip)."""
    last = set(plan.o_indptr[1:])
    return [(b, t0, 2 ** 31 - 1 if slot + 1 in last else t1, slot) for b, t0, t1, slot in plan.chunks]


def plan_window(context_lens: Sequence[int], num_heads: int, q_len: int, block_size: int, window: int, sinks: int = 0,
                dtype: str = "f16", causal: bool = False, dev: Optional[nb.mla_device_info_t] = None,
                max_partitions: int = 0, device="cuda", grow: int = 0) -> WindowPlan:
    """Partitions of the requests' visible runs: at most max_partitions each by mla_plan's thresholds, or (0) as many
    as fill the device. `grow`: tokens by which each context may grow while the plan is used (a run's length goes up
    and down by a page with its context's place in the page, so a plan made for one length may be a page short at the
    next, which its last partition then has to take)."""
    if grow < 0:
        raise ValueError(f"grow: {grow}")
    runs = nb.mla_window_lens(context_lens, q_len, block_size, causal, window, sinks)
    for back in range(min(grow, block_size)):  # the longest run on the way is within a page of its end
        lens = [min(int(n) + grow - back, 2 ** 31 - 1) for n in context_lens]
        runs = [max(a, b) for a, b in zip(runs, nb.mla_window_lens(lens, q_len, block_size, causal, window, sinks))]
    index = torch.device(device).index
    dev = dev if dev is not None else nb.mla_device_query(-1 if index is None else index)
    if max_partitions:
        plan = nb.mla_plan(runs, num_heads, q_len, block_size, dev, max_partitions=max_partitions, dtype=dtype)
        while plan.cluster_ctas < 2 and max_partitions > 1:
            # so many that a CTA pair's share of one would be under 128 tokens: planned for single CTAs, which a
            # windowed call does not run on
            max_partitions //= 2
            plan = nb.mla_plan(runs, num_heads, q_len, block_size, dev, max_partitions=max_partitions, dtype=dtype)
    else:
        plan = _window_partitions(runs, num_heads, q_len, block_size, dtype, dev)
    part, lse = alloc_partials(plan.num_chunks, q_len, num_heads, device)
    return WindowPlan(len(runs), num_heads, q_len, block_size, dtype, causal, window, sinks, plan,
                      chunks_to_device(_open_ended(plan), device),
                      torch.tensor(plan.o_indptr, dtype=torch.int32, device=device), part, lse,
                      alloc_decode_workspace(len(runs), plan.num_chunks, plan.clusters_per_chunk, plan.cluster_ctas,
                                             q_len, num_heads, device))


def decode_window(plan: WindowPlan, q_abs: torch.Tensor, q_pe: torch.Tensor, ckv: torch.Tensor, kpe: torch.Tensor,
                  block_table: torch.Tensor, context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                  out_lse: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                  cache_scale: float = 1.0) -> torch.Tensor:
    """One decode layer call through a sliding window (mla_decode_window), into out [B, q_len, H, 512]."""
    B, q_len, H, bs = plan.num_requests, plan.q_len, plan.num_heads, plan.block_size
    cache_dtype = torch.uint8 if plan.dtype == "e4m3" else TORCH_DTYPE[plan.dtype]
    q_dtype = TORCH_DTYPE[query_dtype(plan.dtype)]
    dev = _device_of(plan.workspace)
    nblk, width = ckv.shape[0], block_table.shape[-1]
    _expect(q_abs, (B, q_len, H, 512), q_dtype, "q_abs", dev)
    _expect(q_pe, (B, q_len, H, 64), q_dtype, "q_pe", dev)
    _expect(ckv, (nblk, bs, 512), cache_dtype, "ckv", dev)
    _expect(kpe, (nblk, bs, 64), cache_dtype, "kpe", dev)
    _expect(out, (B, q_len, H, 512), out.dtype, "out", dev)
    if out_lse is not None:
        _expect(out_lse, (B, q_len, H), torch.float32, "out_lse", dev)
    _expect(context_lens, (B,), torch.int32, "context_lens", dev)
    _expect(block_table, (B, width), torch.int32, "block_table", dev)
    raw_stream = stream.cuda_stream if stream is not None else _current_stream(dev)
    p = plan.plan
    d = nb.mla_decode_desc_t(B, H, q_len, bs, nblk, width, nb.DTYPE_CODES[plan.dtype],
                             1 if plan.causal else 0, plan.chunks.data_ptr(), p.num_chunks, p.cluster_ctas,
                             nb.MLA_KERNEL_TC, raw_stream, p.clusters_per_chunk, plan.workspace.data_ptr(),
                             plan.workspace.numel(), 0, 0, 0, cache_scale, 0)
    nb.mla_decode_window(q_abs.data_ptr(), q_pe.data_ptr(), ckv.data_ptr(), kpe.data_ptr(), block_table.data_ptr(),
                         context_lens.data_ptr(), scale, 0, plan.partials.data_ptr(), plan.lse.data_ptr(),
                         plan.o_indptr.data_ptr(), out.data_ptr(), _code_of(out, "out"),
                         out_lse.data_ptr() if out_lse is not None else None, plan.window, plan.sinks, d)
    return out


# ---------------------------------------------------------------------------
# block-scaled 8-bit caches
# ---------------------------------------------------------------------------

CODE_OF = {torch.float16: nb.MLA_F16, torch.bfloat16: nb.MLA_BF16, torch.float32: nb.MLA_F32}


@dataclasses.dataclass
class Q8Cache:
    """A paged latent cache in E4M3 bytes with an fp32 scale for every `scale_block` tokens of a page."""
    ckv: torch.Tensor     # uint8 [num_blocks, bs, 512]
    kpe: torch.Tensor     # uint8 [num_blocks, bs, 64]
    scales: torch.Tensor  # float32 [num_blocks, bs / scale_block]

    def __post_init__(self):
        nblk, bs = int(self.ckv.shape[0]), int(self.ckv.shape[1])
        dev = self.ckv.get_device()
        _expect(self.ckv, (nblk, bs, 512), torch.uint8, "ckv", dev)
        _expect(self.kpe, (nblk, bs, 64), torch.uint8, "kpe", dev)
        if self.scales.dim() != 2 or self.scales.shape[1] < 1 or bs % int(self.scales.shape[1]):
            raise ValueError(f"scales: {tuple(self.scales.shape)} does not divide pages of {bs} tokens")
        _expect(self.scales, (nblk, int(self.scales.shape[1])), torch.float32, "scales", dev)
        self.num_blocks, self.block_size = nblk, bs
        self.scale_block = bs // int(self.scales.shape[1])


def _device_of(t: torch.Tensor) -> int:
    """The library launches on the current device: a buffer that is elsewhere is refused here."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"a buffer on {t.device}: the call runs on the current CUDA device")
    return dev


# the current stream's handle without a Stream object around it (1 us of a call that takes 4 on the GPU)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _expect(t: torch.Tensor, shape, dtype, what: str, dev: int) -> None:
    """The C ABI takes raw pointers to dense row-major buffers of one device: anything else is refused here."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {shape} beside the call's other "
                         f"buffers, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _code_of(t: torch.Tensor, what: str) -> int:
    code = CODE_OF.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: {t.dtype} is none of {', '.join(str(k) for k in CODE_OF)}")
    return code


def alloc_q8_cache(num_blocks: int, block_size: int, scale_block: int, device="cuda") -> Q8Cache:
    """An empty pool (every byte 0, every scale 1)."""
    if scale_block < 1 or block_size % scale_block:
        raise ValueError(f"scale_block: {scale_block} does not divide pages of {block_size} tokens")
    return Q8Cache(torch.zeros((num_blocks, block_size, 512), dtype=torch.uint8, device=device),
                   torch.zeros((num_blocks, block_size, 64), dtype=torch.uint8, device=device),
                   torch.ones((num_blocks, block_size // scale_block), dtype=torch.float32, device=device))


def cache_append_q8(cache: Q8Cache, ckv_new: torch.Tensor, kpe_new: torch.Tensor, block_table: torch.Tensor,
                    context_lens: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantize each request's newest tokens [B, q_len, 512 / 64] into the cache (mla_cache_append_q8)."""
    dev = _device_of(cache.ckv)
    B, q_len = ckv_new.shape[0], ckv_new.shape[1]
    width = block_table.shape[-1]
    _expect(ckv_new, (B, q_len, 512), ckv_new.dtype, "ckv_new", dev)
    _expect(kpe_new, (B, q_len, 64), ckv_new.dtype, "kpe_new", dev)
    _expect(context_lens, (B,), torch.int32, "context_lens", dev)
    _expect(block_table, (B, width), torch.int32, "block_table", dev)
    raw_stream = stream.cuda_stream if stream is not None else _current_stream(dev)
    nb.mla_cache_append_q8(ckv_new.data_ptr(), kpe_new.data_ptr(), _code_of(ckv_new, "ckv_new"),
                           block_table.data_ptr(), context_lens.data_ptr(), B, q_len, cache.block_size,
                           cache.scale_block, cache.num_blocks, width, cache.ckv.data_ptr(), cache.kpe.data_ptr(),
                           cache.scales.data_ptr(), raw_stream)


@dataclasses.dataclass
class Q8Plan:
    """What calls of one shape keep between them: the descriptor's options and the workspace. Calls that may
    overlap in time (other streams) need a plan each."""
    num_requests: int
    num_heads: int
    q_len: int
    causal: bool
    window: int
    sinks: int
    workspace: torch.Tensor


def plan_q8(num_requests: int, num_heads: int, q_len: int = 1, causal: bool = False, window: int = 0, sinks: int = 0,
            device="cuda") -> Q8Plan:
    """The options and the workspace of decode_q8 calls of one shape: the first `num_requests` lengths and table rows
    count, each request's q_len rows see its tokens up to their own (causal) or all of them, and with window >= 1 only
    the last `window` of those and the request's first `sinks`. Lengths are not part of it."""
    index = torch.device(device).index
    n = nb.mla_decode_q8_workspace_bytes(nb.mla_device_query(-1 if index is None else index), q_len, num_heads)
    if n == 0:
        raise nb.MlaError(nb.MLA_ERR_UNSUPPORTED, "mla_decode_q8_workspace_bytes")
    return Q8Plan(num_requests, num_heads, q_len, causal, window, sinks,
                  torch.empty(n, dtype=torch.uint8, device=device))


def decode_q8(plan: Q8Plan, q_abs: torch.Tensor, q_pe: torch.Tensor, cache: Q8Cache, block_table: torch.Tensor,
              context_lens: torch.Tensor, scale: float, out: torch.Tensor, out_lse: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode layer call over a block-scaled 8-bit cache (mla_decode_q8), into out [B, q_len, H, 512]."""
    B, q_len, H = plan.num_requests, plan.q_len, plan.num_heads
    dev = _device_of(plan.workspace)
    width = block_table.shape[-1]
    _expect(q_abs, (B, q_len, H, 512), q_abs.dtype, "q_abs", dev)
    _expect(q_pe, (B, q_len, H, 64), q_abs.dtype, "q_pe", dev)
    _expect(out, (B, q_len, H, 512), out.dtype, "out", dev)
    if out_lse is not None:
        _expect(out_lse, (B, q_len, H), torch.float32, "out_lse", dev)
    _expect(context_lens, (B,), torch.int32, "context_lens", dev)
    _expect(block_table, (B, width), torch.int32, "block_table", dev)
    if cache.ckv.get_device() != dev:
        raise ValueError(f"cache: on {cache.ckv.device}, the plan's workspace on {plan.workspace.device}")
    raw_stream = stream.cuda_stream if stream is not None else _current_stream(dev)
    d = nb.mla_q8_desc_t(B, H, q_len, cache.block_size, cache.num_blocks, width, _code_of(q_abs, "q_abs"),
                         1 if plan.causal else 0, cache.scale_block, plan.window, plan.sinks, _code_of(out, "out"),
                         plan.workspace.data_ptr(), plan.workspace.numel(), raw_stream)
    nb.mla_decode_q8(q_abs.data_ptr(), q_pe.data_ptr(), cache.ckv.data_ptr(), cache.kpe.data_ptr(),
                     cache.scales.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), scale,
                     out.data_ptr(), out_lse.data_ptr() if out_lse is not None else None, d)
    return out
