// Attention over a block-scaled 8-bit cache, sm_103a.
//
// For each row of a request, over the tokens t that it sees,
//   s_t = scale * z_t * (q_abs . c_t + q_pe . k_t)
//   out = sum_t softmax(s)_t * z_t * c_t,   lse = log2 sum_t exp(s_t)
// with c_t, k_t the E4M3 values of the token's bytes and z_t its block's scale.
#include "q8_schedule.cuh"

namespace mla {

namespace {

constexpr int kNR = 16;       // query rows per CTA
constexpr int kThreads = 256;
constexpr int kStep = 16;     // tokens taken at a time
constexpr int kPad = kQkDim + 1;

struct Smem {
  float q[kNR][kPad];
  float kv[kStep][kPad];
  float prob[kNR][kStep];
  float alpha[kNR], m[kNR], l[kNR];
  int64_t scratch[33];
  int64_t off0;
  int b0;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) mla_decode_q8_kernel(const DecodeQ8Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x;
  const int group = blockIdx.x, gang = blockIdx.y;
  const int rows_total = p.q_len * p.H;
  const int row0 = group * kNR, nrows = min(kNR, rows_total - row0);
  pdl_wait();
  pdl_launch_dependents();
  // this gang's place on the line of tiles
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0, T = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += q8_tiles(p, b);
  const int64_t prefix = block_prefix<kThreads>(mine, sm.scratch, &T);
  const int64_t J = q8_live_gangs(T, p.gangs);
  const bool work = gang < J;
  const int64_t lo = work ? q8_gang_begin(gang, T, J) : 0, hi = work ? q8_gang_begin(gang + 1, T, J) : 0;
  if (work && lo >= prefix && lo < prefix + mine) {
    int64_t at = prefix;
    int b = b_lo;
    while (true) {
      const int64_t n = q8_tiles(p, b);
      if (at + n > lo) break;
      at += n;
      ++b;
    }
    sm.b0 = b;
    sm.off0 = lo - at;
  }
  // requests with nothing to see
  for (int b = gang; b < p.B; b += p.gangs) {
    if (q8_tiles(p, b) != 0) continue;
    for (int r = 0; r < nrows; ++r) {
      const long long at = static_cast<long long>(b) * rows_total + row0 + r;
      if (tid < kRank / 4) store_out4(p.out, p.out_dtype, at * kRank + 4 * tid, make_float4(0.f, 0.f, 0.f, 0.f));
      if (tid == 0 && p.out_lse != nullptr) p.out_lse[at] = -INFINITY;
    }
  }
  __syncthreads();
  if (!work) return;
  int b = sm.b0;
  int64_t ta = sm.off0;
  for (int64_t left = hi - lo; left > 0; ++b, ta = 0) {
    const int64_t n_tiles = q8_tiles(p, b);
    const int64_t tb = min(n_tiles, ta + left);
    if (tb <= ta) continue;
    left -= tb - ta;
    const WindowView v = window_view(__ldcg(p.context_lens + b), p.q_len, p.bs, p.causal, p.window, p.sinks);
    const int u0 = static_cast<int>(ta * kQ8Tile);
    const int u1 = tb == n_tiles ? v.n : static_cast<int>(tb * kQ8Tile);
    for (int x = tid; x < kNR * kQkDim; x += kThreads) {
      const int r = x / kQkDim, c = x % kQkDim;
      const long long at = static_cast<long long>(b) * rows_total + row0 + r;
      sm.q[r][c] = r >= nrows ? 0.f
                              : h2f<BF16>(c < kRank ? p.q_abs[at * kRank + c] : p.q_pe[at * kRope + c - kRank]);
    }
    if (tid < kNR) {
      sm.m[tid] = -INFINITY;
      sm.l[tid] = 0.f;
    }
    float acc[kNR][2] = {};
    const int r = tid / kStep, tl = tid % kStep;
    const long long row_pos = p.causal ? static_cast<long long>(v.n) - p.q_len + (row0 + r) / p.H : v.n - 1LL;
    for (int u = u0; u < u1; u += kStep) {
      __syncthreads();
      for (int x = tid; x < kStep * (kQkDim / 4); x += kThreads) {
        const int t = x / (kQkDim / 4), c = (x % (kQkDim / 4)) * 4;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (u + t < u1) {
          const int tok = u + t + (u + t >= v.sa ? v.skip : 0);
          const int pg = tok / p.bs;
          const int pid = pg < p.max_blocks ? p.block_table[static_cast<long long>(b) * p.max_blocks + pg] : -1;
          if (pid < 0 || pid >= p.num_blocks) {
            flag_error(MLA_DEVERR_BAD_PAGE);
          } else {
            const long long row = static_cast<long long>(pid) * p.bs + tok % p.bs;
            const uint32_t w = c < kRank ? *reinterpret_cast<const uint32_t*>(p.ckv + row * kRank + c)
                                         : *reinterpret_cast<const uint32_t*>(p.kpe + row * kRope + c - kRank);
            const float z = p.scales[row >> p.g_shift];
            uint32_t a, d;
            e4m3x4_to_f16x4(w, a, d);
            const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
            const float2 fd = __half22float2(*reinterpret_cast<const __half2*>(&d));
            f[0] = fa.x * z;
            f[1] = fa.y * z;
            f[2] = fd.x * z;
            f[3] = fd.y * z;
          }
        }
        for (int j = 0; j < 4; ++j) sm.kv[t][c + j] = f[j];
      }
      __syncthreads();
      float s = 0.f;
      for (int c = 0; c < kQkDim; ++c) s = fmaf(sm.q[r][c], sm.kv[tl][c], s);
      const int ut = u + tl;
      bool vis = ut < u1 && r < nrows && ut <= row_pos;
      if (p.window > 0) vis = vis && (ut > row_pos - p.window || ut < p.sinks);
      s = vis ? s * p.scale_log2 : -INFINITY;
      float mx = s;
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_old = sm.m[r], m_new = fmaxf(m_old, mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float pr = vis ? exp2f(s - ref) : 0.f;
      float sum = pr;
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncwarp();
      if (tl == 0) {
        const float al = m_old == -INFINITY ? 0.f : exp2f(m_old - m_new);
        sm.alpha[r] = al;
        sm.m[r] = m_new;
        sm.l[r] = sm.l[r] * al + sum;
      }
      sm.prob[r][tl] = pr;
      __syncthreads();
      for (int rr = 0; rr < kNR; ++rr) {
        const float al = sm.alpha[rr];
        float a0 = acc[rr][0] * al, a1 = acc[rr][1] * al;
        for (int t = 0; t < kStep; ++t) {
          const float w = sm.prob[rr][t];
          if (w != 0.f) {  // (a hidden token's row may hold anything)
            a0 = fmaf(w, sm.kv[t][tid], a0);
            a1 = fmaf(w, sm.kv[t][tid + kThreads], a1);
          }
        }
        acc[rr][0] = a0;
        acc[rr][1] = a1;
      }
    }
    __syncthreads();
    const bool whole = ta == 0 && tb == n_tiles;
    const long long entry = static_cast<long long>(gang) * 2 + (ta == 0 ? 1 : 0);
    for (int rr = 0; rr < nrows; ++rr) {
      const float m = sm.m[rr], l = sm.l[rr];
      if (whole) {
        const long long at = static_cast<long long>(b) * rows_total + row0 + rr;
        for (int j = 0; j < 2; ++j) {
          const float o = l == 0.f ? 0.f : acc[rr][j] / l;
          const long long off = at * kRank + tid + j * kThreads;
          if (p.out_dtype == 2)
            static_cast<float*>(p.out)[off] = o;
          else
            static_cast<uint16_t*>(p.out)[off] = p.out_dtype == 1 ? f2h<true>(o) : f2h<false>(o);
        }
        if (tid == 0 && p.out_lse != nullptr) p.out_lse[at] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(l);
      } else {
        const long long at = entry * p.row_pad + row0 + rr;
        for (int j = 0; j < 2; ++j) p.ws_o[at * kRank + tid + j * kThreads] = acc[rr][j];
        if (tid == 0) {
          p.ws_ml[at * 2] = m;
          p.ws_ml[at * 2 + 1] = l;
        }
      }
    }
  }
}

// The requests cut by gang borders: per (request, row, 64 columns) the parts of its gangs,
//   M = max m_j, w_j = 2^(m_j - M), out = sum w_j O_j / sum w_j l_j, lse = M + log2 sum w_j l_j.
// 16 column quads x 8 part lanes a block; lane e adds parts e, e + 8, ... in order, then the lanes'
// sums are added in lane order: the same bits on every call.
constexpr int kMergeThreads = 128, kMergeLanes = 8, kMergeCols = 64;
constexpr int kMergeLoads = 10;  // parts a lane has in flight: 80 gangs in a round

struct MergeSmem {
  int64_t scratch[33];
  int cut[kMergeThreads / 32];
  int b[kMergeThreads], j0[kMergeThreads], n[kMergeThreads];
  float4 acc[kMergeLanes][kMergeCols / 4];
  float den[kMergeLanes], max[kMergeLanes];
};

__global__ void __launch_bounds__(kMergeThreads) mla_merge_q8_kernel(const DecodeQ8Params p) {
  __shared__ MergeSmem sm;
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the lengths are no output of the decode kernel, whose start waited for the kernel before it
  const int per = (p.B + kMergeThreads - 1) / kMergeThreads;
  const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0, T = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += q8_tiles(p, b);
  int64_t at = block_prefix<kMergeThreads>(mine, sm.scratch, &T);
  const int64_t J = q8_live_gangs(T, p.gangs);
  pdl_wait();
  if (J < 2) return;
  const int rows_total = p.q_len * p.H;
  const int q = tid % (kMergeCols / 4), e = tid / (kMergeCols / 4);
  // requests are taken in rounds of those that the threads' next ones are
  for (int k = 0; k < per; ++k) {
    __syncthreads();
    int j0 = 0, j1 = 0;
    if (b_lo + k < b_hi) {
      const int64_t n = q8_tiles(p, b_lo + k);
      if (n > 0) {
        j0 = q8_gang_of(at, T, J);
        j1 = q8_gang_of(at + n - 1, T, J);
      }
      at += n;
    }
    // the cut ones among them, in thread order: the same list in every block
    const uint32_t cut = __ballot_sync(0xffffffffu, j1 > j0);
    if (lane == 0) sm.cut[warp] = __popc(cut);
    __syncthreads();
    int count = 0, mine_at = __popc(cut & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) {
      if (w < warp) mine_at += sm.cut[w];
      count += sm.cut[w];
    }
    if (j1 > j0) {
      sm.b[mine_at] = b_lo + k;
      sm.j0[mine_at] = j0;
      sm.n[mine_at] = j1 - j0 + 1;
    }
    __syncthreads();
    const long long items = static_cast<long long>(count) * rows_total * (kRank / kMergeCols);
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
      const int c = static_cast<int>(item % (kRank / kMergeCols)) * kMergeCols + 4 * q;
      const long long rest = item / (kRank / kMergeCols);
      const int row = static_cast<int>(rest % rows_total), i = static_cast<int>(rest / rows_total);
      const int b = sm.b[i], j0 = sm.j0[i], n = sm.n[i];
      // part x of the request: gang j0 + x, entry 1 of the first gang, entry 0 of the others
      auto slot = [&](int x) { return (static_cast<long long>(j0 + x) * 2 + (x == 0 ? 1 : 0)) * p.row_pad + row; };
      float M = -INFINITY, den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x0 = 0; x0 < n; x0 += kMergeLanes * kMergeLoads) {
        float2 ml[kMergeLoads];
        float4 v[kMergeLoads];
#pragma unroll
        for (int y = 0; y < kMergeLoads; ++y) {
          const int x = x0 + e + kMergeLanes * y;
          const bool in = x < n;
          ml[y] = in ? __ldcg(reinterpret_cast<const float2*>(p.ws_ml + slot(x) * 2)) : make_float2(-INFINITY, 0.f);
          v[y] = in ? __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot(x) * kRank + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float m = M;
#pragma unroll
        for (int y = 0; y < kMergeLoads; ++y) m = fmaxf(m, ml[y].x);
        const float ref = m == -INFINITY ? 0.f : m;
        const float al = exp2f(M - ref);  // 0 before the first round
        den *= al;
        acc = make_float4(acc.x * al, acc.y * al, acc.z * al, acc.w * al);
        M = m;
#pragma unroll
        for (int y = 0; y < kMergeLoads; ++y) {
          // a part without a visible token has l = 0; one whose every score is NaN has no maximum, and l NaN
          const float w = ml[y].y == 0.f ? 0.f : (ml[y].x == -INFINITY ? 1.f : exp2f(ml[y].x - ref));
          den = fmaf(w, ml[y].y, den);
          acc.x = fmaf(w, v[y].x, acc.x);
          acc.y = fmaf(w, v[y].y, acc.y);
          acc.z = fmaf(w, v[y].z, acc.z);
          acc.w = fmaf(w, v[y].w, acc.w);
        }
      }
      __syncthreads();
      sm.acc[e][q] = acc;
      if (q == 0) {
        sm.den[e] = den;
        sm.max[e] = M;
      }
      __syncthreads();
      if (e == 0) {
        float Mt = -INFINITY;
#pragma unroll
        for (int y = 0; y < kMergeLanes; ++y) Mt = fmaxf(Mt, sm.max[y]);
        const float ref = Mt == -INFINITY ? 0.f : Mt;
        float dt = 0.f;
        float4 at4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kMergeLanes; ++y) {
          const float w = sm.den[y] == 0.f ? 0.f : (sm.max[y] == -INFINITY ? 1.f : exp2f(sm.max[y] - ref));
          const float4 v = sm.acc[y][q];
          dt = fmaf(w, sm.den[y], dt);
          at4.x = fmaf(w, v.x, at4.x);
          at4.y = fmaf(w, v.y, at4.y);
          at4.z = fmaf(w, v.z, at4.z);
          at4.w = fmaf(w, v.w, at4.w);
        }
        const long long br = static_cast<long long>(b) * rows_total + row;
        const bool none = dt == 0.f;
        store_out4(p.out, p.out_dtype, br * kRank + c,
                   none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(at4.x / dt, at4.y / dt, at4.z / dt, at4.w / dt));
        if (p.out_lse != nullptr && c == 0 && q == 0) p.out_lse[br] = none ? -INFINITY : ref + log2f(dt);
      }
    }
  }
}

}  // namespace

int q8_rows_per_cta(int total_rows) {
  (void)total_rows;
  return kNR;
}
int q8_gangs(int total_rows, int sms) {
  const int groups = (total_rows + kNR - 1) / kNR;
  return sms > groups ? sms / groups : 1;
}

cudaError_t launch_decode_q8(const DecodeQ8Params& p, bool bf16, cudaStream_t stream) {
  const void* fn = bf16 ? reinterpret_cast<const void*>(&mla_decode_q8_kernel<true>)
                        : reinterpret_cast<const void*>(&mla_decode_q8_kernel<false>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.groups), static_cast<unsigned>(p.gangs), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = bf16 ? cudaLaunchKernelEx(&cfg, mla_decode_q8_kernel<true>, p)
           : cudaLaunchKernelEx(&cfg, mla_decode_q8_kernel<false>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(2 * 152, 1, 1);
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mla_merge_q8_kernel, p);
}

cudaError_t decode_q8_read_clear_error(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_device_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(uint32_t));
}

}  // namespace mla
