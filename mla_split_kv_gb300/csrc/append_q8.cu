// The write into a block-scaled 8-bit cache, sm_103a.
//
// Each run of g consecutive tokens of a page is a block with one scale s, a
// power of two: a value x is stored as the E4M3 byte nearest to x / s (ties to
// even, +-448 beyond). s is the least power of two in [2^-60, 2^60] with
// max |x| / s <= 448 over the block's tokens, latent and rope columns alike.
// E4M3 is a floating-point format: a scale between two powers of two would
// give no value more bits, while with a power of two the division and, when a
// later token makes the block's scale grow, the move of the bytes already
// there are exact but for the smallest values.
//
// A copy in kind: 1152 bytes read and 576 written per token; HBM-bound for a
// prefill chunk, one chain of dependent loads (length, then token, table entry
// and old scale) for a single token. So a warp takes four consecutive tokens
// and keeps them in registers between the maximum and the bytes (nothing is
// read twice, and 4.6 KB per warp are in flight), the warps of a block meet
// once, and the maximum is taken over the 16-bit patterns themselves: without
// its sign a pattern orders like its value, NaN above infinity. 65,536 tokens
// in blocks of one: 23.3 us, 4.9 TB/s (one token at a time per warp, read
// twice: 87 us); a single token: 3.6 us.
#include "device_common.cuh"

namespace mla {

namespace {

constexpr int kWarps = 16, kFewWarps = 8;  // of a CTA; where a block needs no more, 8: shorter tails (23.3 us, 25.3 with 16)
constexpr int kHold = 4;  // tokens per warp: 16 warps hold a block of the longest page, 64 tokens
constexpr int kMinExp = -60, kMaxExp = 60;

// The least power of two s >= 2^-60 with amax / s <= 448, as float bits; NaN where amax is not finite or
// s would pass 2^60. 448 = 1.75 * 2^8: s = 2^(e - 8) for amax = f 2^e, f in [1, 1.75], twice that above.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7fffffffu;
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  const int k = max(e, kMinExp);  // (zero and subnormal amax: e < kMinExp)
  if (b >= 0x7f800000u || k > kMaxExp) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// the larger pattern without its sign, in each half
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, const uint4 v) {
  m = __vmaxu2(__vmaxu2(m, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
  return __vmaxu2(__vmaxu2(m, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
}

// An fp32 result cut off towards zero, with its last bit set where something was cut off (`rest`): rounded to fewer
// bits, this gives what the exact result does, while a result already rounded to nearest may lie on a tie that the
// exact one does not. (Its 24 bits are many more than E4M3's 4 and two.)
__device__ __forceinline__ float sticky(float cut, float rest) {
  return rest != 0.f ? __uint_as_float(__float_as_uint(cut) | 1u) : cut;
}

// Eight values over the scale: by its inverse where it is a power of two (the same result, s and 1 / s are exact),
// else (a scale from elsewhere that stays in force) by division.
template <bool BF16>
__device__ __forceinline__ uint2 quantize8(const uint4 v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = h2f<BF16>(static_cast<uint16_t>(w[j] & 0xffffu));
    x[2 * j + 1] = h2f<BF16>(static_cast<uint16_t>(w[j] >> 16));
  }
  if (inv != 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = __fdiv_rz(x[j], s);
      x[j] = sticky(q, fmaf(-q, s, x[j]));
    }
  }
  return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}

// a stored byte's value times ratio in fp32 (exact where the old scale is a power of two), four in a word
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
}

// A unit is one aligned run of max(g, kHold) tokens of a request, which lies in one page: `subs` warps of kHold tokens
// each. A run longer than a block (g < kHold) holds kHold / g of them, all one warp's.
template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32, 2) mla_append_q8_kernel(const AppendQ8Params p, uint32_t per_request,
                                                                        int subs) {
  __shared__ uint32_t red[kWarps];
  pdl_wait();  // the kernel before it may produce the new tokens, or still read the cache
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & (subs - 1);
  const uint32_t unit = blockIdx.x * ((blockDim.x >> 5) / subs) + warp / subs;  // (at most 1.25 B q_len + 2 B: below 2^32)
  if (unit >= per_request * p.B) return;
  const uint32_t b = unit / per_request;
  const int run = subs * kHold;
  const long long first = static_cast<long long>(p.context_lens[b]) - p.q_len;  // position of new token 0
  const long long start = max(first, 0ll);
  const long long base = (start / run + unit % per_request) * run;
  const long long end = first + p.q_len;
  if (end <= base) return;  // (the unit's warps alike)
  // the run's new tokens are its [t_lo, t_hi)
  const int t_lo = static_cast<int>(max(start, base) - base), t_hi = static_cast<int>(min(end - base, static_cast<long long>(run)));
  const long long pg = base / p.bs;
  const int pid = pg < p.max_blocks ? p.block_table[static_cast<long long>(b) * p.max_blocks + pg] : -1;

  // lane l holds columns 8 l.. and 256 + 8 l.. of the warp's four tokens, and rope columns 8 (l % 8).. of token l / 8
  const long long tok = static_cast<long long>(b) * p.q_len + (base + sub * kHold - first);
  uint4 c0[kHold], c1[kHold], r = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int t = sub * kHold + j;
    c0[j] = c1[j] = make_uint4(0, 0, 0, 0);
    if (t >= t_lo && t < t_hi) {
      const uint4* const c = reinterpret_cast<const uint4*>(p.ckv_new + (tok + j) * kRank);
      c0[j] = c[lane];
      c1[j] = c[lane + 32];
    }
  }
  const int rt = sub * kHold + (lane >> 3);
  if (rt >= t_lo && rt < t_hi)
    r = reinterpret_cast<const uint4*>(p.kpe_new + (tok + (lane >> 3)) * kRope)[lane & 7];

  const bool bad = pid < 0 || pid >= p.num_blocks;  // outside the table or the pool: nothing is written
  const long long row = bad ? 0 : static_cast<long long>(pid) * p.bs + base % p.bs;
  float* const scales = p.scales + row / p.g;
  const int kept = t_lo & (p.g - 1);  // earlier tokens that stay in the block of the first new one
  const float before = kept != 0 && !bad ? scales[t_lo / p.g] : 0.f;

  uint32_t m[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    uint32_t v = max_abs2(max_abs2(0u, c0[j]), c1[j]);
    if ((lane >> 3) == j) v = max_abs2(v, r);
    m[j] = __reduce_max_sync(0xffffffffu, max(v & 0xffffu, v >> 16));
  }
  if (p.g >= kHold) {  // one block: its maximum over the warps
    uint32_t all = max(max(m[0], m[1]), max(m[2], m[3]));
    if (subs > 1) {
      if (lane == 0) red[warp] = all;
      named_bar_sync(1 + warp / subs, subs * 32);  // (every warp has read the block's old scale, too)
      all = __reduce_max_sync(0xffffffffu, lane < subs ? red[warp - sub + lane] : 0u);
    }
#pragma unroll
    for (int j = 0; j < kHold; ++j) m[j] = all;
  } else if (p.g == 2) {
    m[0] = m[1] = max(m[0], m[1]);
    m[2] = m[3] = max(m[2], m[3]);
  }
  if (bad) {
    if (sub == 0 && lane == 0) flag_error(MLA_DEVERR_BAD_PAGE);
    return;
  }
  __syncwarp();

  float rope_s = 0.f, rope_inv = 0.f;
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int t = sub * kHold + j;
    float s = block_scale(h2f<BF16>(static_cast<uint16_t>(m[j])));
    if (kept != 0 && t / p.g == t_lo / p.g) {  // earlier tokens stay: the scale only grows, and their bytes with it
      s = max_nan(before, s);
      if (t < t_lo && s > before) {
        const float ratio = __fdiv_rn(before, s);
        uint4* const at = reinterpret_cast<uint4*>(p.ckv + (row + t) * kRank) + lane;
        uint4 v = *at;
        v.x = rescale4(v.x, ratio);
        v.y = rescale4(v.y, ratio);
        v.z = rescale4(v.z, ratio);
        v.w = rescale4(v.w, ratio);
        *at = v;
        if (lane < kRope / 4) {
          uint32_t* const kt = reinterpret_cast<uint32_t*>(p.kpe + (row + t) * kRope) + lane;
          *kt = rescale4(*kt, ratio);
        }
      }
    }
    const uint32_t bits = __float_as_uint(s);
    const float inv = (bits & 0x7fffffu) == 0 && bits < (254u << 23) ? __uint_as_float((254u << 23) - bits) : 0.f;
    if (t >= t_lo && t < t_hi) {
      const bool poisoned = s != s;  // the block's values are lost: its scale says so
      const uint2 z = make_uint2(0, 0);
      uint2* const at = reinterpret_cast<uint2*>(p.ckv + (row + t) * kRank) + lane;
      at[0] = poisoned ? z : quantize8<BF16>(c0[j], s, inv);
      at[32] = poisoned ? z : quantize8<BF16>(c1[j], s, inv);
    }
    if ((lane >> 3) == j) {
      rope_s = s;
      rope_inv = inv;
    }
    // one lane writes the scale of each block with a new token
    const int lo = t & ~(p.g - 1);
    if (lane == 0 && t == lo && lo < t_hi && lo + p.g > t_lo) scales[t / p.g] = s;
  }
  if (rt >= t_lo && rt < t_hi)
    reinterpret_cast<uint2*>(p.kpe + (row + rt) * kRope)[lane & 7] =
        rope_s != rope_s ? make_uint2(0, 0) : quantize8<BF16>(r, rope_s, rope_inv);
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Params& p, bool bf16, cudaStream_t stream) {
  const int run = p.g > kHold ? p.g : kHold, subs = run / kHold;
  // aligned runs that q_len consecutive tokens can touch
  const uint32_t per_request = static_cast<uint32_t>((static_cast<int64_t>(p.q_len) + run - 2) / run + 1);
  const int64_t units = static_cast<int64_t>(p.B) * per_request;
  const int warps = subs > kFewWarps ? kWarps : kFewWarps;
  const int64_t blocks = (units + warps / subs - 1) / (warps / subs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(warps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, mla_append_q8_kernel<true>, p, per_request, subs)
              : cudaLaunchKernelEx(&cfg, mla_append_q8_kernel<false>, p, per_request, subs);
}

cudaError_t append_q8_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
