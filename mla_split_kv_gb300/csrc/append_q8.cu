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
// One group of warps per (request, block that its new tokens touch): the
// tokens' maximum, then the bytes. A copy in kind: 1152 bytes read and 576
// written per token; HBM-bound for a prefill chunk, one chain of dependent
// loads (length, table entry, token, old scale) for a single token.
#include "device_common.cuh"

namespace mla {

namespace {

constexpr int kWarps = 8;
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

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = h2f<BF16>(static_cast<uint16_t>(w[j] & 0xffffu));
    x[2 * j + 1] = h2f<BF16>(static_cast<uint16_t>(w[j] >> 16));
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32) mla_append_q8_kernel(const AppendQ8Params p, int per_request,
                                                                     int warps_per_block) {
  __shared__ float red[kWarps];
  pdl_wait();  // the kernel before it may produce the new tokens, or still read the cache
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % warps_per_block;  // this warp takes new tokens sub, sub + warps_per_block, ... of its block
  const long long unit = static_cast<long long>(blockIdx.x) * (kWarps / warps_per_block) + warp / warps_per_block;
  const long long units = static_cast<long long>(p.B) * per_request;
  const int b = static_cast<int>(unit / per_request);
  int t_lo = 0, t_hi = 0;       // the block's new tokens, positions [t_lo, t_hi)
  long long first = 0, row0 = 0;  // position of the request's new token 0; cache row of the block's first token
  if (unit < units) {
    first = static_cast<long long>(p.context_lens[b]) - p.q_len;
    const long long start = first > 0 ? first : 0;
    const long long blk = start / p.g + unit % per_request;
    const long long end = first + p.q_len;
    const long long lo = max(start, blk * p.g), hi = min(end, (blk + 1) * p.g);
    if (lo < hi) {
      const long long pg = blk * p.g / p.bs;
      const int pid = pg < p.max_blocks ? p.block_table[static_cast<long long>(b) * p.max_blocks + pg] : -1;
      if (pid < 0 || pid >= p.num_blocks) {  // outside the table or the pool: nothing is written
        if (sub == 0 && lane == 0) flag_error(MLA_DEVERR_BAD_PAGE);
      } else {
        row0 = static_cast<long long>(pid) * p.bs + blk * p.g % p.bs;
        t_lo = static_cast<int>(lo - blk * p.g);
        t_hi = static_cast<int>(hi - blk * p.g);
        first -= blk * p.g;  // (of the block's own positions from here on)
      }
    }
  }
  // a lane's 16 latent values of a token, and 8 rope values for lanes 0-7
  auto load = [&](int t, float* x) {
    const long long tok = static_cast<long long>(b) * p.q_len + (t - first);
    const uint4* c = reinterpret_cast<const uint4*>(p.ckv_new + tok * kRank) + 2 * lane;
    unpack8<BF16>(c[0], x);
    unpack8<BF16>(c[1], x + 8);
    if (lane < kRope / 8) {
      unpack8<BF16>(reinterpret_cast<const uint4*>(p.kpe_new + tok * kRope)[lane], x + 16);
    } else {
#pragma unroll
      for (int j = 16; j < 24; ++j) x[j] = 0.f;
    }
  };
  float amax = 0.f;
  for (int t = t_lo + sub; t < t_hi; t += warps_per_block) {
    float x[24];
    load(t, x);
#pragma unroll
    for (int j = 0; j < 24; ++j) amax = max_nan(amax, fabsf(x[j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < warps_per_block; ++w) amax = max_nan(amax, red[warp - sub + w]);
  if (t_lo >= t_hi) return;
  float s = block_scale(amax);
  float* const scale_at = p.scales + row0 / p.g;
  if (t_lo > 0) {  // earlier tokens stay in the block: its scale only grows, and their bytes with it
    const float before = *scale_at;
    const float fresh = s;
    s = max_nan(before, fresh);
    if (s > before) {
      const float ratio = __fdiv_rn(before, s);
      for (int t = sub; t < t_lo; t += warps_per_block) {
        auto move4 = [&](uint8_t* at) {
          uint32_t* const w = reinterpret_cast<uint32_t*>(at);
          uint32_t lo, hi;
          e4m3x4_to_f16x4(*w, lo, hi);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          *w = e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) move4(p.ckv + (row0 + t) * kRank + 4 * (lane + 32 * j));
        if (lane < kRope / 4) move4(p.kpe + (row0 + t) * kRope + 4 * lane);
      }
    }
  }
  const bool poisoned = s != s;
  for (int t = t_lo + sub; t < t_hi; t += warps_per_block) {
    float x[24];
    load(t, x);
#pragma unroll
    for (int j = 0; j < 24; ++j) x[j] = poisoned ? 0.f : __fdiv_rn(x[j], s);
    uint4 v;
    v.x = e4m3x4(x[0], x[1], x[2], x[3]);
    v.y = e4m3x4(x[4], x[5], x[6], x[7]);
    v.z = e4m3x4(x[8], x[9], x[10], x[11]);
    v.w = e4m3x4(x[12], x[13], x[14], x[15]);
    reinterpret_cast<uint4*>(p.ckv + (row0 + t) * kRank)[lane] = v;
    if (lane < kRope / 8) {
      uint2 u;
      u.x = e4m3x4(x[16], x[17], x[18], x[19]);
      u.y = e4m3x4(x[20], x[21], x[22], x[23]);
      reinterpret_cast<uint2*>(p.kpe + (row0 + t) * kRope)[lane] = u;
    }
  }
  // written by one lane after every warp of the block has read the old one
  if (warps_per_block > 1)
    named_bar_sync(1 + warp / warps_per_block, warps_per_block * 32);
  else
    __syncwarp();
  if (sub == 0 && lane == 0) *scale_at = s;
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Params& p, bool bf16, cudaStream_t stream) {
  // blocks of g tokens that q_len consecutive ones can touch
  const int per_request = (p.q_len - 1) / p.g + (p.g > 1 ? 2 : 1);
  // a warp takes up to 4 tokens of a block
  int wpb = 1;
  while (wpb < kWarps && wpb * 4 < (p.g < p.q_len ? p.g : p.q_len)) wpb *= 2;
  const long long units = static_cast<long long>(p.B) * per_request;
  const long long blocks = (units + kWarps / wpb - 1) / (kWarps / wpb);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, mla_append_q8_kernel<true>, p, per_request, wpb)
              : cudaLaunchKernelEx(&cfg, mla_append_q8_kernel<false>, p, per_request, wpb);
}

cudaError_t append_q8_read_clear_error(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_device_error, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(uint32_t));
}

}  // namespace mla
