// Gradient of the linear router L = x W_r^T (+ b) for a dense gradient dL of the logits:
//   dW_r (+)= dL^T x,   db (+)= sum_t dL[t],   dx (+)= dL W_r.
// The layer's own backward pass (backward.cu) knows a dL that is zero except on each token's
// chosen experts; a loss on the router (balance_loss.cu) has a gradient on every logit.
//
// CUDA-core path: one launch, two kinds of CTAs. "W" CTAs own 16 experts x 128 columns of dW_r
// and a range of the tokens; "x" CTAs own 16 tokens x 256 columns of dx. Every product is fp32.
// Several token ranges leave partial sums, which a second launch adds in order.
#include <math.h>

#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"
#include "tma_host.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWExperts = 16, kWCols = 128, kWTokens = 32;
constexpr int kXTokens = 16, kXCols = 256, kXExperts = 64;

struct Plan {
  int w_cols, w_experts, chunks;  // grid of the W CTAs
  int64_t most_chunks;            // ranges asked for; never fewer for a larger T
  int64_t chunk;                  // tokens of a range
  int x_cols;
  int64_t x_tokens;               // grid of the x CTAs
};

Plan make_plan(int64_t T, int N, int d) {
  Plan p{};
  p.w_cols = (d + kWCols - 1) / kWCols;
  p.w_experts = (N + kWExperts - 1) / kWExperts;
  const int64_t tiles = static_cast<int64_t>(p.w_cols) * p.w_experts;
  const int64_t most = (T + 2 * kWTokens - 1) / (2 * kWTokens);  // ranges of at least 64 tokens
  p.most_chunks = std::max<int64_t>(1, std::min<int64_t>({most, 2 * 148 / tiles, 64}));
  p.chunk = (T + p.most_chunks - 1) / p.most_chunks;
  p.chunks = T > 0 ? static_cast<int>((T + p.chunk - 1) / p.chunk) : 0;
  p.x_cols = (d + kXCols - 1) / kXCols;
  p.x_tokens = (T + kXTokens - 1) / kXTokens;
  return p;
}

struct Params {
  const uint16_t* x;
  const float* w;
  const float* dl;
  float* d_x;
  float* d_w;
  float* d_b;
  float* part_w;  // [chunks][N][d], several ranges only
  float* part_b;  // [chunks][N]
  int T, N, d, accumulate;
  int w_cols, w_experts, chunks, x_cols;
  int64_t chunk, w_ctas;
};

__device__ __forceinline__ void w_tile(const Params& a, uint32_t (*s_x)[kWCols / 2], float (*s_dl)[kWExperts]) {
  const int tile = static_cast<int>(blockIdx.x % (static_cast<int64_t>(a.w_cols) * a.w_experts));
  const int range = static_cast<int>(blockIdx.x / (static_cast<int64_t>(a.w_cols) * a.w_experts));
  const int c0 = tile % a.w_cols * kWCols, n0 = tile / a.w_cols * kWExperts;
  const int64_t t0 = range * a.chunk, t1 = min(static_cast<int64_t>(a.T), t0 + a.chunk);
  const int cp = threadIdx.x & 63, eg = threadIdx.x >> 6;  // column pair, group of 4 experts
  float acc[4][2] = {};
  float b = 0.f;
  // the next tile's loads are under way while a tile is used: 16 bytes of x and of dL a thread
  constexpr int kXLoads = kWTokens * kWCols / 8 / kThreads, kDlLoads = kWTokens * kWExperts / kThreads;
  uint4 nx[kXLoads];
  float nd[kDlLoads];
  auto fetch = [&](int64_t tb) {
#pragma unroll
    for (int k = 0; k < kXLoads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      const int64_t t = tb + i / (kWCols / 8);
      const int c = c0 + i % (kWCols / 8) * 8;
      nx[k] = t < t1 && c < a.d ? __ldg(reinterpret_cast<const uint4*>(a.x + t * a.d + c)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kDlLoads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      const int64_t t = tb + i / kWExperts;
      const int n = n0 + i % kWExperts;
      nd[k] = t < t1 && n < a.N ? __ldg(a.dl + t * a.N + n) : 0.f;
    }
  };
  fetch(t0);
  for (int64_t tb = t0; tb < t1; tb += kWTokens) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kXLoads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      *reinterpret_cast<uint4*>(&s_x[i / (kWCols / 8)][i % (kWCols / 8) * 4]) = nx[k];
    }
#pragma unroll
    for (int k = 0; k < kDlLoads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      s_dl[i / kWExperts][i % kWExperts] = nd[k];
    }
    __syncthreads();
    fetch(tb + kWTokens);
#pragma unroll 8
    for (int u = 0; u < kWTokens; ++u) {
      const uint32_t xv = s_x[u][cp];
      const float x0 = __uint_as_float(xv << 16), x1 = __uint_as_float(xv & 0xffff0000u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = s_dl[u][eg * 4 + j];
        acc[j][0] += g * x0;
        acc[j][1] += g * x1;
      }
    }
    if (threadIdx.x < kWExperts && c0 == 0)
      for (int u = 0; u < kWTokens; ++u) b += s_dl[u][threadIdx.x];
  }
  const int c = c0 + cp * 2;
  if (a.d_w != nullptr && c < a.d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + eg * 4 + j;
      if (n >= a.N) continue;
      const int64_t o = static_cast<int64_t>(n) * a.d + c;
      float2 v = make_float2(acc[j][0], acc[j][1]);
      float* out = a.chunks > 1 ? a.part_w + static_cast<int64_t>(range) * a.N * a.d : a.d_w;
      if (a.chunks == 1 && a.accumulate) {
        const float2 old = *reinterpret_cast<const float2*>(out + o);
        v.x += old.x;
        v.y += old.y;
      }
      *reinterpret_cast<float2*>(out + o) = v;
    }
  }
  if (a.d_b != nullptr && c0 == 0 && threadIdx.x < kWExperts && n0 + threadIdx.x < a.N) {
    const int n = n0 + threadIdx.x;
    if (a.chunks > 1) a.part_b[static_cast<int64_t>(range) * a.N + n] = b;
    else a.d_b[n] = a.accumulate ? a.d_b[n] + b : b;
  }
}

__device__ __forceinline__ void x_tile(const Params& a, float (*s_dl)[kXExperts]) {
  const int64_t tile = blockIdx.x - a.w_ctas;
  const int c = static_cast<int>(tile % a.x_cols) * kXCols + (threadIdx.x & 63) * 4;
  const int64_t t0 = tile / a.x_cols * kXTokens;
  const int tg = threadIdx.x >> 6;  // group of 4 tokens
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int nb = 0; nb < a.N; nb += kXExperts) {
    __syncthreads();
    for (int i = threadIdx.x; i < kXTokens * kXExperts; i += kThreads) {
      const int64_t t = t0 + i / kXExperts;
      const int n = nb + i % kXExperts;
      s_dl[i / kXExperts][i % kXExperts] = t < a.T && n < a.N ? a.dl[t * a.N + n] : 0.f;
    }
    __syncthreads();
    const int n1 = min(kXExperts, a.N - nb);
    if (c < a.d) {
#pragma unroll 8
      for (int n = 0; n < n1; ++n) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(a.w + static_cast<int64_t>(nb + n) * a.d + c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = s_dl[tg * 4 + i][n];
          acc[i].x += g * w.x;
          acc[i].y += g * w.y;
          acc[i].z += g * w.z;
          acc[i].w += g * w.w;
        }
      }
    }
  }
  if (c >= a.d) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + tg * 4 + i;
    if (t >= a.T) break;
    float4* out = reinterpret_cast<float4*>(a.d_x + t * a.d + c);
    if (a.accumulate) {
      const float4 old = *out;
      acc[i].x += old.x;
      acc[i].y += old.y;
      acc[i].z += old.z;
      acc[i].w += old.w;
    }
    *out = acc[i];
  }
}

__global__ void __launch_bounds__(kThreads) router_backward_kernel(const Params a) {
  __shared__ __align__(16) uint32_t s_x[kWTokens][kWCols / 2];
  __shared__ float s_w[kWTokens][kWExperts];
  __shared__ float s_dl[kXTokens][kXExperts];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x < a.w_ctas) w_tile(a, s_x, s_w);
  else x_tile(a, s_dl);
}

// The token ranges' partial sums. CTAs [0, w_ctas): 256 / SPLIT float4s of dW_r each, SPLIT threads a
// float4 over a part of the ranges each, whose sums are added in order; the bias gradient's by a
// warp an expert, 32 strided sums and their tree.
// Up to here a float4 takes one thread. Device time of dW, one thread and four, us: 5 ranges of 256 x 7168
// 142.6, 145.0; 8 of 64 x 1024 8.8, 9.2; 24 of 64 x 2048 33.6, 32.1; 36 of 32 x 2880 47, 36.
constexpr int kSumAlone = 8;
template <int SPLIT>
__global__ void __launch_bounds__(256) router_backward_sum_kernel(
    const float* __restrict__ part_w, const float* __restrict__ part_b, float* __restrict__ d_w,
    float* __restrict__ d_b, int chunks, int b_parts, int N, int d, int accumulate, int w_ctas) {
  constexpr int kItems = 256 / SPLIT;
  __shared__ float4 s_part[SPLIT][kItems];
  pdl_trigger();
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= w_ctas) {
    const int n = (blockIdx.x - w_ctas) * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (n >= N) return;
    float s = 0.f;
#pragma unroll 4
    for (int c = lane; c < b_parts; c += 32) s += part_b[static_cast<int64_t>(c) * N + n];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) d_b[n] = accumulate ? d_b[n] + s : s;
    return;
  }
  const int64_t items = static_cast<int64_t>(N) * d / 4;
  const int part = threadIdx.x / kItems, j = threadIdx.x % kItems;
  const int64_t i = blockIdx.x * static_cast<int64_t>(kItems) + j;
  float4* out = reinterpret_cast<float4*>(d_w) + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f), old = s;
  if (i < items) {
    if (accumulate && part == 0) old = __ldcs(out);
    const int c1 = chunks * (part + 1) / SPLIT;
#pragma unroll 8
    for (int c = chunks * part / SPLIT; c < c1; ++c) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(part_w) + c * items + i);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  if (SPLIT > 1) {
    s_part[part][j] = s;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int q = 1; q < SPLIT; ++q) {
      const float4 v = s_part[q][j];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  if (i >= items) return;
  if (accumulate) s = make_float4(s.x + old.x, s.y + old.y, s.z + old.z, s.w + old.w);
  *out = s;
}

template <int SPLIT>
cudaError_t launch_sum_split(const float* part_w, const float* part_b, const RouterBackwardArgs& a, int chunks,
                             int b_parts, cudaStream_t s) {
  constexpr int kItems = 256 / SPLIT;
  const int64_t items = static_cast<int64_t>(a.N) * a.d / 4;
  const int w_ctas = a.d_w_router != nullptr ? static_cast<int>((items + kItems - 1) / kItems) : 0;
  const int b_ctas = a.d_logit_bias != nullptr ? (a.N + 7) / 8 : 0;
  return launch_pdl(router_backward_sum_kernel<SPLIT>, dim3(w_ctas + b_ctas), dim3(256), 0, s, part_w, part_b,
                    a.d_w_router, a.d_logit_bias, chunks, b_parts, a.N, a.d, a.accumulate, w_ctas);
}

cudaError_t launch_sum(const float* part_w, const float* part_b, const RouterBackwardArgs& a, int chunks,
                       int b_parts, cudaStream_t s) {
  return chunks <= kSumAlone ? launch_sum_split<1>(part_w, part_b, a, chunks, b_parts, s)
                             : launch_sum_split<4>(part_w, part_b, a, chunks, b_parts, s);
}

// ------------------------------------------------------------------ tensor-core path
// Both products have fp32 operands, which are written once as sums of 16-bit terms:
//   dL^T x   x is exactly bf16, so dL is three bf16 terms (24 bits): three products;
//   dL W_r   both are two fp16 terms after scaling by powers of two, exact: row n of W_r by
//            2^(14 - b_n), b_n the exponent of its largest magnitude, and dL[t, n] by
//            2^(14 + b_n - a_t), a_t that of the largest dL[t, n] 2^(b_n). Three products (the
//            fourth is below 2^-22); the result of token t is scaled back by 2^(a_t - 28). Three bf16
//            terms of each would need six products. Two terms leave at most 2^-22 of a scaled
//            operand, or 2^-25 where the second is subnormal (operands 2^-16 below the largest): in
//            all 3 2^-22 of the products' magnitudes and N 2^-37 of the token's largest dL[t, n]
//            max_c |W_r[n, c]|, which is what a column small in every row gets.
// The accumulator of the MMA truncates: measured, a chain of additions loses 1.1e-8 of its value a
// step of 16 products. dx has 3 N / 16 <= 48 steps. dW's chains would be thousands; they are cut
// after 48 steps and summed in fp32 registers by the epilogue warps, while the other half of
// TMEM takes the next chain.
constexpr int kKb = 32;             // reduction elements of a stage
constexpr int kBox = 64 * kKb * 2;  // one TMA box of an MN-major operand: 64 MN x 32 k, 128B-swizzled
constexpr int kTcThreads = 320;     // TMA producer, MMA issuer, eight epilogue warps
constexpr int kTcMinSmem = 120 * 1024;  // one CTA an SM: the TMEM is not shared
constexpr int kTcMaxSmem = 226 * 1024;  // dynamic; barriers beside it
constexpr int kWTile = 256;         // columns of d a CTA of the weight gradient owns
constexpr int kXTileT = 128, kXTileC = 256;

// Shared-memory descriptor of an MN-major operand of kKb k rows: groups of 8 k rows are 1024 bytes
// (stride offset), blocks of 64 MN elements `lead` bytes apart (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// The same in blocks of 32 MN elements (64-byte rows, 64B-swizzled): groups of 8 k rows are 512 bytes,
// blocks 64 * kKb.
__device__ __forceinline__ uint64_t desc_mn32(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((64u * kKb) >> 4) << 16) |
         (static_cast<uint64_t>(512u >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
// K-major operand with 64-byte rows (32 elements, 64B-swizzled): groups of 8 rows are 512 bytes.
__device__ __forceinline__ uint64_t desc_k64(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) |
         (static_cast<uint64_t>(512u >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

// True on one lane, always the same one. The MMA warp runs its loops as a whole and elects a lane for
// each instruction: loops, waits and operands stay uniform over the warp. With a branch on the lane
// around the loops dW took 36 us at T = 16384, N = 32, d = 2880, and 29 so.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

struct TcPlan {
  int np;  // N rounded up to 8: row length of dL's terms
  int group;  // experts of a weight-gradient tile: 32, 64 or 128
  int planes;  // planes of partial sums a range leaves: 3, 2, 1
  int n_tiles, c_tiles, chunks;
  int64_t chunk;  // tokens of a range of the weight gradient, a multiple of kKb
  int split_rows, split_ctas;  // tokens a CTA of split_dl_kernel takes, and how many such CTAs
  size_t dl16_bytes, dl_bytes, w_bytes, exp_bytes, part_bytes, bias_bytes;
  size_t total() const { return dl16_bytes + dl_bytes + w_bytes + exp_bytes + part_bytes + bias_bytes; }
};
// A stage of the weight gradient: dL's terms (32 or 64 experts: three and a plane of zeros), then x.
__host__ __device__ constexpr int w_a_bytes(int group) { return (group == 32 ? 4 * 32 : group == 64 ? 4 * 64 : 3 * 128) * kKb * 2; }
__host__ __device__ constexpr int w_stage_bytes(int group) { return w_a_bytes(group) + kWTile * kKb * 2; }
__host__ __device__ constexpr int w_stages(int group) {
  return (kTcMaxSmem - 1024) / w_stage_bytes(group) < 8 ? (kTcMaxSmem - 1024) / w_stage_bytes(group) : 8;
}

constexpr int64_t kSplitCtas = 592;  // of split_dl_kernel at most: four an SM
// Lanes a token takes in split_dl_kernel and pairs of values a lane holds: 2 g p >= N.
struct SplitShape {
  int g, p;
};
SplitShape split_shape(int N) {
  return N <= 8 ? SplitShape{4, 1} : N <= 16 ? SplitShape{8, 1} : N <= 32 ? SplitShape{16, 1}
       : N <= 64 ? SplitShape{32, 1} : N <= 128 ? SplitShape{32, 2} : SplitShape{32, 4};
}

// Waves of 148 CTAs that c token ranges of each tile take, and the cost of a wave besides its tokens:
// starting and ending a CTA costs about what 128 tokens do.
int64_t waves(int64_t tiles, int64_t c) { return (tiles * c + 147) / 148; }
constexpr int64_t kWaveTokens = 128;
constexpr int64_t kMaxRanges = 32, kMinRange = 256;  // ranges at most, tokens of one at least

// A bound of the number of token ranges for any batch of up to T tokens, which does not fall as T
// grows. c ranges are chosen over q < c only if waves(c) (t / c + 128) < waves(q) (t / q + 32 + 128),
// 32 covering the rounding of q's ranges. Both sides are linear in t, so a t in [256 c, T] with that
// means that one of the ends has it.
int64_t most_ranges(int64_t T, int64_t tiles) {
  int64_t most = 1;
  for (int64_t c = 2; c <= kMaxRanges && T / c >= kMinRange; ++c) {
    auto over = [&](int64_t q, int64_t t) {
      return waves(tiles, c) * q * (t + kWaveTokens * c) < waves(tiles, q) * c * (t + (kKb + kWaveTokens) * q);
    };
    bool ever = true;
    for (int64_t q = 1; q < c; ++q) ever = ever && (over(q, kMinRange * c) || over(q, T));
    if (ever) most = c;
  }
  return most;
}

// for_any: the sizes are enough for every batch of up to T tokens on this path, not this one's own.
TcPlan make_tc_plan(int64_t T, int N, int d, bool for_any = false) {
  TcPlan p{};
  p.np = (N + 7) / 8 * 8;
  p.group = N <= 32 ? 32 : N <= 64 ? 64 : 128;
  p.planes = p.group == 32 ? 3 : p.group == 64 ? 2 : 1;
  p.n_tiles = (N + p.group - 1) / p.group;
  p.c_tiles = (d + kWTile - 1) / kWTile;
  // Token ranges: the fewest tokens a CTA in all, by whole waves
  const int64_t tiles = static_cast<int64_t>(p.n_tiles) * p.c_tiles;
  int64_t best = 0;
  for (int64_t c = 1; c <= kMaxRanges && (c == 1 || T / c >= kMinRange); ++c) {
    const int64_t len = ((T + c - 1) / c + kKb - 1) / kKb * kKb;
    const int64_t cost = waves(tiles, c) * (len + kWaveTokens);
    if (best == 0 || cost < best) {
      best = cost;
      p.chunk = len;
    }
  }
  p.chunks = static_cast<int>(for_any ? most_ranges(T, tiles) : (T + p.chunk - 1) / p.chunk);
  const int64_t round = kThreads / split_shape(N).g;  // tokens that a CTA splits at once
  p.split_rows = static_cast<int>(((T + kSplitCtas - 1) / kSplitCtas + round - 1) / round * round);
  p.split_ctas = static_cast<int>(for_any ? std::min<int64_t>((T + round - 1) / round, kSplitCtas)
                                          : (T + p.split_rows - 1) / p.split_rows);
  auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
  p.dl16_bytes = r256(static_cast<size_t>(2) * T * p.np * 2);
  p.dl_bytes = r256(static_cast<size_t>(3) * T * p.np * 2);
  p.w_bytes = r256(static_cast<size_t>(2) * N * d * 2);
  p.exp_bytes = r256(static_cast<size_t>(N) * 4) + r256(static_cast<size_t>(T) * 4);
  p.part_bytes = r256(static_cast<size_t>(p.chunks) * p.planes * N * d * 4);
  p.bias_bytes = r256(static_cast<size_t>(p.split_ctas) * N * 4);
  return p;
}

__device__ __forceinline__ uint16_t bf16_term(float& v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  v -= __bfloat162float(h);
  return __bfloat16_as_ushort(h);
}
__device__ __forceinline__ uint16_t fp16_term(float& v) {
  const __half h = __float2half_rn(v);
  v -= __half2float(h);
  return __half_as_ushort(h);
}
// e with |v| < 2^e, and 2^(e-1) <= |v| but for subnormal numbers and zero (-125).
__device__ __forceinline__ int exponent_of(float v) {
  return max(static_cast<int>(__float_as_uint(v) >> 23 & 0xffu), 1) - 126;
}
// v 2^s for a result below 2^15, in two factors: exact where the result is a normal number.
__device__ __forceinline__ float scale_by(float v, int s) {
  const int s1 = max(-126, min(127, s)), s2 = max(-126, min(127, s - s1));
  return v * __uint_as_float(static_cast<uint32_t>(s1 + 127) << 23) * __uint_as_float(static_cast<uint32_t>(s2 + 127) << 23);
}

// CTA n: row n of W_r as two fp16 terms [2][N][d], scaled by 2^(14 - b_n), and b_n.
__global__ void __launch_bounds__(kThreads) split_w_kernel(const float* __restrict__ w,
                                                           uint16_t* __restrict__ terms,
                                                           int32_t* __restrict__ w_exp, int N, int d) {
  __shared__ float s_max[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const float4* src = reinterpret_cast<const float4*>(w + static_cast<int64_t>(blockIdx.x) * d);
  float m = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < d / 4; i += kThreads) {
    const float4 v = __ldg(src + i);
    m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, s_max[i]);
  const int b = exponent_of(m);
  if (threadIdx.x == 0) w_exp[blockIdx.x] = b;
  uint16_t* out = terms + static_cast<int64_t>(blockIdx.x) * d;
  const int64_t plane = static_cast<int64_t>(N) * d;
#pragma unroll 4
  for (int i = threadIdx.x; i < d / 4; i += kThreads) {
    const float4 v4 = __ldg(src + i);
    float v[4] = {scale_by(v4.x, 14 - b), scale_by(v4.y, 14 - b), scale_by(v4.z, 14 - b), scale_by(v4.w, 14 - b)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint16_t t[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] = fp16_term(v[q]);
      *reinterpret_cast<uint2*>(out + k * plane + 4 * i) =
          make_uint2(t[0] | static_cast<uint32_t>(t[1]) << 16, t[2] | static_cast<uint32_t>(t[3]) << 16);
    }
  }
}

// G lanes a token, P pairs of values a lane (2 G P >= N): dL's row as two scaled fp16 terms [2][T][np]
// with a_t (for dx; w_exp null: left out) and as three bf16 terms [3][T][np] (for dW; dl_terms null: left
// out); the CTA's sums over its tokens for the bias. (A warp a token whatever N: the whole call 49 us and
// not 43 at T = 16384, N = 8, d = 1024; 34 and not 28 at d = 512.)
template <int G, int P>
__global__ void __launch_bounds__(kThreads) split_dl_kernel(
    const float* __restrict__ dl, const int32_t* __restrict__ w_exp, uint16_t* __restrict__ dl16,
    int32_t* __restrict__ row_exp, uint16_t* __restrict__ dl_terms, float* __restrict__ bias_part, int64_t T,
    int N, int np, int rows) {
  constexpr int kTokens = kThreads / G;  // of a round
  __shared__ float s_sum[kThreads / 32][2 * G * P];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * rows, t1 = min(T, t0 + rows);
  const int64_t plane = T * np;
  float acc[2 * P];
  int b[2 * P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    // values 2 j, 2 j + 1 of this lane: experts (j * G + gl) * 2 and the next
    const int n = (j * G + gl) * 2;
    acc[2 * j] = acc[2 * j + 1] = 0.f;
    b[2 * j] = w_exp != nullptr && n < N ? w_exp[n] : 0;
    b[2 * j + 1] = w_exp != nullptr && n + 1 < N ? w_exp[n + 1] : 0;
  }
  for (int64_t tb = t0; tb < t1; tb += kTokens) {
    const int64_t t = tb + threadIdx.x / G;
    const bool live = t < t1;
    float v[2 * P];
    int top = -1000;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int n = (j * G + gl) * 2;
      v[2 * j] = live && n < N ? dl[t * N + n] : 0.f;
      v[2 * j + 1] = live && n + 1 < N ? dl[t * N + n + 1] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) {
      acc[j] += v[j];
      if (v[j] != 0.f) top = max(top, exponent_of(v[j]) + b[j]);
    }
    if (w_exp != nullptr) {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
      if (gl == 0 && live) row_exp[t] = top;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int n = (j * G + gl) * 2;
        if (n >= np || !live) break;
        float x = scale_by(v[2 * j], 14 + b[2 * j] - top), y = scale_by(v[2 * j + 1], 14 + b[2 * j + 1] - top);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = fp16_term(x), hi = fp16_term(y);
          *reinterpret_cast<uint32_t*>(dl16 + k * plane + t * np + n) = lo | hi << 16;
        }
      }
    }
    if (dl_terms != nullptr) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int n = (j * G + gl) * 2;
        if (n >= np || !live) break;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t lo = bf16_term(v[2 * j]), hi = bf16_term(v[2 * j + 1]);
          *reinterpret_cast<uint32_t*>(dl_terms + k * plane + t * np + n) = lo | hi << 16;
        }
      }
    }
  }
  if (bias_part == nullptr) return;
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
  }
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) s_sum[warp][(j / 2 * G + gl) * 2 + j % 2] = acc[j];
  }
  __syncthreads();
  for (int n = threadIdx.x; n < N; n += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += s_sum[w][n];
    bias_part[static_cast<int64_t>(blockIdx.x) * N + n] = s;
  }
}

struct TcShared {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t done;
  uint32_t tmem;
  volatile int abort;
};

// Barriers and TMEM of a CTA; columns: a power of two.
__device__ __forceinline__ void tc_setup(TcShared& sh, int warp, uint32_t columns) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.tfull[i]), 1);
      mbar_init(smem_u32(&sh.tempty[i]), kTcThreads - 64);
    }
    mbar_init(smem_u32(&sh.done), 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), columns);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
}

// Weight gradient: one CTA for 256 columns of d, GROUP experts and one range of the tokens. A: the
// terms of dL [t][n], MN-major; B: x [t][c], MN-major; D[n][c] on 128 rows:
//   32 experts   rows 0-31 are the high terms' products, 32-63 the middle, 64-95 the low ones
//                (one MMA a k step; the fourth plane is zeros);
//   64 experts   rows 0-63 high and low, 64-127 middle (two MMAs: planes 0 and 1, planes 2 and zeros);
//   128 experts  all three terms in each row (three MMAs).
// What bounds it is shared memory's bandwidth to the tensor core, half of the usual for MN-major
// operands as measured: experts on the rows and 256 columns an MMA read 12 KB for 128 x 256 x 16
// products. (d on the rows, one MMA for each term, 128 columns of d and 128 experts: 160 us at T =
// 16384, N = 256, d = 7168; for 32 experts, d = 2880 29 us.)
// A stage's operands come in few, large copies: one for x (box [4][32 t][64 c]), one for the terms
// (two with 128 experts). Two chains in TMEM, 256 columns each. The range's sums, a plane for each
// group of rows, leave through shared memory: part [range][plane][N][d].
template <int GROUP>
__global__ void __launch_bounds__(kTcThreads, 1)
    router_wgrad_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dl,
                        const __grid_constant__ CUtensorMap tm_part, int64_t T, int N, int d, int c_tiles,
                        int n_tiles, int64_t chunk, int* status, uint64_t timeout_ns) {
  constexpr int kStages = w_stages(GROUP), kStageBytes = w_stage_bytes(GROUP), kABytes = w_a_bytes(GROUP);
  constexpr int kPlanes = GROUP == 32 ? 3 : GROUP == 64 ? 2 : 1;
  constexpr int kFlush = GROUP == 32 ? 24 : GROUP == 64 ? 12 : 8;  // stages of a chain: 48 steps
  constexpr int kMmas = GROUP == 32 ? 1 : GROUP == 64 ? 2 : 3;     // a k step
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  __shared__ TcShared sh;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  tc_setup(sh, warp, 512);
  pdl_wait();
  const uint32_t tmem = sh.tmem;
  // neighbouring CTAs share a range and columns of x
  const int n0 = static_cast<int>(blockIdx.x) % n_tiles * GROUP;
  const int c0 = static_cast<int>(blockIdx.x) / n_tiles % c_tiles * kWTile;
  const int range = static_cast<int>(blockIdx.x) / (n_tiles * c_tiles);
  const int64_t t0 = range * chunk, t1 = min(T, t0 + chunk);
  const int nkb = static_cast<int>((t1 - t0 + kKb - 1) / kKb);
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t last = l2_policy_evict_last();
      int it = 0;
      bool ok = true;
      for (; it < nkb; ++it) {
        const int s = it % kStages;
        if (!mbar_wait(smem_u32(&sh.empty[s]), ((it / kStages) & 1) ^ 1u, timeout_ns, &sh.abort)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&sh.full[s]);
        const uint32_t dst = base + s * kStageBytes;
        const int t = static_cast<int>(t0) + it * kKb;
        mbar_arrive_expect_tx(fb, kStageBytes);
        tma_load_3d(dst, &tm_dl, fb, n0, t, 0, last);
        if (GROUP == 128) tma_load_3d(dst + 3 * kBox, &tm_dl, fb, n0 + 64, t, 0, last);
        tma_load_3d(dst + kABytes, &tm_x, fb, 0, t, c0 / 64, last);
      }
      if (!ok) {
        sh.abort = 1;
        report_error(status, MOE_ERR_TIMEOUT);
      }
      for (int i = max(0, it - kStages); i < it; ++i)  // no copy is still landing when the CTA exits
        mbar_wait(smem_u32(&sh.full[i % kStages]), (i / kStages) & 1, kDrainTimeoutNs, nullptr);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, kWTile) | (1u << 15) | (1u << 16);
    bool ok = true, issued = false;
    for (int it = 0; it < nkb; ++it) {
      const int s = it % kStages, u = it / kFlush;
      if (it % kFlush == 0) {
        const bool free_buf = mbar_wait(smem_u32(&sh.tempty[u & 1]), ((u >> 1) & 1) ^ 1u, timeout_ns, &sh.abort);
        if (!__all_sync(kFull, free_buf)) {
          ok = false;
          break;
        }
      }
      const bool got = mbar_wait(smem_u32(&sh.full[s]), (it / kStages) & 1, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t st = base + s * kStageBytes;
      const uint64_t a = GROUP == 32 ? desc_mn32(st) : GROUP == 64 ? desc_mn(st, kBox) : desc_mn(st, 3 * kBox);
      const uint64_t b = desc_mn(st + kABytes, kBox);
      const bool add = it % kFlush > 0;
#pragma unroll
      for (int kk = 0; kk < kKb / 16; ++kk)
#pragma unroll
        for (int k = 0; k < kMmas; ++k)  // address offsets in the descriptors, in 16-byte units
          if (elect_one())
            tc_mma_f16(tmem + (u & 1) * kWTile,
                       a + ((k * (GROUP == 64 ? 2 : 1) * kBox + kk * (GROUP == 32 ? 1024 : 2048)) >> 4),
                       b + ((kk * 2048) >> 4), idesc, kk > 0 || k > 0 ? 1u : add);
      if (elect_one()) {
        tc_commit(smem_u32(&sh.empty[s]));
        if (it % kFlush == kFlush - 1 || it == nkb - 1) tc_commit(smem_u32(&sh.tfull[u & 1]));
      }
      issued = true;
      __syncwarp();
    }
    if (!ok && lane == 0) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    }
    if (issued && elect_one()) {  // every MMA has finished before the TMEM is freed
      tc_commit(smem_u32(&sh.done));
      mbar_wait(smem_u32(&sh.done), 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    const int q = warp & 3;            // TMEM lane quadrant
    const int half = (warp - 2) >> 2;  // columns [half * 128, half * 128 + 128) of the tile
    const int plane = GROUP == 32 ? q : GROUP == 64 ? q >> 1 : 0;
    const int n = n0 + (GROUP == 32 ? 0 : GROUP == 64 ? (q & 1) * 32 : q * 32);  // expert of lane 0
    const int c = c0 + half * 128;
    const bool mine = plane < kPlanes && n < N && c < d;
    float acc[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0.f;
    const uint32_t row = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    bool ok = true;
    for (int u = 0; u * kFlush < nkb; ++u) {
      const bool got = mbar_wait(smem_u32(&sh.tfull[u & 1]), (u >> 1) & 1, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (mine) {
#pragma unroll
        for (int j = 0; j < 128; j += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(row + (u & 1) * kWTile + j, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j + i] += __uint_as_float(v[i]);
        }
      }
      tc_fence_before_sync();
      mbar_arrive(smem_u32(&sh.tempty[u & 1]));
    }
    if (!ok) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    } else if (mine) {
      // the last chain's barrier: every MMA is done, so the stages are free for the blocks that leave
      const uint32_t stage = base + (warp - 2) * (32 * 32 * 4);
      uint8_t* const stg = dyn_smem + (stage - smem_u32(dyn_smem));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + 32 * j < d) {
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_float4(
                acc[32 * j + 4 * i], acc[32 * j + 4 * i + 1], acc[32 * j + 4 * i + 2], acc[32 * j + 4 * i + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {  // experts past N are not written
            tma_store_3d(&tm_part, stage, c + 32 * j, n, range * kPlanes + plane);
            tma_store_commit();
          }
        }
      }
      if (lane == 0) tma_store_wait_all();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// dx: persistent CTAs over tiles of 128 tokens x 256 columns of d. A: dL's terms [t][n], K-major; B:
// W_r's terms [n][c], MN-major; three products a k step into D[t][c]; two accumulators, so one
// tile's epilogue runs beside the next one's MMAs. A lane holds a token, so scaling back is one
// factor a lane; 32 x 32 blocks go through shared memory to TMA stores. Accumulating is the same
// store as a reduction: the L2 adds (one addition an element, so the order is fixed) and no SM
// waits for the old values, which are called to the L2 a tile ahead (T = 16384, dL's and W_r's
// terms included: N = 32, d = 2880 86 us, 102 without; N = 256, d = 7168 221 and 235). (Lanes along
// c, and 128-byte reductions from registers: 299 us for the latter, bound by their issue.)
constexpr int kXStages = 3;
constexpr int kXStageBytes = 2 * kXTileT * kKb * 2 + 2 * (kXTileC / 64) * kBox;
constexpr int kXStaging = 32 * 32 * 4;  // one block; two for each epilogue warp
constexpr int kXSmem = kXStages * kXStageBytes + 16 * kXStaging + 1024;
static_assert(kXSmem <= kTcMaxSmem, "shared memory");

__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__global__ void __launch_bounds__(kTcThreads, 1)
    router_dgrad_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_dl,
                        const __grid_constant__ CUtensorMap tm_out, const float* out,
                        const int32_t* __restrict__ row_exp, int64_t T, int N, int d, int c_tiles, int64_t tiles,
                        int accumulate, int* status, uint64_t timeout_ns) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  __shared__ TcShared sh;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  constexpr int kABytes = kXTileT * kKb * 2, kBBytes = kXTileC / 64 * kBox;  // one term
  tc_setup(sh, warp, 512);
  pdl_wait();
  const uint32_t tmem = sh.tmem;
  const int nkb = (N + kKb - 1) / kKb;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t last = l2_policy_evict_last();
      int it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int c0 = static_cast<int>(t % c_tiles) * kXTileC;
        const int r0 = static_cast<int>(t / c_tiles) * kXTileT;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kXStages;
          if (!mbar_wait(smem_u32(&sh.empty[s]), ((it / kXStages) & 1) ^ 1u, timeout_ns, &sh.abort)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&sh.full[s]);
          const uint32_t a = base + s * kXStageBytes, b = a + 2 * kABytes;
          mbar_arrive_expect_tx(fb, kXStageBytes);
          tma_load_3d(a, &tm_dl, fb, kb * kKb, r0, 0, last);
          tma_load_4d(b, &tm_w, fb, 0, kb * kKb, c0 / 64, 0, last);
        }
      }
      if (!ok) {
        sh.abort = 1;
        report_error(status, MOE_ERR_TIMEOUT);
      }
      for (int i = max(0, it - kXStages); i < it; ++i)
        mbar_wait(smem_u32(&sh.full[i % kXStages]), (i / kXStages) & 1, kDrainTimeoutNs, nullptr);
    }
  } else if (warp == 1) {
    // fp16 operands (formats 0), A K-major, B MN-major
    constexpr uint32_t idesc = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(kXTileC >> 3) << 17) |
                               (static_cast<uint32_t>(kXTileT >> 4) << 24);
    bool ok = true, issued = false;
    int it = 0, uc = 0;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++uc) {
      const int buf = uc & 1;
      const bool free_buf = mbar_wait(smem_u32(&sh.tempty[buf]), ((uc >> 1) & 1) ^ 1u, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, free_buf)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int s = it % kXStages;
        const bool got = mbar_wait(smem_u32(&sh.full[s]), (it / kXStages) & 1, timeout_ns, &sh.abort);
        if (!__all_sync(kFull, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t a = desc_k64(base + s * kXStageBytes), b = desc_mn(base + s * kXStageBytes + 2 * kABytes, kBox);
        const int steps = (N - kb * kKb + 15) / 16;
#pragma unroll
        for (int kk = 0; kk < kKb / 16; ++kk) {
          if (kk < steps) {
#pragma unroll
            for (int k = 0; k < 3; ++k)  // terms (0, 0), (0, 1), (1, 0)
              if (elect_one())
                tc_mma_f16(tmem + buf * kXTileC, a + (((k == 2 ? kABytes : 0) + kk * 32) >> 4),
                           b + (((k == 1 ? kBBytes : 0) + kk * 2048) >> 4), idesc, kk > 0 || k > 0 ? 1u : kb > 0);
          }
        }
        if (elect_one()) tc_commit(smem_u32(&sh.empty[s]));
        issued = true;
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) tc_commit(smem_u32(&sh.tfull[buf]));
    }
    if (!ok && lane == 0) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    }
    if (issued && elect_one()) {
      tc_commit(smem_u32(&sh.done));
      mbar_wait(smem_u32(&sh.done), 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    const int q = warp & 3;            // TMEM lane quadrant: tokens q * 32 .. of the tile
    const int half = (warp - 2) >> 2;  // columns [half * 128, half * 128 + 128) of the tile
    const uint32_t stage0 = base + kXStages * kXStageBytes + (warp - 2) * 2 * kXStaging;
    // old values of this warp's part of a tile, one row a lane, to the L2
    auto ahead = [&](int64_t t) {
      if (!accumulate || t >= tiles) return;
      const int64_t r0 = t / c_tiles * kXTileT + q * 32;
      const int c0 = static_cast<int>(t % c_tiles) * kXTileC + half * 128;
      if (c0 < d && r0 + lane < T) l2_prefetch(out + (r0 + lane) * d + c0, min(128, d - c0) * 4);
    };
    ahead(blockIdx.x);
    int uc = 0, n = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++uc) {
      const int buf = uc & 1;
      const int64_t r0 = t / c_tiles * kXTileT + q * 32;
      const int c0 = static_cast<int>(t % c_tiles) * kXTileC + half * 128;
      const int e = r0 + lane < T ? row_exp[r0 + lane] : 0;
      ahead(t + gridDim.x);
      // 2^(a_t - 28) in two factors, the second 1 but for tokens below 2^-98
      const float f = scalbnf(1.0f, min(127, max(-126, e - 28)));
      const float f2 = scalbnf(1.0f, max(-149, min(0, e - 28 + 126)));
      const bool tiny = __any_sync(kFull, f2 != 1.0f);
      const bool got = mbar_wait(smem_u32(&sh.tfull[buf]), (uc >> 1) & 1, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, got)) {
        sh.abort = 1;
        report_error(status, MOE_ERR_TIMEOUT);
        break;
      }
      tc_fence_after_sync();
      const uint32_t row = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kXTileC + half * 128;
#pragma unroll 1
      for (int cc = 0; cc < 128 && c0 + cc < d && r0 < T; cc += 32, ++n) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(row + cc, v);
        tmem_ld_wait();
        const uint32_t stage = stage0 + (n & 1) * kXStaging;
        uint8_t* const stg = dyn_smem + (stage - smem_u32(dyn_smem));
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the block before the last
        __syncwarp();
        float r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(v[i]) * f;
        if (tiny) {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] *= f2;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        fence_proxy_async_smem();  // generic stores -> visible to the TMA engine
        __syncwarp();
        if (lane == 0) {  // rows past T and columns past d are not written
          if (accumulate) tma_reduce_add_2d(&tm_out, stage, c0 + cc, static_cast<int>(r0));
          else tma_store_2d(&tm_out, stage, c0 + cc, static_cast<int>(r0));
          tma_store_commit();
        }
      }
      tc_fence_before_sync();
      mbar_arrive(smem_u32(&sh.tempty[buf]));
    }
    if (lane == 0) tma_store_wait_all();  // every store of this warp has landed
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor cores where the products are worth the five launches, from T N d = 2^26 on. Device time
// of the two paths, CUDA cores first, us, at (T, d, N): (256, 1024, 64) 11.3, 18.3; (512, 2880, 32) 15.9,
// 19.5; (1024, 1024, 64) 18.1, 20.1; (16384, 512, 8) 27.6, 27.9; (64, 4096, 256) 26.5, 22.6; (4096, 512, 64)
// 30.2, 22.8; (4096, 2880, 32) 69, 32; (1024, 4096, 128) 83, 24. At the threshold itself either may be
// ahead, by 2 us at most of those measured. Below 64 tokens a row block of the MMA is half empty.
constexpr int64_t kTcMinTokens = 64, kTcMinProducts = 1 << 26;
bool use_tensor_cores(int64_t T, int N, int d) { return T >= kTcMinTokens && static_cast<double>(T) * N * d >= kTcMinProducts; }

template <int GROUP>
cudaError_t launch_wgrad(const CUtensorMap& mx, const CUtensorMap& mdl, const CUtensorMap& mp,
                         const RouterBackwardArgs& a, const TcPlan& p, cudaStream_t s) {
  constexpr int smem = std::max(kTcMinSmem, w_stages(GROUP) * w_stage_bytes(GROUP) + 1024);
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(router_wgrad_kernel<GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(router_wgrad_kernel<GROUP>, dim3(p.n_tiles * p.c_tiles * p.chunks), dim3(kTcThreads), smem, s,
                    mx, mdl, mp, static_cast<int64_t>(a.T), a.N, a.d, p.c_tiles, p.n_tiles, p.chunk, a.status,
                    a.timeout_ns);
}

cudaError_t launch_tc(const RouterBackwardArgs& a, cudaStream_t s) {
  const TcPlan p = make_tc_plan(a.T, a.N, a.d);
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  char* ws = static_cast<char*>(a.scratch);
  auto take = [&ws](size_t bytes) {
    char* r = ws;
    ws += bytes;
    return r;
  };
  uint16_t* dl16 = reinterpret_cast<uint16_t*>(take(p.dl16_bytes));
  uint16_t* dl_terms = reinterpret_cast<uint16_t*>(take(p.dl_bytes));
  uint16_t* w_terms = reinterpret_cast<uint16_t*>(take(p.w_bytes));
  int32_t* row_exp = reinterpret_cast<int32_t*>(take(p.exp_bytes));  // [T], then [N]
  int32_t* w_exp = row_exp + (static_cast<int64_t>(a.T) + 63) / 64 * 64;
  float* part = reinterpret_cast<float*>(take(p.part_bytes));
  float* bias_part = reinterpret_cast<float*>(take(p.bias_bytes));
  const uint64_t T = static_cast<uint64_t>(a.T), d = static_cast<uint64_t>(a.d), np = static_cast<uint64_t>(p.np);
  const bool want_x = a.d_x != nullptr, want_w = a.d_w_router != nullptr, want_b = a.d_logit_bias != nullptr;
  if (want_x) {
    e = launch_pdl(split_w_kernel, dim3(a.N), dim3(kThreads), 0, s, a.w_router, w_terms, w_exp, a.N, a.d);
    if (e != cudaSuccess) return e;
  }
  const SplitShape ss = split_shape(a.N);
  auto* split = ss.g == 4 ? split_dl_kernel<4, 1> : ss.g == 8 ? split_dl_kernel<8, 1>
              : ss.g == 16 ? split_dl_kernel<16, 1> : ss.p == 1 ? split_dl_kernel<32, 1>
              : ss.p == 2 ? split_dl_kernel<32, 2> : split_dl_kernel<32, 4>;
  e = launch_pdl(split, dim3(p.split_ctas), dim3(kThreads), 0, s, a.d_logits,
                 want_x ? static_cast<const int32_t*>(w_exp) : nullptr, dl16, row_exp, want_w ? dl_terms : nullptr,
                 want_b ? bias_part : nullptr, static_cast<int64_t>(a.T), a.N, p.np, p.split_rows);
  if (e != cudaSuccess) return e;
  if (want_w) {
    CUtensorMap mx, mdl, mp;
    // x as [d / 64][T][64]
    const uint64_t xd[3] = {64, T, d / 64}, xs[2] = {d * 2, 128}, ld[3] = {np, T, 3}, ls[2] = {np * 2, T * np * 2};
    const uint64_t pd[3] = {d, static_cast<uint64_t>(a.N), static_cast<uint64_t>(p.chunks * p.planes)};
    const uint64_t ps[2] = {d * 4, static_cast<uint64_t>(a.N) * d * 4};
    const uint32_t xb[3] = {64, kKb, kWTile / 64}, pb[3] = {32, 32, 1};
    // past the third term, and past N: zeros
    const uint32_t lb[3] = {p.group == 32 ? 32u : 64u, kKb, p.group == 128 ? 3u : 4u};
    if (!make_map(&mx, a.x, 3, xd, xs, xb) ||
        !make_map(&mdl, dl_terms, 3, ld, ls, lb,
                  p.group == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_f32(&mp, part, 3, pd, ps, pb))
      return cudaErrorInvalidValue;
    e = p.group == 32   ? launch_wgrad<32>(mx, mdl, mp, a, p, s)
        : p.group == 64 ? launch_wgrad<64>(mx, mdl, mp, a, p, s)
                        : launch_wgrad<128>(mx, mdl, mp, a, p, s);
    if (e != cudaSuccess) return e;
  }
  if (want_x) {
    CUtensorMap mw, mdl, mo;
    const uint64_t od[2] = {d, T}, os[1] = {d * 4};
    const uint32_t ob[2] = {32, 32};
    // W_r's terms as [2][d / 64][N][64]
    const uint64_t wd[4] = {64, static_cast<uint64_t>(a.N), d / 64, 2};
    const uint64_t wst[3] = {d * 2, 128, static_cast<uint64_t>(a.N) * d * 2};
    const uint64_t ld[3] = {np, T, 2}, ls[2] = {np * 2, T * np * 2};
    const uint32_t wb[4] = {64, kKb, kXTileC / 64, 2}, lb[3] = {kKb, kXTileT, 2};
    // 16-bit elements either way: the copy does not look at the format
    if (!make_map(&mw, w_terms, 4, wd, wst, wb) ||
        !make_map(&mdl, dl16, 3, ld, ls, lb, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map_f32(&mo, a.d_x, 2, od, os, ob))
      return cudaErrorInvalidValue;
    static PerDeviceOnce once;
    e = once.run([] {
      return cudaFuncSetAttribute(router_dgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmem);
    });
    if (e != cudaSuccess) return e;
    const int c_tiles = (a.d + kXTileC - 1) / kXTileC;
    const int64_t tiles = c_tiles * ((static_cast<int64_t>(a.T) + kXTileT - 1) / kXTileT);
    const int grid = static_cast<int>(std::min<int64_t>(tiles, di.sm_count));
    e = launch_pdl(router_dgrad_kernel, dim3(grid), dim3(kTcThreads), kXSmem, s, mw, mdl, mo,
                   static_cast<const float*>(a.d_x), static_cast<const int32_t*>(row_exp),
                   static_cast<int64_t>(a.T), a.N, a.d, c_tiles, tiles, a.accumulate, a.status, a.timeout_ns);
    if (e != cudaSuccess) return e;
  }
  if (!want_w && !want_b) return cudaSuccess;
  return launch_sum(part, bias_part, a, p.chunks * p.planes, p.split_ctas, s);
}

}  // namespace

size_t router_backward_scratch_bytes(int64_t T, int N, int d) {
  if (use_tensor_cores(T, N, d)) return make_tc_plan(T, N, d).total();
  const Plan p = make_plan(T, N, d);
  return p.chunks > 1 ? static_cast<size_t>(p.chunks) * N * (d + 1) * sizeof(float) : 0;
}

size_t router_backward_scratch_bytes_up_to(int64_t T, int N, int d) {
  // the longest batch of these that takes the CUDA cores (see use_tensor_cores), then the tensor cores
  const int64_t longest = std::max<int64_t>(kTcMinTokens, (kTcMinProducts - 1) / (static_cast<int64_t>(N) * d) + 1) - 1;
  const Plan p = make_plan(std::min(T, longest), N, d);
  const size_t cores = p.most_chunks > 1 ? static_cast<size_t>(p.most_chunks) * N * (d + 1) * sizeof(float) : 0;
  return T > longest ? std::max(cores, make_tc_plan(T, N, d, true).total()) : cores;
}

cudaError_t launch_router_backward(const RouterBackwardArgs& a, cudaStream_t s) {
  if (use_tensor_cores(a.T, a.N, a.d)) return launch_tc(a, s);
  const Plan pl = make_plan(a.T, a.N, a.d);
  Params p{};
  p.x = a.x;
  p.w = a.w_router;
  p.dl = a.d_logits;
  p.d_x = a.d_x;
  p.d_w = a.d_w_router;
  p.d_b = a.d_logit_bias;
  p.part_w = static_cast<float*>(a.scratch);
  p.part_b = p.part_w + static_cast<int64_t>(pl.chunks) * a.N * a.d;
  p.T = a.T;
  p.N = a.N;
  p.d = a.d;
  p.accumulate = a.accumulate;
  p.w_cols = pl.w_cols;
  p.w_experts = pl.w_experts;
  p.chunks = pl.chunks;
  p.x_cols = pl.x_cols;
  p.chunk = pl.chunk;
  const bool want_w = a.d_w_router != nullptr || a.d_logit_bias != nullptr;
  p.w_ctas = want_w ? static_cast<int64_t>(pl.w_cols) * pl.w_experts * pl.chunks : 0;
  const int64_t x_ctas = a.d_x != nullptr ? pl.x_tokens * pl.x_cols : 0;
  if (p.w_ctas + x_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (p.w_ctas + x_ctas == 0) return cudaSuccess;
  cudaError_t e = launch_pdl(router_backward_kernel, dim3(static_cast<unsigned>(p.w_ctas + x_ctas)),
                             dim3(kThreads), 0, s, p);
  if (e != cudaSuccess || !want_w || pl.chunks == 1) return e;
  return launch_sum(p.part_w, p.part_b, a, pl.chunks, pl.chunks, s);
}

}  // namespace moe
