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

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWExperts = 16, kWCols = 128, kWTokens = 32;
constexpr int kXTokens = 16, kXCols = 256, kXExperts = 64;

struct Plan {
  int w_cols, w_experts, chunks;  // grid of the W CTAs
  int64_t chunk;                  // tokens of a range
  int x_cols;
  int64_t x_tokens;               // grid of the x CTAs
};

Plan make_plan(int64_t T, int N, int d) {
  Plan p{};
  p.w_cols = (d + kWCols - 1) / kWCols;
  p.w_experts = (N + kWExperts - 1) / kWExperts;
  const int64_t tiles = static_cast<int64_t>(p.w_cols) * p.w_experts;
  const int64_t most = (T + 4 * kWTokens - 1) / (4 * kWTokens);  // ranges of at least 128 tokens
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>({most, 2 * 148 / tiles, 64}));
  p.chunk = (T + chunks - 1) / chunks;
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
  for (int64_t tb = t0; tb < t1; tb += kWTokens) {
    __syncthreads();
    for (int i = threadIdx.x; i < kWTokens * (kWCols / 2); i += kThreads) {
      const int64_t t = tb + i / (kWCols / 2);
      const int c = c0 + i % (kWCols / 2) * 2;
      s_x[i / (kWCols / 2)][i % (kWCols / 2)] =
          t < t1 && c < a.d ? *reinterpret_cast<const uint32_t*>(a.x + t * a.d + c) : 0u;
    }
    for (int i = threadIdx.x; i < kWTokens * kWExperts; i += kThreads) {
      const int64_t t = tb + i / kWExperts;
      const int n = n0 + i % kWExperts;
      s_dl[i / kWExperts][i % kWExperts] = t < t1 && n < a.N ? a.dl[t * a.N + n] : 0.f;
    }
    __syncthreads();
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
#pragma unroll 4
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
  __shared__ uint32_t s_x[kWTokens][kWCols / 2];
  __shared__ float s_w[kWTokens][kWExperts];
  __shared__ float s_dl[kXTokens][kXExperts];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x < a.w_ctas) w_tile(a, s_x, s_w);
  else x_tile(a, s_dl);
}

// The token ranges' partial sums, added in order.
__global__ void __launch_bounds__(256) router_backward_sum_kernel(
    const float* __restrict__ part_w, const float* __restrict__ part_b, float* __restrict__ d_w,
    float* __restrict__ d_b, int chunks, int N, int d, int accumulate) {
  pdl_trigger();
  pdl_wait();
  const int64_t items = static_cast<int64_t>(N) * d / 4;
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (d_w != nullptr && i < items) {
    float4 s = accumulate ? reinterpret_cast<const float4*>(d_w)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
      const float4 v = reinterpret_cast<const float4*>(part_w)[c * items + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<float4*>(d_w)[i] = s;
  }
  if (d_b != nullptr && i < N) {
    float s = accumulate ? d_b[i] : 0.f;
    for (int c = 0; c < chunks; ++c) s += part_b[static_cast<int64_t>(c) * N + i];
    d_b[i] = s;
  }
}

}  // namespace

size_t router_backward_scratch_bytes(int64_t T, int N, int d) {
  const Plan p = make_plan(T, N, d);
  return p.chunks > 1 ? static_cast<size_t>(p.chunks) * N * (d + 1) * sizeof(float) : 0;
}

cudaError_t launch_router_backward(const RouterBackwardArgs& a, cudaStream_t s) {
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
  const int64_t items = std::max<int64_t>(static_cast<int64_t>(a.N) * a.d / 4, a.N);
  return launch_pdl(router_backward_sum_kernel, dim3(static_cast<unsigned>((items + 255) / 256)),
                    dim3(256), 0, s, static_cast<const float*>(p.part_w),
                    static_cast<const float*>(p.part_b), a.d_w_router, a.d_logit_bias, pl.chunks, a.N,
                    a.d, a.accumulate);
}

}  // namespace moe
