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
#include "tma_host.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr double kTcWork = 33554432.0;
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
    float* __restrict__ d_b, int chunks, int b_parts, int N, int d, int accumulate) {
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
#pragma unroll 8
    for (int c = 0; c < b_parts; ++c) s += part_b[static_cast<int64_t>(c) * N + i];
    d_b[i] = s;
  }
}

// ------------------------------------------------------------------ tensor-core path
// An fp32 number is the sum of three bf16 terms (8 significant bits each). dL^T x with x exact in
// bf16 takes three products; dL W_r takes the six whose size reaches 2^-16 of the leading one
// (those left out are below 2^-24). The terms are written once, by split_kernel, and both GEMMs
// put the axis d on the 128 rows of the MMA: the accumulator's lanes then run along the
// contiguous axis of the outputs, and a warp's 32 lanes store 128 consecutive bytes straight
// from registers.
constexpr int kKb = 32;           // reduction elements of a stage
constexpr int kBox = 64 * kKb * 2;  // one TMA box of an MN-major operand: 64 MN x 32 k, 128B-swizzled
constexpr int kTcThreads = 320;   // TMA producer, MMA issuer, eight epilogue warps
constexpr int kTcMinSmem = 120 * 1024;  // one CTA an SM: the TMEM is not shared
constexpr int kTcMaxSmem = 227 * 1024;
constexpr int kWTile = 256;       // columns of d a CTA of the weight gradient owns (two MMA row blocks)
constexpr int kXTileC = 128, kXTileT = 256;

// Shared-memory descriptor of an MN-major operand of kKb k rows: groups of 8 k rows are 1024 bytes
// (stride offset), blocks of 64 MN elements one box (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kBox >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// K-major operand with 64-byte rows (32 bf16, 64B-swizzled): groups of 8 rows are 512 bytes.
__device__ __forceinline__ uint64_t desc_k64(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) |
         (static_cast<uint64_t>(512u >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

struct TcPlan {
  int np;       // N rounded up to 8: row length of the terms of dL
  int nu;       // N rounded up to 16: MMA columns of the weight gradient
  int n_boxes;  // boxes of 64 experts
  int c_tiles, chunks;
  int64_t chunk;  // tokens of a range of the weight gradient, a multiple of kKb
  int w_stages, w_stage_bytes;
  int split_rows, split_ctas;  // tokens a CTA of split_kernel takes, and how many such CTAs
  size_t dl_bytes, w_bytes, part_bytes, bias_bytes;
};

TcPlan make_tc_plan(int64_t T, int N, int d) {
  TcPlan p{};
  p.np = (N + 7) / 8 * 8;
  p.nu = (N + 15) / 16 * 16;
  p.n_boxes = (N + 63) / 64;
  p.c_tiles = (d + kWTile - 1) / kWTile;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>(148 / p.c_tiles, T / 128));
  p.chunk = ((T + chunks - 1) / chunks + kKb - 1) / kKb * kKb;
  p.chunks = static_cast<int>((T + p.chunk - 1) / p.chunk);
  p.w_stage_bytes = (kWTile / 64 + 3 * p.n_boxes) * kBox;
  p.w_stages = std::min(8, (kTcMaxSmem - 2048) / p.w_stage_bytes);
  p.split_rows = static_cast<int>(std::max<int64_t>(8, (T + 295) / 296));
  p.split_ctas = static_cast<int>((T + p.split_rows - 1) / p.split_rows);
  auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
  p.dl_bytes = r256(static_cast<size_t>(3) * T * p.np * 2);
  p.w_bytes = r256(static_cast<size_t>(3) * N * d * 2);
  p.part_bytes = r256(static_cast<size_t>(p.chunks) * N * d * 4);
  p.bias_bytes = r256(static_cast<size_t>(p.split_ctas) * N * 4);
  return p;
}

__device__ __forceinline__ void split3(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(h);
  const __nv_bfloat16 m = __float2bfloat16_rn(r);
  const __nv_bfloat16 l = __float2bfloat16_rn(r - __bfloat162float(m));
  hi = __bfloat16_as_ushort(h);
  mid = __bfloat16_as_ushort(m);
  lo = __bfloat16_as_ushort(l);
}

// CTAs [0, split_ctas): dL's terms [3][T][np] and the bias gradient's partial sums of their tokens;
// the others: W_r's terms [3][N][d].
__global__ void __launch_bounds__(kThreads) split_kernel(const float* __restrict__ dl,
                                                         const float* __restrict__ w,
                                                         uint16_t* __restrict__ dl_terms,
                                                         uint16_t* __restrict__ w_terms,
                                                         float* __restrict__ bias_part, int64_t T,
                                                         int N, int np, int64_t w_items, int rows,
                                                         int dl_ctas) {
  pdl_trigger();
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= dl_ctas) {
    const int64_t plane = w_items;
    for (int64_t i = ((blockIdx.x - dl_ctas) * static_cast<int64_t>(kThreads) + threadIdx.x) * 4; i < w_items;
         i += static_cast<int64_t>(gridDim.x - dl_ctas) * kThreads * 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + i));
      const float f[4] = {v.x, v.y, v.z, v.w};
      uint16_t t[3][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) split3(f[q], t[0][q], t[1][q], t[2][q]);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2*>(w_terms + k * plane + i) =
            make_uint2(t[k][0] | static_cast<uint32_t>(t[k][1]) << 16, t[k][2] | static_cast<uint32_t>(t[k][3]) << 16);
    }
    return;
  }
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * rows;
  const int n_rows = static_cast<int>(min(static_cast<int64_t>(rows), T - t0));
  const int64_t plane = T * np;
  const int pairs = np / 2;
  for (int i = threadIdx.x; i < n_rows * pairs; i += kThreads) {
    const int r = i / pairs, n = i % pairs * 2;
    const float* src = dl + (t0 + r) * N + n;
    const float a = n < N ? src[0] : 0.f, b = n + 1 < N ? src[1] : 0.f;
    uint16_t ta[3], tb[3];
    split3(a, ta[0], ta[1], ta[2]);
    split3(b, tb[0], tb[1], tb[2]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint32_t*>(dl_terms + k * plane + (t0 + r) * np + n) =
          ta[k] | static_cast<uint32_t>(tb[k]) << 16;
  }
  if (bias_part != nullptr) {
    for (int n = threadIdx.x; n < N; n += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int r = 0; r < n_rows; ++r) s += dl[(t0 + r) * N + n];
      bias_part[static_cast<int64_t>(blockIdx.x) * N + n] = s;
    }
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
__device__ __forceinline__ void tc_setup(TcShared& sh, int warp, uint32_t columns, int epilogue_threads) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.tfull[i]), 1);
      mbar_init(smem_u32(&sh.tempty[i]), epilogue_threads);
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

// Weight gradient: one CTA for 256 columns of d and one range of the tokens. A: x [t][c], MN-major,
// two row blocks of 128 columns; B: the terms of dL [t][n], MN-major; D[c][n] in TMEM, columns
// [0, nu) and [nu, 2 nu). The sum over the range goes to part [chunk][N][d].
__global__ void __launch_bounds__(kTcThreads, 1)
    router_wgrad_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dl,
                        float* __restrict__ part, int64_t T, int N, int d, int nu, int n_boxes, int c_tiles,
                        int64_t chunk, int stages, uint32_t columns, int* status, uint64_t timeout_ns) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  __shared__ TcShared sh;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  tc_setup(sh, warp, columns, kTcThreads - 64);
  pdl_wait();
  const uint32_t tmem = sh.tmem;
  const int c0 = static_cast<int>(blockIdx.x) % c_tiles * kWTile;
  const int range = static_cast<int>(blockIdx.x) / c_tiles;
  const int64_t t0 = range * chunk, t1 = min(T, t0 + chunk);
  const int nkb = static_cast<int>((t1 - t0 + kKb - 1) / kKb);
  const int a_boxes = min(kWTile / 64, (d - c0) / 64);  // d is a multiple of 64
  const int stage_bytes = (kWTile / 64 + 3 * n_boxes) * kBox;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
      int it = 0;
      bool ok = true;
      for (; it < nkb; ++it) {
        const int s = it % stages;
        if (!mbar_wait(smem_u32(&sh.empty[s]), ((it / stages) & 1) ^ 1u, timeout_ns, &sh.abort)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&sh.full[s]);
        const uint32_t dst = base + s * stage_bytes, b_dst = dst + kWTile / 64 * kBox;
        const int t = static_cast<int>(t0) + it * kKb;
        mbar_arrive_expect_tx(fb, (a_boxes + 3 * n_boxes) * kBox);
        for (int i = 0; i < a_boxes; ++i) tma_load_2d(dst + i * kBox, &tm_x, fb, c0 + 64 * i, t, first);
        for (int k = 0; k < 3; ++k)
          for (int i = 0; i < n_boxes; ++i)
            tma_load_3d(b_dst + (k * n_boxes + i) * kBox, &tm_dl, fb, 64 * i, t, k, last);
      }
      if (!ok) {
        sh.abort = 1;
        report_error(status, MOE_ERR_TIMEOUT);
      }
      for (int i = max(0, it - stages); i < it; ++i)  // no copy is still landing when the CTA exits
        mbar_wait(smem_u32(&sh.full[i % stages]), (i / stages) & 1, kDrainTimeoutNs, nullptr);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(128, nu) | (1u << 15) | (1u << 16);
    const int blocks = (a_boxes + 1) / 2;  // row blocks of 128 columns
    bool ok = true, issued = false;
    for (int it = 0; it < nkb; ++it) {
      const int s = it % stages;
      const bool got = mbar_wait(smem_u32(&sh.full[s]), (it / stages) & 1, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (lane == 0) {
        const uint32_t a = base + s * stage_bytes, b = a + kWTile / 64 * kBox;
        for (int m = 0; m < blocks; ++m)
          for (int kk = 0; kk < kKb / 16; ++kk)
#pragma unroll
            for (int k = 0; k < 3; ++k)
              tc_mma_f16(tmem + m * nu, desc_mn(a + 2 * m * kBox + kk * 2048),
                         desc_mn(b + k * n_boxes * kBox + kk * 2048), idesc, it > 0 || kk > 0 || k > 0);
        tc_commit(smem_u32(&sh.empty[s]));
      }
      issued = true;
      __syncwarp();
    }
    if (ok && lane == 0) tc_commit(smem_u32(&sh.tfull[0]));
    if (!ok && lane == 0) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    }
    if (issued && lane == 0) {  // every MMA has finished before the TMEM is freed
      tc_commit(smem_u32(&sh.done));
      mbar_wait(smem_u32(&sh.done), 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    const int q = warp & 3;           // TMEM lane quadrant
    const int m = (warp - 2) >> 2;    // row block
    const int c = c0 + m * 128 + q * 32;  // the warp's first column of d; 32-column groups are whole
    const bool got = mbar_wait(smem_u32(&sh.tfull[0]), 0, timeout_ns, &sh.abort);
    if (!__all_sync(kFull, got)) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    } else if (c < d) {
      tc_fence_after_sync();
      float* out = part + static_cast<int64_t>(range) * N * d + c + lane;
      const uint32_t row = tmem + (static_cast<uint32_t>(q * 32) << 16) + m * nu;
      for (int n = 0; n < nu; n += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(row + n, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (n + i < N) out[static_cast<int64_t>(n + i) * d] = __uint_as_float(v[i]);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, columns);
  }
}

// dx: persistent CTAs over tiles of 128 columns of d x 256 tokens. A: W_r's terms [n][c], MN-major;
// B: dL's terms [t][n], K-major; six products a k step into D[c][t]; two accumulators, so one
// tile's epilogue runs beside the next one's MMAs. Accumulating adds in the L2 (a reduction
// without a return: one addition an element, so the order is fixed, and no SM waits for the old
// values).
constexpr int kXStages = 3;
constexpr int kXStageBytes = 3 * 2 * kBox + 3 * kXTileT * kKb * 2;
constexpr int kXSmem = kXStages * kXStageBytes + 1024;
static_assert(kXSmem + 1024 <= kTcMaxSmem, "shared memory");

__global__ void __launch_bounds__(kTcThreads, 1)
    router_dgrad_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_dl,
                        float* __restrict__ d_x, int64_t T, int N, int d, int c_tiles, int64_t tiles,
                        int accumulate, int* status, uint64_t timeout_ns) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  __shared__ TcShared sh;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  tc_setup(sh, warp, 512, kTcThreads - 64);
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
        const int a_boxes = min(2, (d - c0) / 64);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kXStages;
          if (!mbar_wait(smem_u32(&sh.empty[s]), ((it / kXStages) & 1) ^ 1u, timeout_ns, &sh.abort)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&sh.full[s]);
          const uint32_t a = base + s * kXStageBytes, b = a + 3 * 2 * kBox;
          mbar_arrive_expect_tx(fb, 3 * (a_boxes * kBox + kXTileT * kKb * 2));
          for (int k = 0; k < 3; ++k) {
            for (int i = 0; i < a_boxes; ++i)
              tma_load_3d(a + (2 * k + i) * kBox, &tm_w, fb, c0 + 64 * i, kb * kKb, k, last);
            tma_load_3d(b + k * (kXTileT * kKb * 2), &tm_dl, fb, kb * kKb, r0, k, last);
          }
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
    constexpr uint32_t idesc = idesc_bf16_f32(kXTileC, kXTileT) | (1u << 15);  // A MN-major, B K-major
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
        if (lane == 0) {
          const uint32_t a = base + s * kXStageBytes, b = a + 3 * 2 * kBox;
          const int steps = min(kKb / 16, (N - kb * kKb + 15) / 16);
          for (int kk = 0; kk < steps; ++kk)
#pragma unroll
            for (int ka = 0; ka < 3; ++ka)
#pragma unroll
              for (int kt = 0; kt + ka < 3; ++kt)
                tc_mma_f16(tmem + buf * kXTileT, desc_mn(a + 2 * ka * kBox + kk * 2048),
                           desc_k64(b + kt * (kXTileT * kKb * 2) + kk * 32), idesc,
                           kb > 0 || kk > 0 || ka > 0 || kt > 0);
          tc_commit(smem_u32(&sh.empty[s]));
        }
        issued = true;
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) tc_commit(smem_u32(&sh.tfull[buf]));
    }
    if (!ok && lane == 0) {
      sh.abort = 1;
      report_error(status, MOE_ERR_TIMEOUT);
    }
    if (issued && lane == 0) {
      tc_commit(smem_u32(&sh.done));
      mbar_wait(smem_u32(&sh.done), 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    const int q = warp & 3;                  // TMEM lane quadrant: columns q * 32 .. of the tile
    const int half = (warp - 2) >> 2;        // tokens [half * 128, half * 128 + 128) of the tile
    int uc = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++uc) {
      const int buf = uc & 1;
      const bool got = mbar_wait(smem_u32(&sh.tfull[buf]), (uc >> 1) & 1, timeout_ns, &sh.abort);
      if (!__all_sync(kFull, got)) {
        sh.abort = 1;
        report_error(status, MOE_ERR_TIMEOUT);
        break;
      }
      tc_fence_after_sync();
      const int c = static_cast<int>(t % c_tiles) * kXTileC + q * 32;
      const int64_t r0 = t / c_tiles * kXTileT + half * 128;
      const uint32_t row = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kXTileT + half * 128;
      if (c < d) {
        for (int j = 0; j < 128 && r0 + j < T; j += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(row + j, v);
          tmem_ld_wait();
          float* out = d_x + (r0 + j) * d + c + lane;
          const int rows = static_cast<int>(min(static_cast<int64_t>(32), T - r0 - j));
          if (accumulate) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < rows) atomicAdd(out + static_cast<int64_t>(i) * d, __uint_as_float(v[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < rows) __stcs(out + static_cast<int64_t>(i) * d, __uint_as_float(v[i]));
          }
        }
      }
      tc_fence_before_sync();
      mbar_arrive(smem_u32(&sh.tempty[buf]));
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor cores where the products are worth the five launches.
bool use_tensor_cores(int64_t T, int N, int d) { return T >= 256 && static_cast<double>(T) * N * d >= kTcWork; }

cudaError_t launch_tc(const RouterBackwardArgs& a, cudaStream_t s) {
  const TcPlan p = make_tc_plan(a.T, a.N, a.d);
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  char* ws = static_cast<char*>(a.scratch);
  uint16_t* dl_terms = reinterpret_cast<uint16_t*>(ws);
  uint16_t* w_terms = reinterpret_cast<uint16_t*>(ws + p.dl_bytes);
  float* part = reinterpret_cast<float*>(ws + p.dl_bytes + p.w_bytes);
  float* bias_part = reinterpret_cast<float*>(ws + p.dl_bytes + p.w_bytes + p.part_bytes);
  const uint64_t T = static_cast<uint64_t>(a.T), d = static_cast<uint64_t>(a.d), np = static_cast<uint64_t>(p.np);
  {
    const int64_t w_items = a.d_x != nullptr ? static_cast<int64_t>(a.N) * a.d : 0;
    const int w_ctas = static_cast<int>(std::min<int64_t>((w_items / 4 + kThreads - 1) / kThreads, 592));
    e = launch_pdl(split_kernel, dim3(p.split_ctas + w_ctas), dim3(kThreads), 0, s, a.d_logits, a.w_router,
                   dl_terms, w_terms, a.d_logit_bias != nullptr ? bias_part : nullptr,
                   static_cast<int64_t>(a.T), a.N, p.np, w_items, p.split_rows, p.split_ctas);
    if (e != cudaSuccess) return e;
  }
  const uint64_t dl_dims[3] = {np, T, 3}, dl_str[2] = {np * 2, T * np * 2};
  static PerDeviceOnce once;
  e = once.run([] {
    const cudaError_t r = cudaFuncSetAttribute(router_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMaxSmem - 1024);
    return r != cudaSuccess ? r : cudaFuncSetAttribute(router_dgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmem);
  });
  if (e != cudaSuccess) return e;
  if (a.d_w_router != nullptr) {
    CUtensorMap mx, mdl;
    const uint64_t xd[2] = {d, T}, xs[1] = {d * 2};
    const uint32_t xb[2] = {64, kKb}, db[3] = {64, kKb, 1};
    if (!make_map(&mx, a.x, 2, xd, xs, xb) || !make_map(&mdl, dl_terms, 3, dl_dims, dl_str, db))
      return cudaErrorInvalidValue;
    uint32_t columns = 32;
    while (columns < 2u * p.nu) columns *= 2;
    const int smem = std::max(kTcMinSmem, p.w_stages * p.w_stage_bytes + 1024);
    e = launch_pdl(router_wgrad_kernel, dim3(p.c_tiles * p.chunks), dim3(kTcThreads), smem, s, mx, mdl, part,
                   static_cast<int64_t>(a.T), a.N, a.d, p.nu, p.n_boxes, p.c_tiles, p.chunk, p.w_stages, columns,
                   a.status, a.timeout_ns);
    if (e != cudaSuccess) return e;
  }
  if (a.d_x != nullptr) {
    CUtensorMap mw, mdl;
    const uint64_t wd[3] = {d, static_cast<uint64_t>(a.N), 3}, wst[2] = {d * 2, static_cast<uint64_t>(a.N) * d * 2};
    const uint32_t wb[3] = {64, kKb, 1}, db[3] = {kKb, kXTileT, 1};
    if (!make_map(&mw, w_terms, 3, wd, wst, wb) ||
        !make_map(&mdl, dl_terms, 3, dl_dims, dl_str, db, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
    const int c_tiles = (a.d + kXTileC - 1) / kXTileC;
    const int64_t tiles = c_tiles * ((static_cast<int64_t>(a.T) + kXTileT - 1) / kXTileT);
    const int grid = static_cast<int>(std::min<int64_t>(tiles, di.sm_count));
    e = launch_pdl(router_dgrad_kernel, dim3(grid), dim3(kTcThreads), kXSmem, s, mw, mdl, a.d_x,
                   static_cast<int64_t>(a.T), a.N, a.d, c_tiles, tiles, a.accumulate, a.status, a.timeout_ns);
    if (e != cudaSuccess) return e;
  }
  if (a.d_w_router == nullptr && a.d_logit_bias == nullptr) return cudaSuccess;
  const int64_t items = std::max<int64_t>(static_cast<int64_t>(a.N) * a.d / 4, a.N);
  return launch_pdl(router_backward_sum_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, s,
                    static_cast<const float*>(part), static_cast<const float*>(bias_part), a.d_w_router,
                    a.d_logit_bias, p.chunks, p.split_ctas, a.N, a.d, a.accumulate);
}

}  // namespace

size_t router_backward_scratch_bytes(int64_t T, int N, int d) {
  if (use_tensor_cores(T, N, d)) {
    const TcPlan t = make_tc_plan(T, N, d);
    return t.dl_bytes + t.w_bytes + t.part_bytes + t.bias_bytes;
  }
  const Plan p = make_plan(T, N, d);
  return p.chunks > 1 ? static_cast<size_t>(p.chunks) * N * (d + 1) * sizeof(float) : 0;
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
  const int64_t items = std::max<int64_t>(static_cast<int64_t>(a.N) * a.d / 4, a.N);
  return launch_pdl(router_backward_sum_kernel, dim3(static_cast<unsigned>((items + 255) / 256)),
                    dim3(256), 0, s, static_cast<const float*>(p.part_w),
                    static_cast<const float*>(p.part_b), a.d_w_router, a.d_logit_bias, pl.chunks, pl.chunks,
                    a.N, a.d, a.accumulate);
}

}  // namespace moe
