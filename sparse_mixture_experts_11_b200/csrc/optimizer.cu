// The update that follows the layer's backward pass: the global norm of many gradients, and one
// AdamW step over many tensors.
//
// Both read a table of the tensors from the kernel's parameters (no device memory, no copy
// before the launch) and cut every tensor into chunks of whole 128-element blocks; the chunks of
// all tensors, end to end, are dealt to the CTAs, so hundreds of small tensors and one tensor of
// gigabytes both fill the GPU with one launch.
//
// AdamW (decoupled weight decay), element by element:
//   g' = g * grad_scale
//   m' = beta1 m + (1 - beta1) g',   v' = beta2 v + (1 - beta2) g'^2
//   p' = p (1 - lr wd) - lr / (1 - beta1^t) * m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
// All of it is fp32. What bounds it is HBM: it reads and writes every state once and shares
// nothing between elements.
//
// Moments in 8 bits: m and r = sqrt(v) are held as E4M3 codes with one fp32 scale per 128
// elements, amax / 448. sqrt(v) and not v, because E4M3's 18 binades then cover 36 binades of v,
// and because r is what divides the update. The fresh m' and r make this step's update; only
// what is kept for the next step is rounded. That rounding is stochastic: a moving average
// moves by less than half a code step in most steps (v by 0.1 % a step at beta2 = 0.999, the
// codes lie 6 to 12 % apart), so rounding to nearest would hold it where it is, while up with the
// probability of the part cut off keeps its expectation. A nonzero r keeps a nonzero code, so
// that no m is divided by eps alone. The random bits are a function of (seed, step, place of the
// tensor in the list, element), so a step is reproducible.
// A bf16 parameter without an fp32 master copy is rounded the same way: most updates are below
// half its spacing.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kOptThreads = 256;
constexpr int kOptWarps = kOptThreads / 32;
constexpr int kQBlock = MOE_ADAMW_BLOCK;  // elements of a block: one warp, four a lane
static_assert(kQBlock == 128, "a warp takes one block, four elements a lane");

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x2F5A6B1Du;
  x ^= x >> 15;
  x *= 0xB4C3D7A9u;
  x ^= x >> 16;
  return x;
}

// Index of the last entry whose first chunk is at or before c (entries hold ascending chunk0).
template <typename Entry>
__device__ __forceinline__ int find_entry(const Entry* e, int n, int c) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (e[mid].chunk0 <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ gradient norm
struct NormEntry {
  const void* grad;
  int64_t numel;
  int32_t chunk0;
  int32_t bf16;
};
constexpr int kNormTable = 1024;  // entries of one launch: 24 KB of kernel parameters
struct NormTable {
  int n, chunks, chunk;  // chunk: elements of a chunk
  int first, last;       // first launch of the call: slots start at zero; last: it finishes
  NormEntry e[kNormTable];
};

// Sum of squares. A thread adds 8 squares in fp32 and the eights in fp64 (fp32 alone would lose
// the small terms of a sum of 1e9); warps, CTAs and the CTAs' slots add in a fixed order. The
// last CTA to arrive adds the slots and forms the norm and the clipping scale.
__global__ void __launch_bounds__(kOptThreads) grad_norm_kernel(const __grid_constant__ NormTable tab,
                                                                double* __restrict__ slots,
                                                                int* __restrict__ counter,
                                                                float max_norm,
                                                                float* __restrict__ norm,
                                                                float* __restrict__ scale) {
  __shared__ double s_sum[kOptWarps];
  __shared__ int s_last;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double sum = 0.0;
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const NormEntry& t = tab.e[find_entry(tab.e, tab.n, c)];
    const int64_t i0 = static_cast<int64_t>(c - t.chunk0) * tab.chunk;
    const int64_t i1 = min(t.numel, i0 + tab.chunk);
    if (t.bf16) {
      const uint16_t* g = static_cast<const uint16_t*>(t.grad);
      const int64_t full = i0 + (i1 - i0) / 8 * 8;
#pragma unroll 4
      for (int64_t i = i0 + threadIdx.x * 8; i < full; i += kOptThreads * 8) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(g + i));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float lo = __uint_as_float(w[q] << 16), hi = __uint_as_float(w[q] & 0xffff0000u);
          s += lo * lo + hi * hi;
        }
        sum += static_cast<double>(s);
      }
      if (threadIdx.x < i1 - full) {
        const float v = bf16_bits_to_float(g[full + threadIdx.x]);
        sum += static_cast<double>(v) * v;
      }
    } else {
      const float* g = static_cast<const float*>(t.grad);
      const int64_t full = i0 + (i1 - i0) / 4 * 4;
      int64_t i = i0 + threadIdx.x * 4;
#pragma unroll 2
      for (; i + kOptThreads * 4 < full; i += kOptThreads * 8) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(g + i));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(g + i + kOptThreads * 4));
        sum += static_cast<double>((a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w) +
                                   (b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w));
      }
      if (i < full) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(g + i));
        sum += static_cast<double>(a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w);
      }
      if (threadIdx.x < i1 - full) {
        const float v = g[full + threadIdx.x];
        sum += static_cast<double>(v) * v;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kOptWarps; ++w) s += s_sum[w];
    slots[blockIdx.x] = tab.first ? s : slots[blockIdx.x] + s;
    __threadfence();
    s_last = tab.last && atomicAdd(counter, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // every launch of the call has the same grid, so the slots are the grid's
  sum = 0.0;
  for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kOptThreads) sum += __ldcg(slots + b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kOptWarps; ++w) s += s_sum[w];
    const float n = static_cast<float>(sqrt(s));
    *norm = n;
    // a norm that is not finite: the scale is NaN, and the AdamW step is left out
    *scale = isfinite(n) ? fminf(1.0f, max_norm / (n + 1e-6f)) : nanf("");
    *counter = 0;
  }
}

// ------------------------------------------------------------------ AdamW
enum { kFp32 = 0, kMaster = 1, kAlone = 2 };  // fp32 parameter; bf16 with fp32 master; bf16 alone

struct AdamEntry {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t numel;
  int32_t chunk0;
  int32_t index;  // place in the caller's list
  float weight_decay;
  uint8_t params, grad_bf16, bits8, pad;
};
struct AdamScalars {
  float lr, b1, omb1, b2, omb2, eps;
  float inv_bc1, inv_sqrt_bc2;  // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double beta1, beta2;          // for a step number read on the device
  uint32_t seed;
  int32_t step;
  const int32_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
};
template <int CAP>
struct AdamTable {
  int n, chunks, chunk_blocks;
  AdamEntry e[CAP];
};

struct StepScalars {  // what every element needs
  float gs, lr_wd1, step_size, b1, omb1, b2, omb2, inv_sqrt_bc2, eps;
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// |x| <= 448 to an E4M3 code, up with the probability of the part that is cut off (u: 16 random
// bits). E4M3 keeps 3 of fp32's 23 mantissa bits: adding random bits below the cut and
// truncating rounds so, across binades too. Below 2^-6 the codes are 2^-9 apart, as they are in
// [2^-6, 2^-5): those values are moved up by 2^-6 and their codes down by 8.
__device__ __forceinline__ uint32_t e4m3_stochastic(float x, uint32_t u) {
  float y = fabsf(x);
  const bool small = y < 0.015625f;
  y = small ? y + 0.015625f : y;
  const uint32_t code = ((__float_as_uint(y) + (u << 4) + 8u) >> 20) - (small ? 968u : 960u);
  return min(code, 126u) | ((__float_as_uint(x) >> 24) & 0x80u);
}

// Four E4M3 codes to fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// Four consecutive elements from p (16-, 8- or 4-byte aligned when `full`), zeros past `rem`.
__device__ __forceinline__ void load4(const float* p, bool full, int rem, float (&f)[4]) {
  if (full) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = a.z;
    f[3] = a.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < rem ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void load4(const uint16_t* p, bool full, int rem, float (&f)[4]) {
  if (full) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
    f[0] = __uint_as_float(a.x << 16);
    f[1] = __uint_as_float(a.x & 0xffff0000u);
    f[2] = __uint_as_float(a.y << 16);
    f[3] = __uint_as_float(a.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < rem ? bf16_bits_to_float(p[i]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t load4(const uint8_t* p, bool full, int rem) {
  if (full) return __ldcs(reinterpret_cast<const uint32_t*>(p));
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < rem) w |= static_cast<uint32_t>(p[i]) << (8 * i);
  return w;
}
__device__ __forceinline__ void store4(float* p, bool full, int rem, const float (&f)[4]) {
  if (full) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < rem) p[i] = f[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, bool full, int rem, uint32_t lo, uint32_t hi) {
  if (full) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(lo, hi));
  } else {
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < rem) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store4(uint8_t* p, bool full, int rem, uint32_t w) {
  if (full) {
    __stcs(reinterpret_cast<uint32_t*>(p), w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < rem) p[i] = static_cast<uint8_t>(w >> (8 * i));
  }
}

// One warp, U consecutive blocks of a tensor from block b0 (those below b1 exist). Lane l takes
// elements 4 l .. 4 l + 3 of each block: 16-byte accesses to fp32, one cache line a warp to the
// codes, and a block's amax is one warp reduction. All loads of the U blocks are issued first.
template <int PARAMS, bool GRAD_BF16, bool BITS8, int U>
__device__ __forceinline__ void adam_blocks(const AdamEntry& t, const StepScalars& s, uint32_t key,
                                            int64_t b0, int64_t b1, int lane) {
  float p[U][4], g[U][4], m[U][4], v[U][4], ms[U], vs[U];
  uint32_t mq[U], vq[U];
  int rem[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = (b0 + u) * kQBlock + lane * 4;
    const int64_t left = t.numel - i;
    rem[u] = b0 + u < b1 && left > 0 ? static_cast<int>(min(left, static_cast<int64_t>(4))) : 0;
    const bool full = rem[u] == 4;
    if (PARAMS == kFp32) load4(static_cast<const float*>(t.param) + i, full, rem[u], p[u]);
    else if (PARAMS == kMaster) load4(t.master + i, full, rem[u], p[u]);
    else load4(static_cast<const uint16_t*>(t.param) + i, full, rem[u], p[u]);
    if (GRAD_BF16) load4(static_cast<const uint16_t*>(t.grad) + i, full, rem[u], g[u]);
    else load4(static_cast<const float*>(t.grad) + i, full, rem[u], g[u]);
    if (BITS8) {
      mq[u] = load4(static_cast<const uint8_t*>(t.m) + i, full, rem[u]);
      vq[u] = load4(static_cast<const uint8_t*>(t.v) + i, full, rem[u]);
      ms[u] = b0 + u < b1 ? t.m_scale[b0 + u] : 0.f;
      vs[u] = b0 + u < b1 ? t.v_scale[b0 + u] : 0.f;
    } else {
      load4(static_cast<const float*>(t.m) + i, full, rem[u], m[u]);
      load4(static_cast<const float*>(t.v) + i, full, rem[u], v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b0 + u >= b1) break;  // warp-uniform
    const int64_t i = (b0 + u) * kQBlock + lane * 4;
    const bool full = rem[u] == 4;
    float r[4];
    if (BITS8) {
      e4m3x4_to_float(mq[u], m[u]);
      e4m3x4_to_float(vq[u], v[u]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (BITS8) {
        m[u][q] *= ms[u];
        v[u][q] *= vs[u];
        v[u][q] *= v[u][q];
      }
      const float gv = g[u][q] * s.gs;
      m[u][q] = s.b1 * m[u][q] + s.omb1 * gv;
      v[u][q] = s.b2 * v[u][q] + s.omb2 * gv * gv;
      r[q] = sqrt_approx(v[u][q]);
      p[u][q] = p[u][q] * s.lr_wd1 -
                s.step_size * __fdividef(m[u][q], r[q] * s.inv_sqrt_bc2 + s.eps);
    }
    uint32_t h[4];
    if (BITS8 || PARAMS == kAlone) {
      const uint32_t base = static_cast<uint32_t>(i) * 0x9E3779B1u + key +
                            static_cast<uint32_t>(i >> 32) * 0x85EBCA6Bu;
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = mix32(base + q * 0x9E3779B1u);
    }
    if (PARAMS == kFp32) {
      store4(static_cast<float*>(t.param) + i, full, rem[u], p[u]);
    } else if (PARAMS == kMaster) {
      store4(t.master + i, full, rem[u], p[u]);
      store4(static_cast<uint16_t*>(t.param) + i, full, rem[u], pack_bf16x2(p[u][0], p[u][1]),
             pack_bf16x2(p[u][2], p[u][3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = __float_as_uint(p[u][q]) + ((h[q] * 0xD1B54A35u + key) >> 16);
      store4(static_cast<uint16_t*>(t.param) + i, full, rem[u], __byte_perm(w[0], w[1], 0x7632),
             __byte_perm(w[2], w[3], 0x7632));
    }
    if (BITS8) {
      uint32_t ma = 0, ra = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        ma = max(ma, __float_as_uint(fabsf(m[u][q])));
        ra = max(ra, __float_as_uint(r[q]));
      }
      ma = __reduce_max_sync(kFull, ma);
      ra = __reduce_max_sync(kFull, ra);
      // a block below 2^-96 (its reciprocal would overflow) is kept as zeros
      const float m_max = __uint_as_float(ma) < 0x1p-96f ? 0.f : __uint_as_float(ma);
      const float r_max = __uint_as_float(ra) < 0x1p-96f ? 0.f : __uint_as_float(ra);
      const float m_inv = m_max > 0.f ? 448.f / m_max : 0.f;
      const float r_inv = r_max > 0.f ? 448.f / r_max : 0.f;
      uint32_t mw = 0, rw = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t mc = m_max > 0.f ? e4m3_stochastic(m[u][q] * m_inv, h[q] & 0xffffu) : 0u;
        uint32_t rc = r_max > 0.f ? e4m3_stochastic(r[q] * r_inv, h[q] >> 16) : 0u;
        if (r_max > 0.f && r[q] > 0.f) rc = max(rc, 1u);
        mw |= mc << (8 * q);
        rw |= rc << (8 * q);
      }
      store4(static_cast<uint8_t*>(t.m) + i, full, rem[u], mw);
      store4(static_cast<uint8_t*>(t.v) + i, full, rem[u], rw);
      if (lane == 0) {
        t.m_scale[b0 + u] = m_max * (1.0f / 448.0f);
        t.v_scale[b0 + u] = r_max * (1.0f / 448.0f);
      }
    } else {
      store4(static_cast<float*>(t.m) + i, full, rem[u], m[u]);
      store4(static_cast<float*>(t.v) + i, full, rem[u], v[u]);
    }
  }
}

template <int PARAMS, bool GRAD_BF16, bool BITS8>
__device__ __forceinline__ void adam_chunk(const AdamEntry& t, const StepScalars& s, uint32_t key,
                                           int64_t b0, int64_t b1) {
  constexpr int U = 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t b = b0 + warp * U; b < b1; b += kOptWarps * U)
    adam_blocks<PARAMS, GRAD_BF16, BITS8, U>(t, s, key, b, b1, lane);
}

template <int CAP>
__global__ void __launch_bounds__(kOptThreads)
    adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, const AdamScalars sc) {
  __shared__ float s_bc[2];
  pdl_trigger();
  pdl_wait();
  const float gs = sc.grad_scale != nullptr ? *sc.grad_scale : 1.0f;
  if (!isfinite(gs)) return;  // the whole step is left out
  int step = sc.step;
  float inv_bc1 = sc.inv_bc1, inv_sqrt_bc2 = sc.inv_sqrt_bc2;
  if (sc.step_dev != nullptr) {
    step = *sc.step_dev;
    if (step < 1) return;
    if (threadIdx.x == 0) {
      s_bc[0] = static_cast<float>(1.0 / (1.0 - pow(sc.beta1, static_cast<double>(step))));
      s_bc[1] = static_cast<float>(1.0 / sqrt(1.0 - pow(sc.beta2, static_cast<double>(step))));
    }
    __syncthreads();
    inv_bc1 = s_bc[0];
    inv_sqrt_bc2 = s_bc[1];
  }
  const float lr = sc.lr_dev != nullptr ? *sc.lr_dev : sc.lr;
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const AdamEntry& t = tab.e[find_entry(tab.e, tab.n, c)];
    const int64_t blocks = (t.numel + kQBlock - 1) / kQBlock;
    const int64_t b0 = static_cast<int64_t>(c - t.chunk0) * tab.chunk_blocks;
    const int64_t b1 = min(blocks, b0 + tab.chunk_blocks);
    const StepScalars s{gs,      1.0f - lr * t.weight_decay, lr * inv_bc1, sc.b1, sc.omb1, sc.b2,
                        sc.omb2, inv_sqrt_bc2,               sc.eps};
    const uint32_t key =
        mix32(mix32(static_cast<uint32_t>(t.index) * 0x632BE5ABu + sc.seed) +
              static_cast<uint32_t>(step) * 0x9E3779B1u);
    // uniform over the CTA
    switch ((t.params * 2 + t.grad_bf16) * 2 + t.bits8) {
      case 0: adam_chunk<kFp32, false, false>(t, s, key, b0, b1); break;
      case 1: adam_chunk<kFp32, false, true>(t, s, key, b0, b1); break;
      case 2: adam_chunk<kFp32, true, false>(t, s, key, b0, b1); break;
      case 3: adam_chunk<kFp32, true, true>(t, s, key, b0, b1); break;
      case 4: adam_chunk<kMaster, false, false>(t, s, key, b0, b1); break;
      case 5: adam_chunk<kMaster, false, true>(t, s, key, b0, b1); break;
      case 6: adam_chunk<kMaster, true, false>(t, s, key, b0, b1); break;
      case 7: adam_chunk<kMaster, true, true>(t, s, key, b0, b1); break;
      case 8: adam_chunk<kAlone, false, false>(t, s, key, b0, b1); break;
      case 9: adam_chunk<kAlone, false, true>(t, s, key, b0, b1); break;
      case 10: adam_chunk<kAlone, true, false>(t, s, key, b0, b1); break;
      default: adam_chunk<kAlone, true, true>(t, s, key, b0, b1); break;
    }
  }
}

constexpr int kAdamTable = 384;  // entries of one launch: 30 KB of kernel parameters
static_assert(sizeof(AdamTable<kAdamTable>) + sizeof(AdamScalars) <= 32764, "kernel parameters");
static_assert(sizeof(NormTable) + 64 <= 32764, "kernel parameters");

}  // namespace

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int n, float max_norm, float* norm,
                             float* scale, void* ws, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  int* counter = reinterpret_cast<int*>(static_cast<char*>(ws) + 64);
  double* slots = reinterpret_cast<double*>(static_cast<char*>(ws) + kStatusBytes);
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += tensors[i].numel;
  const int grid = std::min(kGradNormSlots, di.sm_count * 6);
  // chunks: small enough that a small total reaches every SM, large enough (32 KB of bf16) that
  // finding the tensor costs nothing beside it
  int chunk = 2048;
  while (chunk < 16384 && total / chunk > grid) chunk *= 2;
  NormTable tab;
  tab.first = 1;
  int i = 0;
  do {
    tab.n = 0;
    tab.chunk = chunk;
    int64_t chunks = 0;
    for (; i < n && tab.n < kNormTable; ++i) {
      if (tensors[i].numel == 0) continue;
      const int64_t c = (tensors[i].numel + chunk - 1) / chunk;
      if (chunks + c > INT32_MAX) return cudaErrorInvalidValue;
      NormEntry& t = tab.e[tab.n++];
      t.grad = tensors[i].grad;
      t.numel = tensors[i].numel;
      t.chunk0 = static_cast<int32_t>(chunks);
      t.bf16 = tensors[i].dtype == MOE_DTYPE_BF16;
      chunks += c;
    }
    tab.chunks = static_cast<int>(chunks);
    tab.last = i >= n;
    e = launch_pdl(grad_norm_kernel, dim3(grid), dim3(kOptThreads), 0, s, tab, slots, counter,
                   max_norm, norm, scale);
    if (e != cudaSuccess) return e;
    tab.first = 0;
  } while (i < n);
  return cudaSuccess;
}

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int n, const moe_adamw_config& cfg,
                         cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  AdamScalars sc{};
  sc.lr = static_cast<float>(cfg.lr);
  sc.b1 = static_cast<float>(cfg.beta1);
  sc.omb1 = static_cast<float>(1.0 - cfg.beta1);
  sc.b2 = static_cast<float>(cfg.beta2);
  sc.omb2 = static_cast<float>(1.0 - cfg.beta2);
  sc.eps = static_cast<float>(cfg.eps);
  sc.beta1 = cfg.beta1;
  sc.beta2 = cfg.beta2;
  sc.step = cfg.step;
  if (cfg.step_dev == nullptr) {
    sc.inv_bc1 = static_cast<float>(1.0 / (1.0 - pow(cfg.beta1, cfg.step)));
    sc.inv_sqrt_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(cfg.beta2, cfg.step)));
  }
  sc.seed = cfg.seed;
  sc.step_dev = cfg.step_dev;
  sc.lr_dev = cfg.lr_dev;
  sc.grad_scale = cfg.grad_scale;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += (tensors[i].numel + kQBlock - 1) / kQBlock;
  const int64_t resident = static_cast<int64_t>(di.sm_count) * 8;
  // blocks of a chunk: one pass of the CTA's warps (16 blocks) while that leaves fewer chunks
  // than CTAs, up to eight passes for large totals
  int chunk_blocks = 16;
  while (chunk_blocks < 128 && total / chunk_blocks > resident) chunk_blocks *= 2;
  AdamTable<kAdamTable> tab;
  for (int i = 0; i < n;) {
    tab.n = 0;
    tab.chunk_blocks = chunk_blocks;
    int64_t chunks = 0;
    for (; i < n && tab.n < kAdamTable; ++i) {
      const moe_adamw_tensor& in = tensors[i];
      if (in.numel == 0) continue;
      const int64_t c = ((in.numel + kQBlock - 1) / kQBlock + chunk_blocks - 1) / chunk_blocks;
      if (chunks + c > INT32_MAX) return cudaErrorInvalidValue;
      AdamEntry& t = tab.e[tab.n++];
      t.param = in.param;
      t.master = in.master;
      t.grad = in.grad;
      t.m = in.m;
      t.v = in.v;
      t.m_scale = in.m_scale;
      t.v_scale = in.v_scale;
      t.numel = in.numel;
      t.chunk0 = static_cast<int32_t>(chunks);
      t.index = i;
      t.weight_decay = in.weight_decay;
      t.params = in.param_dtype == MOE_DTYPE_F32 ? kFp32 : in.master != nullptr ? kMaster : kAlone;
      t.grad_bf16 = in.grad_dtype == MOE_DTYPE_BF16;
      t.bits8 = in.state_bits == 8;
      t.pad = 0;
      chunks += c;
    }
    if (chunks == 0) break;
    tab.chunks = static_cast<int>(chunks);
    const int grid = static_cast<int>(std::min<int64_t>(chunks, resident));
    e = launch_pdl(adamw_kernel<kAdamTable>, dim3(grid), dim3(kOptThreads), 0, s, tab, sc);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
