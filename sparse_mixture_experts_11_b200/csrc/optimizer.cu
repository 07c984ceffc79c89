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
//   m' = beta1 m + (1 - beta1) g',   v' = beta2 v + ((1 - beta2) g') g'
//   p' = p (1 - lr wd) - (lr / (1 - beta1^t) m') / (sqrt(v') c + eps),   c = 1 / sqrt(1 - beta2^t)
// All of it is fp32; what does not depend on the element is formed once, in fp64, and rounded (c: the
// root is rounded, then its reciprocal). What bounds it is HBM: it reads and writes every state once
// and shares nothing between elements.
//
// Moments in 8 bits: m and r = sqrt(v) are held as E4M3 codes with one fp32 scale per 128
// elements, amax / 448. sqrt(v) and not v, because E4M3's 18 binades then cover 36 binades of v,
// and because r is what divides the update. The fresh m' and r make this step's update; only
// what is kept for the next step is rounded. That rounding is stochastic: a moving average
// moves by less than half a code step in most steps (v by 0.1 % a step at beta2 = 0.999, the
// codes lie 6 to 12 % apart), so rounding to nearest would hold it where it is, while up with the
// probability of the part cut off keeps the expectation of m and of r. It is r^2 that the next step
// reads, and that gains the rounding's variance: with a step of r of d (0.05 % of it, mostly) between
// codes h apart, h |d| a step, decaying by 1 - beta2, so v settles about (h / r) E|g^2 / v - 1| / 2 above
// its fp32 value, and as much again at most since the scale moves too (5 to 7 % in the mean for normal
// and for heavy-tailed gradients). A nonzero r keeps a nonzero code, so that no m is divided by eps
// alone. The random bits are a function of (seed, step, place of the tensor in the list, element), so a
// step is reproducible.
// A bf16 parameter without an fp32 master copy is rounded the same way: most updates are below
// half its spacing.
//
// Where a value lies next to a border of the codes, its last bit decides between codes 6 to 12 %
// apart, and a block's next scale can hang on one code. So every fp32 operation is rounded by
// itself, in the order of the formulas (no fused multiply-add; square root, quotient and
// reciprocal to nearest), a block's scale being top (1 / 448) and its values times (1 / top) 448: any
// fp32 implementation of these lines has the same results, bit by bit.
// 537M elements with masters took 2365 us so and 2305 with approximate roots and quotients.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kOptThreads = 256;
constexpr int kOptWarps = kOptThreads / 32;
// Mixed lists up to here (in tiles) take one launch for both kinds of moments. Device time of one
// launch and of two, us: 384 tiles 5.1, 9.8; 1930 tiles 19.0, 22.8; 6146 tiles 50.3, 53.3; 36888 tiles
// 308.9, 287.5. Between the limit and that, which is ahead goes by the kinds in the list (24584 tiles with
// masters 208.0, 221.5): of the lists measured past the limit two launches lose 6 % at most.
constexpr int64_t kBothTiles = 8192;
constexpr int kTileBlocks = 2 * kOptWarps;  // a tile: two blocks for each warp of a CTA
constexpr int64_t kMaxChunks = 1 << 30;  // of a launch: a kernel's chunk index plus its grid is an int
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

// The same by a whole warp, where most chunks are their CTA's only one: chunk0 ascends and ends in
// INT_MAX, so the entries at or before c are counted, all loads at once. Generic loads: an access to the
// parameters by lane would be one constant load for every lane, and the binary search waits for a
// cold constant line at each of its steps (AdamW, 256 tensors of 10000, fp32 moments 11.2 us with it and
// 9.6; 8-bit 13.7 and 12.9. The persistent norm kernel loses by it: 200 tensors 5.4 and 5.8).
template <int CAP>
__device__ __forceinline__ int find_entry_warp(const int32_t (&chunk0)[CAP], int c) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  if constexpr (CAP == 32) {
    int v;
    asm("ld.s32 %0, [%1];" : "=r"(v) : "l"(&chunk0[lane]));
    n = v <= c;
  } else {
    static_assert(CAP % 128 == 0, "four a lane");
#pragma unroll 3
    for (int j = 0; j < CAP; j += 128) {
      int4 v;
      asm("ld.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(&chunk0[j + lane * 4]));
      n += (v.x <= c) + (v.y <= c) + (v.z <= c) + (v.w <= c);
    }
  }
  return __reduce_add_sync(kFull, n) - 1;
}

// ------------------------------------------------------------------ gradient norm
struct NormEntry {
  const void* grad;
  int64_t numel;
  int32_t chunk0;
  int32_t bf16;
};
// Entries of one launch: 24 KB of kernel parameters, or 0.8 KB for short lists (the launch copies
// its parameters: 1.5 us more for the large table).
constexpr int kNormTable = 1024, kNormTableShort = 32;
template <int CAP>
struct NormTable {
  int n, chunks, chunk;  // chunk: elements of a chunk
  int first, last;       // first launch of the call: slots start at zero; last: it finishes
  NormEntry e[CAP];
};

// Sum of squares. A thread adds 8 squares in fp32 and the eights in fp64 (fp32 alone would lose
// the small terms of a sum of 1e9); warps, CTAs and the CTAs' slots add in a fixed order. The
// last CTA to arrive adds the slots and forms the norm and the clipping scale.
template <int CAP>
__global__ void __launch_bounds__(kOptThreads)
    grad_norm_kernel(const __grid_constant__ NormTable<CAP> tab, double* __restrict__ slots,
                     int* __restrict__ counter, float max_norm, float* __restrict__ norm,
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
  int32_t index;  // place in the caller's list
  float weight_decay;
  uint8_t params, grad_bf16, bits8;
};
struct AdamScalars {
  float b1, omb1, b2, omb2, eps;  // omb: 1 - beta
  float step_size, inv_sqrt_bc2;  // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double rate, beta1, beta2;      // for a step number or rate read on the device
  uint32_t seed;
  int32_t step;
  const int32_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
};
template <int CAP>
struct AdamTable {
  int n, chunks, chunk_tiles;
  alignas(16) int32_t chunk0[CAP];  // first chunk of each entry, then INT_MAX
  AdamEntry e[CAP];
};

struct StepScalars {  // what every element needs; omb: 1 - beta
  float gs, b1, omb1, b2, omb2;
  float lr_wd1, step_size, inv_sqrt_bc2, eps;  // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
};

// Two fp32 operations in one instruction (sm_100): the kernel is bound by instruction issue where
// the moments are 8 bits wide (73 % of the issue slots, DRAM at 3 of 6.5 TB/s).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Products that are added next, and their sums, each rounded by itself: by the scalar intrinsics, which
// are documented never to be merged into a fused operation. Packed ones have no such promise, and with
// them no kind of tensor has the bits of the same lines in plain fp32 operations.
__device__ __forceinline__ float2 mul2_rn(float2 a, float b) {
  return make_float2(__fmul_rn(a.x, b), __fmul_rn(a.y, b));
}
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
// The largest of three; NaN where one is (fmaxf would drop it, and a block's scale hide it).
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two bf16, each rounded up in magnitude with the probability of the part that is cut off: the 16
// random bits (rbits' low half for x, high for y) are added to the bits and the sum is cut, except
// that a NaN stays one.
__device__ __forceinline__ uint32_t bf16x2_by_chance(float2 a, uint32_t rbits) {
  uint32_t d;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(d) : "f"(a.y), "f"(a.x), "r"(rbits));
  return d;
}

// E4M3 rounding, up with the probability of the part that is cut off. z = x 2^-120 for |x| <= 448:
// x = 2^-6, E4M3's smallest normal, becomes 2^-126, fp32's, and the subnormals of the two formats
// coincide, so the code of x is z's bits above the 20 that E4M3 does not have. Adding 20 random
// bits (u: 16 of them at bits 4-19) and cutting rounds across binades and into the subnormals
// alike. Returns the code in bits 24-30; the bits below are noise.
__device__ __forceinline__ uint32_t e4m3_up(uint32_t z, uint32_t u) {
  return min(z + u, 0x7EFFFFFu) << 4;
}

// Four E4M3 codes to fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float2 (&f)[2]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  f[0] = __half22float2(*reinterpret_cast<__half2*>(&lo));
  f[1] = __half22float2(*reinterpret_cast<__half2*>(&hi));
}

// Four consecutive elements as loaded: fp32 in 16 bytes, bf16 in 8, codes in 4. Elements past
// `rem` read as zero and are not written; FULL: there are four.
template <bool FULL>
__device__ __forceinline__ uint4 load_f32x4(const float* p, int rem) {
  if (FULL || rem >= 4) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint4 a = make_uint4(0u, 0u, 0u, 0u);
  if (rem > 0) a.x = __float_as_uint(p[0]);
  if (rem > 1) a.y = __float_as_uint(p[1]);
  if (rem > 2) a.z = __float_as_uint(p[2]);
  return a;
}
template <bool FULL>
__device__ __forceinline__ uint2 load_bf16x4(const uint16_t* p, int rem) {
  if (FULL || rem >= 4) return __ldcs(reinterpret_cast<const uint2*>(p));
  uint2 a = make_uint2(0u, 0u);
  if (rem > 0) a.x = p[0];
  if (rem > 1) a.x |= static_cast<uint32_t>(p[1]) << 16;
  if (rem > 2) a.y = p[2];
  return a;
}
template <bool FULL>
__device__ __forceinline__ uint32_t load_u8x4(const uint8_t* p, int rem) {
  if (FULL || rem >= 4) return __ldcs(reinterpret_cast<const uint32_t*>(p));
  uint32_t w = 0;
  if (rem > 0) w = p[0];
  if (rem > 1) w |= static_cast<uint32_t>(p[1]) << 8;
  if (rem > 2) w |= static_cast<uint32_t>(p[2]) << 16;
  return w;
}
__device__ __forceinline__ void unpack(const uint4& a, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
  f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
}
__device__ __forceinline__ void unpack(const uint2& a, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u));
  f[1] = make_float2(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
}
template <bool FULL>
__device__ __forceinline__ void store4(float* p, int rem, const float2 (&f)[2]) {
  if (FULL || rem >= 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
  } else {
    if (rem > 0) p[0] = f[0].x;
    if (rem > 1) p[1] = f[0].y;
    if (rem > 2) p[2] = f[1].x;
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint16_t* p, int rem, uint32_t lo, uint32_t hi) {
  if (FULL || rem >= 4) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(lo, hi));
  } else {
    if (rem > 0) p[0] = static_cast<uint16_t>(lo);
    if (rem > 1) p[1] = static_cast<uint16_t>(lo >> 16);
    if (rem > 2) p[2] = static_cast<uint16_t>(hi);
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint8_t* p, int rem, uint32_t w) {
  if (FULL || rem >= 4) {
    __stcs(reinterpret_cast<uint32_t*>(p), w);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < rem) p[i] = static_cast<uint8_t>(w >> (8 * i));
  }
}

template <bool FULL>
__device__ __forceinline__ void load4(const void* p, int64_t i, int rem, uint4& a) {
  a = load_f32x4<FULL>(static_cast<const float*>(p) + i, rem);
}
template <bool FULL>
__device__ __forceinline__ void load4(const void* p, int64_t i, int rem, uint2& a) {
  a = load_bf16x4<FULL>(static_cast<const uint16_t*>(p) + i, rem);
}

// A lane's four elements of one block, as loaded: elements 4 l .. 4 l + 3 for lane l, so that fp32
// takes 16-byte accesses, the codes one cache line a warp, and a block's amax one warp reduction.
template <int PARAMS, bool GRAD_BF16, bool BITS8>
struct Work {
  std::conditional_t<PARAMS == kAlone, uint2, uint4> p;
  std::conditional_t<GRAD_BF16, uint2, uint4> g;
  uint4 m, v;         // fp32 moments
  uint32_t m8, v8;    // or codes
  float ms, vs;       // and scales
  template <bool FULL>
  __device__ __forceinline__ void load(const AdamEntry& t, int64_t b, int64_t i, int rem) {
    load4<FULL>(PARAMS == kMaster ? t.master : t.param, i, rem, p);
    load4<FULL>(t.grad, i, rem, g);
    if (BITS8) {
      m8 = load_u8x4<FULL>(static_cast<const uint8_t*>(t.m) + i, rem);
      v8 = load_u8x4<FULL>(static_cast<const uint8_t*>(t.v) + i, rem);
      ms = t.m_scale[b];
      vs = t.v_scale[b];
    } else {
      load4<FULL>(t.m, i, rem, m);
      load4<FULL>(t.v, i, rem, v);
    }
  }
};

// The step on one block b, by a warp; i: the lane's first element. FULL: the block is whole, else
// only `rem` of the lane's elements exist.
template <int PARAMS, bool GRAD_BF16, bool BITS8, bool FULL>
__device__ __forceinline__ void adam_block(const AdamEntry& t, const StepScalars& s, uint32_t key,
                                           int64_t b, int64_t i, int rem, int lane,
                                           const Work<PARAMS, GRAD_BF16, BITS8>& w) {
  float2 p[2], g[2], m[2], v[2], r[2];
  unpack(w.p, p);
  unpack(w.g, g);
  if (BITS8) {
    e4m3x4_to_float(w.m8, m);
    e4m3x4_to_float(w.v8, v);
  } else {
    unpack(w.m, m);
    unpack(w.v, v);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    // every operation rounded by itself, in the order of the formulas: see the top of the file
    const float2 gv = mul2(g[q], both(s.gs));
    if (BITS8) {
      m[q] = mul2(m[q], both(w.ms));
      v[q] = mul2(v[q], both(w.vs));
      v[q] = mul2(v[q], v[q]);
    }
    m[q] = add2_rn(mul2_rn(m[q], s.b1), mul2_rn(gv, s.omb1));
    const float2 gg = mul2(gv, both(s.omb2));
    v[q] = add2_rn(mul2_rn(v[q], s.b2), make_float2(__fmul_rn(gg.x, gv.x), __fmul_rn(gg.y, gv.y)));
    r[q] = make_float2(__fsqrt_rn(v[q].x), __fsqrt_rn(v[q].y));
    const float2 num = mul2(both(s.step_size), m[q]), keep = mul2_rn(p[q], s.lr_wd1);
    const float2 den = add2_rn(mul2_rn(r[q], s.inv_sqrt_bc2), both(s.eps));
    p[q] = make_float2(__fsub_rn(keep.x, __fdiv_rn(num.x, den.x)), __fsub_rn(keep.y, __fdiv_rn(num.y, den.y)));
  }
  uint32_t h[4];
  if (BITS8 || PARAMS == kAlone) {
    const uint32_t base = static_cast<uint32_t>(i) * 0x9E3779B1u + key +
                          static_cast<uint32_t>(i >> 32) * 0x85EBCA6Bu;
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = mix32(base + q * 0x9E3779B1u);
  }
  if (PARAMS == kFp32) {
    store4<FULL>(static_cast<float*>(t.param) + i, rem, p);
  } else if (PARAMS == kMaster) {
    store4<FULL>(t.master + i, rem, p);
    store4<FULL>(static_cast<uint16_t*>(t.param) + i, rem, pack_bf16x2(p[0].x, p[0].y),
                 pack_bf16x2(p[1].x, p[1].y));
  } else {
    uint32_t u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = h[q] * 0xD1B54A35u + key;
    store4<FULL>(static_cast<uint16_t*>(t.param) + i, rem, bf16x2_by_chance(p[0], __byte_perm(u[0], u[1], 0x7632)),
                 bf16x2_by_chance(p[1], __byte_perm(u[2], u[3], 0x7632)));
  }
  if (BITS8) {
    const float m1 = fabsf(m[1].y), ma4 = max3_nan(fabsf(m[0].x), fabsf(m[0].y), max3_nan(fabsf(m[1].x), m1, m1));
    const float ra4 = max3_nan(r[0].x, r[0].y, max3_nan(r[1].x, r[1].y, r[1].y));
    const float ma = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(ma4)));
    const float ra = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(ra4)));
    // a block below 2^-96 (its reciprocal could overflow) is kept as zeros: codes and scale
    const float m_max = ma < 0x1p-96f ? 0.f : ma, r_max = ra < 0x1p-96f ? 0.f : ra;
    // lane 0 takes m's reciprocal, the others r's: one exact division for both
    const float x_max = lane == 0 ? m_max : r_max;
    const float x_inv = x_max > 0.f ? __frcp_rn(x_max) * 448.f : 0.f;
    const float m_inv = __shfl_sync(kFull, x_inv, 0), r_inv = __shfl_sync(kFull, x_inv, 1);
    const uint32_t least = r_max > 0.f ? 1u << 24 : 0u;  // a nonzero r's smallest code
    uint32_t mc[4], rc[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float2 mz = mul2(mul2(m[q], both(m_inv)), both(0x1p-120f));
      const float2 rz = mul2(mul2(r[q], both(r_inv)), both(0x1p-120f));
      const float mzv[2] = {mz.x, mz.y}, rzv[2] = {rz.x, rz.y}, rv[2] = {r[q].x, r[q].y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t hw = h[2 * q + j], mb = __float_as_uint(mzv[j]);
        // rounding leaves a zero zero: the random bits alone never reach a code
        mc[2 * q + j] = (e4m3_up(mb & 0x7fffffffu, ((hw << 4) & 0xffff0u) + 8u) & 0x7fffffffu) |
                        (mb & 0x80000000u);
        rc[2 * q + j] = max(e4m3_up(__float_as_uint(rzv[j]), ((hw >> 12) & 0xffff0u) + 8u),
                            min(__float_as_uint(rv[j]), least));
      }
    }
    store4<FULL>(static_cast<uint8_t*>(t.m) + i, rem,
                 __byte_perm(__byte_perm(mc[0], mc[1], 0x0073), __byte_perm(mc[2], mc[3], 0x0073), 0x5410));
    store4<FULL>(static_cast<uint8_t*>(t.v) + i, rem,
                 __byte_perm(__byte_perm(rc[0], rc[1], 0x0073), __byte_perm(rc[2], rc[3], 0x0073), 0x5410));
    if (lane == 0) {
      t.m_scale[b] = m_max * (1.0f / 448.0f);
      t.v_scale[b] = r_max * (1.0f / 448.0f);
    }
  } else {
    store4<FULL>(static_cast<float*>(t.m) + i, rem, m);
    store4<FULL>(static_cast<float*>(t.v) + i, rem, v);
  }
}

// A tensor's last block, when it is not whole, by the warp whose turn it is.
template <int PARAMS, bool GRAD_BF16, bool BITS8>
__device__ __forceinline__ void adam_rest(const AdamEntry& t, const StepScalars& s, uint32_t key,
                                          int64_t b, int lane) {
  const int64_t i = b * kQBlock + lane * 4;
  const int rem = static_cast<int>(max(min(t.numel - i, static_cast<int64_t>(4)), static_cast<int64_t>(0)));
  Work<PARAMS, GRAD_BF16, BITS8> w;
  w.template load<false>(t, b, i, rem);
  adam_block<PARAMS, GRAD_BF16, BITS8, false>(t, s, key, b, i, rem, lane, w);
}

// Tiles [tile, tile + n) of a tensor; a warp takes two blocks of each, their loads issued together.
// Only the tensor's last tile can be short.
template <int PARAMS, bool GRAD_BF16, bool BITS8>
__device__ __forceinline__ void adam_run(const AdamEntry& t, const StepScalars& s, int64_t tile,
                                         int n, uint32_t key) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t whole = t.numel / kQBlock;
  int64_t b = tile * kTileBlocks + warp * 2;
  for (; n > 0; --n, b += kTileBlocks) {
    const int64_t i = b * kQBlock + lane * 4;
    if (b + 2 <= whole) {
      Work<PARAMS, GRAD_BF16, BITS8> w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) w[u].template load<true>(t, b + u, i + u * kQBlock, 4);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        adam_block<PARAMS, GRAD_BF16, BITS8, true>(t, s, key, b + u, i + u * kQBlock, 4, lane, w[u]);
    } else {
      for (int64_t c = b; c < b + 2 && c * kQBlock < t.numel; ++c)
        adam_rest<PARAMS, GRAD_BF16, BITS8>(t, s, key, c, lane);
    }
  }
}

// KIND: the table holds tensors with fp32 moments, with 8-bit ones, or both. Large lists take a
// kernel for each (the conversions of the one would cost the other its registers), small mixed
// lists one launch for both.
enum { kMoments32 = 0, kMoments8 = 1, kBoth = 2 };
template <int KIND, int CAP>
__global__ void __launch_bounds__(kOptThreads, KIND == kMoments8 ? 4 : 3)
    adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, const AdamScalars sc) {
  __shared__ float s_bc[2];
  pdl_trigger();
  pdl_wait();
  const float gs = sc.grad_scale != nullptr ? *sc.grad_scale : 1.0f;
  if (!isfinite(gs)) return;  // the whole step is left out
  int step = sc.step;
  double rate = sc.rate;
  float step_size = sc.step_size, inv_sqrt_bc2 = sc.inv_sqrt_bc2;
  if (sc.step_dev != nullptr || sc.lr_dev != nullptr) {
    if (sc.step_dev != nullptr) step = *sc.step_dev;
    if (sc.lr_dev != nullptr) rate = *sc.lr_dev;
    if (step < 1 || !isfinite(rate)) return;
    if (threadIdx.x == 0) {
      s_bc[0] = static_cast<float>(rate / (1.0 - pow(sc.beta1, static_cast<double>(step))));
      s_bc[1] = 1.0f / static_cast<float>(sqrt(1.0 - pow(sc.beta2, static_cast<double>(step))));
    }
    __syncthreads();
    step_size = s_bc[0];
    inv_sqrt_bc2 = s_bc[1];
  }
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int entry = find_entry_warp(tab.chunk0, c);
    const AdamEntry& t = tab.e[entry];
    const int64_t tile = static_cast<int64_t>(c - tab.chunk0[entry]) * tab.chunk_tiles;
    const int64_t tiles = (t.numel - 1) / (kTileBlocks * kQBlock) + 1;
    const int n = static_cast<int>(min(tiles - tile, static_cast<int64_t>(tab.chunk_tiles)));
    const StepScalars s{gs,      sc.b1,
                        sc.omb1, sc.b2,
                        sc.omb2, static_cast<float>(1.0 - rate * static_cast<double>(t.weight_decay)),
                        step_size, inv_sqrt_bc2,
                        sc.eps};
    const uint32_t key =
        mix32(mix32(static_cast<uint32_t>(t.index) * 0x632BE5ABu + sc.seed) +
              static_cast<uint32_t>(step) * 0x9E3779B1u);
    // uniform over the CTA
    if (KIND == kMoments8 || (KIND == kBoth && t.bits8)) {
      switch (t.params * 2 + t.grad_bf16) {
        case 0: adam_run<kFp32, false, true>(t, s, tile, n, key); break;
        case 1: adam_run<kFp32, true, true>(t, s, tile, n, key); break;
        case 2: adam_run<kMaster, false, true>(t, s, tile, n, key); break;
        case 3: adam_run<kMaster, true, true>(t, s, tile, n, key); break;
        case 4: adam_run<kAlone, false, true>(t, s, tile, n, key); break;
        default: adam_run<kAlone, true, true>(t, s, tile, n, key); break;
      }
    } else {
      switch (t.params * 2 + t.grad_bf16) {
        case 0: adam_run<kFp32, false, false>(t, s, tile, n, key); break;
        case 1: adam_run<kFp32, true, false>(t, s, tile, n, key); break;
        case 2: adam_run<kMaster, false, false>(t, s, tile, n, key); break;
        case 3: adam_run<kMaster, true, false>(t, s, tile, n, key); break;
        case 4: adam_run<kAlone, false, false>(t, s, tile, n, key); break;
        default: adam_run<kAlone, true, false>(t, s, tile, n, key); break;
      }
    }
  }
}

// entries of one launch: 30 KB of kernel parameters, or 2.5 KB for short lists
constexpr int kAdamTable = 384, kAdamTableShort = 32;
static_assert(sizeof(AdamTable<kAdamTable>) + sizeof(AdamScalars) <= 32764, "kernel parameters");
static_assert(sizeof(NormTable<kNormTable>) + 64 <= 32764, "kernel parameters");

template <int KIND>
bool of_kind(const moe_adamw_tensor& t) {
  return t.numel > 0 && (KIND == kBoth || (t.state_bits == 8) == (KIND == kMoments8));
}

template <int KIND>
int64_t tiles_of(const moe_adamw_tensor* tensors, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i)
    if (of_kind<KIND>(tensors[i])) total += (tensors[i].numel - 1) / (kTileBlocks * kQBlock) + 1;
  return total;
}

// The tensors of a kind, CAP a launch.
template <int KIND, int CAP>
cudaError_t launch_adamw_kind(const moe_adamw_tensor* tensors, int n, int64_t total, const AdamScalars& sc, int sms,
                              cudaStream_t s) {
  // fp32 moments: a CTA a tile, in the tensor's order. What bounds the kernel is how well the
  // memory streams, and CTAs that start in order keep all SMs within a few pages of each other
  // (537M elements with masters: 2348 us; persistent CTAs on chunks of 16 tiles, 2687 us).
  // 8 bits: as many CTAs as are resident, on chunks that grow with the total: here instructions
  // bound, and a CTA's start is a part of a tile's (1775 us; a CTA a tile, 1877 us).
  const int64_t resident = static_cast<int64_t>(sms) * 4;
  int chunk_tiles = 1;
  while (KIND == kMoments8 && chunk_tiles < 32 && total / chunk_tiles > 8 * resident) chunk_tiles *= 2;
  AdamTable<CAP> tab;
  for (int i = 0; i < n;) {
    tab.n = 0;
    tab.chunk_tiles = chunk_tiles;
    int64_t chunks = 0;
    for (; i < n && tab.n < CAP; ++i) {
      const moe_adamw_tensor& in = tensors[i];
      if (!of_kind<KIND>(in)) continue;
      const int64_t c = ((in.numel - 1) / (kTileBlocks * kQBlock) + chunk_tiles) / chunk_tiles;
      if (chunks + c > kMaxChunks) return cudaErrorInvalidValue;
      tab.chunk0[tab.n] = static_cast<int32_t>(chunks);
      AdamEntry& t = tab.e[tab.n++];
      t.param = in.param;
      t.master = in.master;
      t.grad = in.grad;
      t.m = in.m;
      t.v = in.v;
      t.m_scale = in.m_scale;
      t.v_scale = in.v_scale;
      t.numel = in.numel;
      t.index = i;
      t.weight_decay = in.weight_decay;
      t.params = in.param_dtype == MOE_DTYPE_F32 ? kFp32 : in.master != nullptr ? kMaster : kAlone;
      t.grad_bf16 = in.grad_dtype == MOE_DTYPE_BF16;
      t.bits8 = in.state_bits == 8;
      chunks += c;
    }
    if (chunks == 0) break;
    std::fill(tab.chunk0 + tab.n, tab.chunk0 + CAP, INT32_MAX);
    tab.chunks = static_cast<int>(chunks);
    const int grid = static_cast<int>(KIND == kMoments8 ? std::min<int64_t>(chunks, resident) : chunks);
    const cudaError_t e = launch_pdl(adamw_kernel<KIND, CAP>, dim3(grid), dim3(kOptThreads), 0, s, tab, sc);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int CAP>
cudaError_t launch_adamw_tables(const moe_adamw_tensor* tensors, int n, const AdamScalars& sc, int sms,
                                cudaStream_t s) {
  const int64_t t32 = tiles_of<kMoments32>(tensors, n), t8 = tiles_of<kMoments8>(tensors, n);
  if (t32 > 0 && t8 > 0 && t32 + t8 <= kBothTiles)
    return launch_adamw_kind<kBoth, CAP>(tensors, n, t32 + t8, sc, sms, s);
  cudaError_t e = cudaSuccess;
  if (t32 > 0) e = launch_adamw_kind<kMoments32, CAP>(tensors, n, t32, sc, sms, s);
  if (e == cudaSuccess && t8 > 0) e = launch_adamw_kind<kMoments8, CAP>(tensors, n, t8, sc, sms, s);
  return e;
}

template <int CAP>
cudaError_t launch_grad_norm_tables(const moe_grad_tensor* tensors, int n, float max_norm, float* norm,
                                    float* scale, void* ws, int sms, cudaStream_t s) {
  int* counter = reinterpret_cast<int*>(static_cast<char*>(ws) + 64);
  double* slots = reinterpret_cast<double*>(static_cast<char*>(ws) + kStatusBytes);
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += tensors[i].numel;
  // chunks: small enough that a small total reaches every SM, large enough (32 KB of bf16) that
  // finding the tensor costs nothing beside it; no more CTAs than 2048-element chunks
  const int most = std::min(kGradNormSlots, sms * 6);
  int chunk = 2048;
  while (chunk < 16384 && total / chunk > most) chunk *= 2;
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, total / chunk + n)));
  NormTable<CAP> tab;
  tab.first = 1;
  int i = 0;
  do {
    tab.n = 0;
    tab.chunk = chunk;
    int64_t chunks = 0;
    for (; i < n && tab.n < CAP; ++i) {
      if (tensors[i].numel == 0) continue;
      const int64_t c = (tensors[i].numel + chunk - 1) / chunk;
      if (chunks + c > kMaxChunks) return cudaErrorInvalidValue;
      NormEntry& t = tab.e[tab.n++];
      t.grad = tensors[i].grad;
      t.numel = tensors[i].numel;
      t.chunk0 = static_cast<int32_t>(chunks);
      t.bf16 = tensors[i].dtype == MOE_DTYPE_BF16;
      chunks += c;
    }
    tab.chunks = static_cast<int>(chunks);
    tab.last = i >= n;
    const cudaError_t e = launch_pdl(grad_norm_kernel<CAP>, dim3(grid), dim3(kOptThreads), 0, s, tab, slots,
                                     counter, max_norm, norm, scale);
    if (e != cudaSuccess) return e;
    tab.first = 0;
  } while (i < n);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int n, float max_norm, float* norm,
                             float* scale, void* ws, cudaStream_t s) {
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  return n <= kNormTableShort
             ? launch_grad_norm_tables<kNormTableShort>(tensors, n, max_norm, norm, scale, ws, di.sm_count, s)
             : launch_grad_norm_tables<kNormTable>(tensors, n, max_norm, norm, scale, ws, di.sm_count, s);
}

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int n, const moe_adamw_config& cfg,
                         cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  AdamScalars sc{};
  sc.rate = cfg.lr;
  sc.b1 = static_cast<float>(cfg.beta1);
  sc.omb1 = static_cast<float>(1.0 - cfg.beta1);
  sc.b2 = static_cast<float>(cfg.beta2);
  sc.omb2 = static_cast<float>(1.0 - cfg.beta2);
  sc.eps = static_cast<float>(cfg.eps);
  sc.beta1 = cfg.beta1;
  sc.beta2 = cfg.beta2;
  sc.step = cfg.step;
  if (cfg.step_dev == nullptr) {
    sc.step_size = static_cast<float>(cfg.lr / (1.0 - pow(cfg.beta1, cfg.step)));
    sc.inv_sqrt_bc2 = 1.0f / static_cast<float>(sqrt(1.0 - pow(cfg.beta2, cfg.step)));
  }
  sc.seed = cfg.seed;
  sc.step_dev = cfg.step_dev;
  sc.lr_dev = cfg.lr_dev;
  sc.grad_scale = cfg.grad_scale;
  return n <= kAdamTableShort ? launch_adamw_tables<kAdamTableShort>(tensors, n, sc, di.sm_count, s)
                              : launch_adamw_tables<kAdamTable>(tensors, n, sc, di.sm_count, s);
}

}  // namespace moe
