// Load-balancing loss and router z-loss with their gradient, per-expert counts, padding mask.
//
// With p_t = softmax(L_t), n the number of tokens that count, c_e the (token, choice) pairs of
// those tokens that chose expert e, and P_e = sum_t p_te / n (page «Sparse Mixture-of-Experts»,
// section «Маршрутизация токена и auxiliary loss», for the first term):
//   loss = alpha N sum_e (c_e / n) P_e + z sum_t lse_t^2 / n,   lse_t = log sum_e exp(L_te)
//   dL_te = g p_te [alpha N / n (c_e / n - sum_i (c_i / n) p_ti) + 2 z lse_t / n]
// g being the upstream gradient; the counts pass none. The gradient needs the counts of the
// whole batch but not P, so one pass over the logits gives everything: the counts come first,
// from topk_idx alone (4 k bytes a token against 4 N), and every CTA holds them while it reads
// its tokens' logits once and writes their gradients.
//
//   pass 1 (only past kInlineTokens tokens)  per-chunk counts, one row of the workspace a chunk
//   pass 2  the counts (of the rows, or of topk_idx itself), then the tokens; P's partial sums
//           leave one row a CTA, and the last CTA to finish adds the rows in order
// No floating-point atomics: the results do not depend on the order the CTAs run in.
// Bound by memory: 8 T N bytes with the gradient, about 10 instructions a logit.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalPerSm = 1;
// A lane with fewer values of a token than this takes two tokens at a time (T = 16384, device time in
// us: N = 100 13.9, one at a time 16.5; N = 256, eight values a lane, 18.7 and 17.5).
constexpr int kWide = 8;
constexpr int kMaxN = 256;
// Up to here every CTA counts all tokens' pairs itself (two rounds of its threads); past it they are
// counted in chunks by a first launch. Device time of both, us: T = 1000, N = 64, k = 4 6.4 and
// 7.7; T = 2048, k = 4 8.0 and 8.6; T = 4096, k = 1 11.0 and 9.9; k = 4 11.5 and 10.3.
constexpr int64_t kInlineTokens = 2048;
constexpr int kCountRows = 64;  // rows of partial counts, at most
// lse^2 passes fp32's range where |lse| does 1.8e19 (a counted row of the type's lowest value), and the
// loss divides the sum by n and may multiply it by 0. So there are two sums: the squares below 2^96, and
// those of the larger |lse| times 2^-80. Neither overflows for any number of tokens (2^31 of at most
// 2^96), and what the first has under 2^96 the second has as normal numbers.
constexpr float kFarLse = 0x1p48f, kFarScale = 0x1p-80f;

struct CountPlan {
  int64_t chunk;  // tokens a row
  int rows;       // 0: counted inline
};
CountPlan count_plan(int64_t T) {
  if (T <= kInlineTokens) return {0, 0};
  const int64_t want = std::min<int64_t>(kCountRows, (T + kBalThreads - 1) / kBalThreads);
  const int64_t chunk = (T + want - 1) / want;
  return {chunk, static_cast<int>((T + chunk - 1) / chunk)};
}

// Lanes a token takes (G), loads a lane makes of its row (C) and values a load brings (VEC = 4
// where rows are 16-byte aligned): G * C * VEC >= N, G as small as that allows with C = 1.
struct TokenShape {
  int g, c, vec;
};
TokenShape token_shape(int N) {
  if (N % 4 == 0)
    return N <= 16 ? TokenShape{4, 1, 4} : N <= 32 ? TokenShape{8, 1, 4}
         : N <= 64 ? TokenShape{16, 1, 4} : N <= 128 ? TokenShape{32, 1, 4} : TokenShape{32, 2, 4};
  return N <= 8 ? TokenShape{8, 1, 1} : N <= 16 ? TokenShape{16, 1, 1} : N <= 32 ? TokenShape{32, 1, 1}
       : N <= 64 ? TokenShape{32, 2, 1} : N <= 128 ? TokenShape{32, 4, 1} : TokenShape{32, 8, 1};
}

// CTAs of pass 2: one an SM, fewer when the tokens do not fill them or the workspace has fewer rows.
int balance_ctas(int64_t T, int N, int64_t most) {
  const int per_cta = kBalWarps * (32 / token_shape(N).g);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((T + per_cta - 1) / per_cta, most)));
}
// ints of a row of partial counts: N counts and the tokens, rounded up to four
__host__ __device__ constexpr int count_ints(int N) { return (N + 4) / 4 * 4; }
// floats of a CTA's row: N probabilities rounded up to four, then the two sums of lse^2 and padding
__host__ __device__ constexpr int row_floats(int N) { return (N + 3) / 4 * 4 + 4; }

// Counts of tokens [t0, t1): pairs of counted tokens that chose expert e into s_cnt[e], counted
// tokens into s_cnt[N]. A thread takes two tokens a round, their loads issued together. Integer
// shared-memory atomics: the result has no order, and a token's choices differ, so at most 32 / k
// lanes of an access meet at one expert.
__device__ __forceinline__ void count_pairs(const int32_t* __restrict__ topk_idx,
                                            const uint8_t* __restrict__ mask, int64_t t0, int64_t t1,
                                            int N, int k, int* s_cnt) {
  int n = 0;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += 2 * kBalThreads) {
    int e[2][8];
    bool keep[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t r = t + u * kBalThreads;
      keep[u] = r < t1 && (mask == nullptr || mask[r] != 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[u][j] = r < t1 && j < k ? __ldg(topk_idx + r * k + j) : -1;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      n += keep[u];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (keep[u] && e[u][j] >= 0 && e[u][j] < N) atomicAdd(&s_cnt[e[u][j]], 1);
    }
  }
  n = __reduce_add_sync(kFull, n);
  if ((threadIdx.x & 31) == 0 && n != 0) atomicAdd(&s_cnt[N], n);
}

__global__ void __launch_bounds__(kBalThreads) balance_count_kernel(
    const int32_t* __restrict__ topk_idx, const uint8_t* __restrict__ mask,
    int32_t* __restrict__ rows, int T, int64_t chunk, int N, int k) {
  __shared__ int s_cnt[kMaxN + 1];
  pdl_trigger();
  for (int e = threadIdx.x; e <= N; e += kBalThreads) s_cnt[e] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t t0 = blockIdx.x * chunk;
  count_pairs(topk_idx, mask, t0, min(static_cast<int64_t>(T), t0 + chunk), N, k, s_cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < count_ints(N); e += kBalThreads)
    rows[blockIdx.x * count_ints(N) + e] = e <= N ? s_cnt[e] : 0;
}

struct BalanceParams {
  const float* logits;
  const int32_t* topk_idx;
  const uint8_t* mask;
  const float* d_loss;
  float alpha, z_coef;
  int32_t* counts;
  int32_t* n_tokens;
  float* prob_mean;
  float* loss;
  float* d_logits;
  const int32_t* count_rows;
  int n_count_rows;
  float* part;   // [gridDim.x][row_floats(N)]
  int* counter;  // zero between calls
  int T, N, k;
};

template <int G, int C, int VEC>
__global__ void __launch_bounds__(kBalThreads, kBalPerSm) balance_loss_kernel(const BalanceParams a) {
  constexpr int V = C * VEC;          // values a lane holds of a token
  constexpr int kGroups = 32 / G;     // tokens a warp takes at once
  constexpr int U = V >= kWide ? 1 : 2;  // and rounds of them whose work overlaps
  __shared__ int s_cnt[kMaxN + 4];
  __shared__ float s_acc[kBalWarps][G * V];
  __shared__ float s_z[2][kBalWarps];  // the two sums of lse^2
  __shared__ float4 s_red[kBalThreads];
  __shared__ int s_last;
  const int N = a.N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e <= N; e += kBalThreads) s_cnt[e] = 0;
  pdl_trigger();
  pdl_wait();
  const int gl = lane % G;  // lane within the token's group
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kBalWarps * kGroups;
  int64_t t = (blockIdx.x * kBalWarps + warp) * kGroups + lane / G;
  // a token's logits, -inf where there is none (past N, past T, or padding: not even read)
  auto load = [&](int64_t tok, float (&x)[V]) {
    const bool counted = tok < a.T && (a.mask == nullptr || a.mask[tok] != 0);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * G + gl) * VEC;
      if (VEC == 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (counted && e < N) q = __ldcs(reinterpret_cast<const float4*>(a.logits + tok * N + e));
        x[c * VEC] = q.x;
        x[c * VEC + VEC / 4] = q.y;
        x[c * VEC + VEC / 2] = q.z;
        x[c * VEC + VEC * 3 / 4] = q.w;
      } else {
        x[c] = counted && e < N ? __ldcs(a.logits + tok * N + e) : -INFINITY;
      }
    }
  };
  // U tokens at a time: one's shuffles and exponentials fill the other's waits
  float next[U][V];  // under way while the counts are formed
#pragma unroll
  for (int u = 0; u < U; ++u) load(t + u * stride, next[u]);
  __syncthreads();
  if (a.n_count_rows == 0) {
    count_pairs(a.topk_idx, a.mask, 0, a.T, N, a.k, s_cnt);
  } else {
    // four columns a thread, and every (kBalThreads / quads)-th row
    const int quads = count_ints(N) / 4, groups = kBalThreads / quads;
    const int q = threadIdx.x % quads, g = threadIdx.x / quads;
    if (g < groups) {
      int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 8
      for (int r = g; r < a.n_count_rows; r += groups) {
        const int4 v = __ldcg(reinterpret_cast<const int4*>(a.count_rows) + r * quads + q);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      const int c[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c[i] != 0) atomicAdd(&s_cnt[q * 4 + i], c[i]);
    }
  }
  __syncthreads();
  const int n = s_cnt[N];
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < N; e += kBalThreads) a.counts[e] = s_cnt[e];
    if (threadIdx.x == 0) *a.n_tokens = n;
  }
  const float inv_n = 1.0f / static_cast<float>(max(n, 1));
  const float g = a.d_loss != nullptr ? *a.d_loss : 1.0f;
  const float c_bal = g * a.alpha * static_cast<float>(N) * inv_n;
  const float c_z = g * 2.0f * a.z_coef * inv_n;
  float f[V], acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j / VEC * G + gl) * VEC + j % VEC;
    f[j] = e < N ? static_cast<float>(s_cnt[e]) * inv_n : 0.f;
    acc[j] = 0.f;
  }
  float z_near = 0.f, z_far = 0.f;
  for (; t - lane / G < a.T; t += U * stride) {
    float v[U][V], m[U], base[U], sum[U], inner[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[u][j] = next[u][j];
        m[u] = fmaxf(m[u], v[u][j]);
      }
      load(t + (U + u) * stride, next[u]);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(kFull, m[u], o));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      base[u] = m[u] == -INFINITY ? 0.f : m[u];  // a row of -inf only (or one that is not counted)
      sum[u] = inner[u] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[u][j] = expf(v[u][j] - base[u]);
        sum[u] += v[u][j];
        inner[u] += v[u][j] * f[j];
      }
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        sum[u] += __shfl_xor_sync(kFull, sum[u], o);
        inner[u] += __shfl_xor_sync(kFull, inner[u], o);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float inv = sum[u] > 0.f ? 1.0f / sum[u] : 0.f;
      const float lse = sum[u] > 0.f ? base[u] + logf(sum[u]) : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[u][j] *= inv;
        acc[j] += v[u][j];
      }
      if (gl == 0) {
        const bool far = fabsf(lse) >= kFarLse;
        const float x = far ? lse * kFarScale : lse;
        if (far) z_far += x * x;
        else z_near += x * x;
      }
      const int64_t tok = t + u * stride;
      if (a.d_logits != nullptr && tok < a.T) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[u][j] *= c_bal * (f[j] - inner[u] * inv) + c_z * lse;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int e = (c * G + gl) * VEC;
          if (e < N) {
            if (VEC == 4)
              *reinterpret_cast<float4*>(a.d_logits + tok * N + e) =
                  make_float4(v[u][c * VEC], v[u][c * VEC + VEC / 4], v[u][c * VEC + VEC / 2],
                              v[u][c * VEC + VEC * 3 / 4]);
            else
              a.d_logits[tok * N + e] = v[u][c];
          }
        }
      }
    }
  }
  // P's partial sums: groups of a warp, then the warps in order
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z_near += __shfl_xor_sync(kFull, z_near, o);
    z_far += __shfl_xor_sync(kFull, z_far, o);
  }
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < V; ++j) s_acc[warp][(j / VEC * G + gl) * VEC + j % VEC] = acc[j];
  }
  if (lane == 0) {
    s_z[0][warp] = z_near;
    s_z[1][warp] = z_far;
  }
  __syncthreads();
  const int rf = row_floats(N);
  float* my_row = a.part + static_cast<int64_t>(blockIdx.x) * rf;
  for (int e = threadIdx.x; e < rf; e += kBalThreads) {
    float s = 0.f;
    if (e < N)
      for (int w = 0; w < kBalWarps; ++w) s += s_acc[w][e];
    else if (e == rf - 4 || e == rf - 3)
      for (int w = 0; w < kBalWarps; ++w) s += s_z[e - (rf - 4)][w];
    my_row[e] = s;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.counter, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // rows in order, four columns a thread: the threads of a column take a contiguous range of the
  // rows each, and their sums are added in range order
  const int quads = rf / 4;
  const int ranges = kBalThreads / quads;
  const int q = threadIdx.x % quads, r = threadIdx.x / quads;
  float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < ranges) {
    const int n_rows = gridDim.x;
    const int r0 = static_cast<int>(static_cast<int64_t>(n_rows) * r / ranges);
    const int r1 = static_cast<int>(static_cast<int64_t>(n_rows) * (r + 1) / ranges);
#pragma unroll 8
    for (int b = r0; b < r1; ++b) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(b) * rf) + q);
      s4.x += v.x;
      s4.y += v.y;
      s4.z += v.z;
      s4.w += v.w;
    }
  }
  s_red[threadIdx.x] = s4;
  __syncthreads();
  float term = 0.f;
  if (threadIdx.x < quads) {
    for (int i = 1; i < ranges; ++i) {
      const float4 v = s_red[i * quads + q];
      s4.x += v.x;
      s4.y += v.y;
      s4.z += v.z;
      s4.w += v.w;
    }
    if (q == quads - 1) {
      // in fp64: the far sum counts 2^160 times, and z_coef may be 0
      const double z = static_cast<double>(a.z_coef) * inv_n * (s4.x + s4.y * 0x1p160);
      s_z[0][0] = static_cast<float>(z);
    } else {
      const float P[4] = {s4.x * inv_n, s4.y * inv_n, s4.z * inv_n, s4.w * inv_n};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = q * 4 + i;
        if (e < N) {
          a.prob_mean[e] = P[i];
          term += static_cast<float>(s_cnt[e]) * inv_n * P[i];
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
  if (lane == 0) s_acc[warp][0] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < kBalWarps; ++w) t += s_acc[w][0];
    const float balance = a.alpha * static_cast<float>(N) * t;
    const float zl = s_z[0][0];
    a.loss[0] = balance + zl;
    a.loss[1] = balance;
    a.loss[2] = zl;
    *a.counter = 0;
  }
}

}  // namespace

// The counts and one row. The region that the stages share has a row for every SM's CTA but at a few
// sizes (N > 200, d_model = 64, 4100 to 5300 tokens: 115 rows at least), where there are fewer CTAs
// (T = 4300, N = 250 11.5 us, with 148 10.4; T = 5000, N = 256 11.2 and 11.5): asking for more would
// raise what every stage's call needs.
size_t balance_scratch_bytes(int64_t T, int N) {
  if (T == 0) return 0;
  return static_cast<size_t>(count_plan(T).rows) * count_ints(N) * sizeof(int32_t) + row_floats(N) * sizeof(float);
}

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const CountPlan cp = count_plan(a.T);
  BalanceParams p{};
  p.logits = a.logits;
  p.topk_idx = a.topk_idx;
  p.mask = a.token_mask;
  p.d_loss = a.d_loss;
  p.alpha = a.alpha;
  p.z_coef = a.z_coef;
  p.counts = a.counts;
  p.n_tokens = a.n_tokens;
  p.prob_mean = a.prob_mean;
  p.loss = a.loss;
  p.d_logits = a.d_logits;
  p.count_rows = static_cast<const int32_t*>(a.scratch);
  p.n_count_rows = cp.rows;
  const size_t count_bytes = static_cast<size_t>(cp.rows) * count_ints(a.N) * sizeof(int32_t);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.scratch) + count_bytes);
  p.counter = a.counter;
  p.T = a.T;
  p.N = a.N;
  p.k = a.k;
  if (cp.rows > 0) {
    e = launch_pdl(balance_count_kernel, dim3(cp.rows), dim3(kBalThreads), 0, s, a.topk_idx,
                   a.token_mask, static_cast<int32_t*>(a.scratch), a.T, cp.chunk, a.N, a.k);
    if (e != cudaSuccess) return e;
  }
  const TokenShape ts = token_shape(a.N);
  void (*kern)(BalanceParams) = nullptr;
  if (ts.vec == 4)
    kern = ts.g == 4 ? balance_loss_kernel<4, 1, 4> : ts.g == 8 ? balance_loss_kernel<8, 1, 4>
         : ts.g == 16 ? balance_loss_kernel<16, 1, 4> : ts.c == 1 ? balance_loss_kernel<32, 1, 4>
         : balance_loss_kernel<32, 2, 4>;
  else
    kern = ts.g == 8 ? balance_loss_kernel<8, 1, 1> : ts.g == 16 ? balance_loss_kernel<16, 1, 1>
         : ts.c == 1 ? balance_loss_kernel<32, 1, 1> : ts.c == 2 ? balance_loss_kernel<32, 2, 1>
         : ts.c == 4 ? balance_loss_kernel<32, 4, 1> : balance_loss_kernel<32, 8, 1>;
  const int64_t rows = (a.scratch_bytes - count_bytes) / (row_floats(a.N) * sizeof(float));
  const int grid = balance_ctas(a.T, a.N, std::min<int64_t>(di.sm_count * kBalPerSm, rows));
  return launch_pdl(kern, dim3(grid), dim3(kBalThreads), 0, s, p);
}

}  // namespace moe
