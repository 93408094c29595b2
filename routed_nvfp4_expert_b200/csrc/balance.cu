// The router's balance loss with its per-expert counts, and the gradient of
// the logits from the balance loss and from the routing weights.
//
// With s = sigmoid(l) (the router's score) and, for sequence b of T_b tokens,
//   c_be = assignments of its tokens to expert e,   f_be = E c_be / (k T_b)
//   P_be = 1/T_b sum_t s_te / S_t,                  S_t = sum_e s_te
//   loss_b = coef sum_e f_be P_be
// f is a count and carries no gradient, so with g_b = d loss_b (upstream)
//   d s_te = g_b coef / (T_b S_t) (f_be - sum_j f_bj s_tj / S_t)
// and with the routing weights w_j = rsf s_j / C, C = sum over the token's
// chosen experts, and upstream v_j = d w_j
//   d s_(id_j) += rsf / C (v_j - sum_i v_i s_i / C)
// and d l = d s * s (1 - s).
//
// Both directions are streams over the logits [T, E]: one warp owns a row in
// registers, so its sums are warp shuffles and every logit is read once. HBM
// bounds long inputs (4 T E bytes forward, 8 T E backward).

#include "common.cuh"
#include "kernels.h"

namespace rnx {

namespace {

constexpr int kSumWarps = 32;          // forward: one 1024-thread CTA per SM, one row per warp
constexpr int kGradWarps = 8;

// e = exp(-|l|) <= 1 and r = 1 / (1 + e) = sigmoid(|l|): then sigmoid(l) is r
// or e r, and sigmoid(l) (1 - sigmoid(l)) = e r r, none with a subtraction, so
// all keep their relative accuracy in the tails. The exponential is 2^(l log2 e)
// with the product's rounding error put back to first order, the two function
// units' approximations are within 2^-22, and a score below 2^-126 is 0: at a
// few instructions per logit the sums stay behind the memory (expf and a full
// division were 2.5 times the HBM time at 131072 x 288).
RNX_DEVICE void exp_parts(float l, float& e, float& r) {
  const float x = fabsf(l);
  const float t = -1.4426950408889634f * x;
  const float lost = fmaf(-1.4426950408889634f, x, -t);
  float p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
  e = fmaf(p * 0.6931471805599453f, lost, p);
  e = x > 126.f ? 0.f : e;                     // an infinity's lost part is NaN
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
}

RNX_DEVICE float score_of(float l) {
  float e, r;
  exp_parts(l, e, r);
  return l >= 0.f ? r : e * r;
}

// Start of sequence b, clamped into [0, T] so that a wrong offset never leads
// outside the rows (offsets NULL: one sequence of T rows).
RNX_DEVICE int seq_start(const int32_t* off, int b, int T) {
  if (!off) return b > 0 ? T : 0;
  return min(max(*(off + b), 0), T);
}

// First sequence that ends behind `row` (B if none).
RNX_DEVICE int seq_of_row(const int32_t* off, int B, int T, int row) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(off, mid + 1, T) > row) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Sums of the rows [lo, hi) by the whole CTA: normalised scores into
// sums[0 .. E) (fixed order: rows within a warp, then the warps) and
// assignment counts into hist[0 .. E). warp_sums: kSumWarps * E floats.
// All threads call it; the results are published by its last barrier.
template <int NV>
RNX_DEVICE void sum_rows(const float* logits, const int32_t* ids, int E, int k, int lo,
                         int hi, float* warp_sums, int* hist) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < E; e += kSumWarps * 32) hist[e] = 0;
  __syncthreads();
  float acc[NV], next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  int next_id = -1;
  auto load = [&](int row) {                        // the next row's loads go out before this row's arithmetic
    if (row < hi) {
      const float* p = logits + (size_t)row * E + lane;
#pragma unroll
      for (int i = 0; i < NV; ++i) next[i] = lane + 32 * i < E ? *(p + 32 * i) : -INFINITY;
      next_id = lane < k ? *(ids + (size_t)row * k + lane) : -1;
    }
  };
  load(lo + warp);
  for (int row = lo + warp; row < hi; row += kSumWarps) {
    float s[NV], total = 0.f;
    const int id = next_id;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = next[i];
    load(row + kSumWarps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = score_of(s[i]);                               // 0 behind the last expert
      total += s[i];
    }
    total = warp_sum(total);
    const float inv = total == 0.f ? 0.f : 1.0f / total;   // a row of zero scores has no shares
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
    if (id >= 0 && id < E) atomicAdd(hist + id, 1);        // integer: the order does not matter
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < E) warp_sums[warp * E + lane + 32 * i] = acc[i];
  __syncthreads();
  for (int e = tid; e < E; e += kSumWarps * 32) {
    float v = 0.f;
#pragma unroll 8
    for (int w = 0; w < kSumWarps; ++w) v += warp_sums[w * E + e];
    warp_sums[e] = v;                                      // only this thread reads or writes column e
  }
  __syncthreads();
}

// One sequence's results from its column sums and counts (published in shared
// memory). n = T_b. red: kSumWarps floats.
RNX_DEVICE void finish_sequence(const float* sums, const int* hist, int E, int k, int n, float coef, int32_t* counts,
                                float* mean, float* loss, float* red) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  const float fs = n > 0 ? (float)E / ((float)k * (float)n) : 0.f;
  float part = 0.f;
  for (int e = tid; e < E; e += kSumWarps * 32) {
    const float p = sums[e] * inv_n;
    counts[e] = hist[e];
    mean[e] = p;
    part = fmaf((float)hist[e] * fs, p, part);
  }
  part = warp_sum(part);
  if (lane == 0) red[warp] = part;
  __syncthreads();
  if (warp == 0) {
    const float v = warp_sum(red[lane]);
    if (lane == 0) *loss = coef * v;
  }
}

struct BalanceParams {
  const float* logits;
  const int32_t* ids;
  const int32_t* off;
  int T, E, k, B, rows_per_block;
  float coef;
  float* psum;      // [blocks + B, E] partial sums, slot = block + sequence
  int* pcnt;        // [blocks + B, E]
  int32_t* counts;  // [B, E]
  float* mean;      // [B, E]
  float* loss;      // [B]
};

// Few tokens: one CTA per sequence does all of it, one launch.
template <int NV>
__global__ void __launch_bounds__(kSumWarps * 32, 1) balance_seq_kernel(const BalanceParams p) {
  extern __shared__ float dyn[];
  __shared__ float red[kSumWarps];
  float* warp_sums = dyn;
  int* hist = reinterpret_cast<int*>(dyn + (size_t)kSumWarps * p.E);
  const int b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int lo = seq_start(p.off, b, p.T), hi = max(lo, seq_start(p.off, b + 1, p.T));
  sum_rows<NV>(p.logits, p.ids, p.E, p.k, lo, hi, warp_sums, hist);
  finish_sequence(warp_sums, hist, p.E, p.k, hi - lo, p.coef, p.counts + (size_t)b * p.E, p.mean + (size_t)b * p.E,
                  p.loss + b, red);
}

// Many tokens, step 1: CTA i sums rows [i R, (i + 1) R). It may meet several
// sequences; its part of sequence b goes to slot i + b, which is its own since
// both only grow.
template <int NV>
__global__ void __launch_bounds__(kSumWarps * 32, 1) balance_partial_kernel(const BalanceParams p) {
  extern __shared__ float dyn[];
  float* warp_sums = dyn;
  int* hist = reinterpret_cast<int*>(dyn + (size_t)kSumWarps * p.E);
  pdl_wait();
  pdl_trigger();
  const int r0 = (int)min((long long)blockIdx.x * p.rows_per_block, (long long)p.T);
  const int r1 = (int)min((long long)r0 + p.rows_per_block, (long long)p.T);
  for (int b = seq_of_row(p.off, p.B, p.T, r0); b < p.B; ++b) {
    const int start = seq_start(p.off, b, p.T);
    if (start >= r1) break;
    const int lo = max(r0, start), hi = min(r1, seq_start(p.off, b + 1, p.T));
    if (lo >= hi) continue;
    sum_rows<NV>(p.logits, p.ids, p.E, p.k, lo, hi, warp_sums, hist);
    const size_t slot = (size_t)(blockIdx.x + b) * p.E;
    for (int e = threadIdx.x; e < p.E; e += kSumWarps * 32) {
      p.psum[slot + e] = warp_sums[e];
      p.pcnt[slot + e] = hist[e];
    }
    __syncthreads();
  }
}

// Step 2: one CTA per sequence adds its slots in order. Warps split the slots
// into `parts` interleaved runs per group of 32 experts.
__global__ void __launch_bounds__(kSumWarps * 32, 1) balance_join_kernel(const BalanceParams p) {
  extern __shared__ float dyn[];
  __shared__ float red[kSumWarps];
  const int E = p.E, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (E + 31) / 32, parts = kSumWarps / groups;   // E <= 1024: at least one part
  float* sums = dyn;                                              // [parts, E]
  int* hist = reinterpret_cast<int*>(dyn + (size_t)parts * E);    // [parts, E]
  const int b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int lo = seq_start(p.off, b, p.T), hi = max(lo, seq_start(p.off, b + 1, p.T));
  const int i0 = lo / p.rows_per_block, i1 = hi > lo ? (hi - 1) / p.rows_per_block + 1 : i0;
  const int part = warp / groups, e = (warp - part * groups) * 32 + lane;
  if (part < parts && e < E) {
    float v = 0.f;
    int c = 0;
    const size_t step = (size_t)parts * E;
    size_t at = (size_t)(i0 + part + b) * E + e;
#pragma unroll 8
    for (int i = i0 + part; i < i1; i += parts, at += step) {
      v += *(p.psum + at);
      c += *(p.pcnt + at);
    }
    sums[part * E + e] = v;
    hist[part * E + e] = c;
  }
  __syncthreads();
  for (int x = tid; x < E; x += kSumWarps * 32) {
    for (int q = 1; q < parts; ++q) {
      sums[x] += sums[q * E + x];
      hist[x] += hist[q * E + x];
    }
  }
  __syncthreads();
  finish_sequence(sums, hist, E, p.k, hi - lo, p.coef, p.counts + (size_t)b * E, p.mean + (size_t)b * E, p.loss + b,
                  red);
}

struct GradParams {
  const float* logits;
  const int32_t* ids;
  const float* d_weights;    // nullable
  const int32_t* off;
  const int32_t* counts;     // [B, E], nullable with d_loss
  const float* d_loss;       // [B], nullable
  float* d_logits;
  int T, E, k, B, rows_per_warp;
  float coef, rsf;
};

// One warp per row, each warp a run of consecutive rows (so that the loads f
// of its sequence stay in registers); the next row's logits are in flight
// meanwhile. The routing weights' part of a row, k values, is spread over the
// experts through a zeroed row in shared memory (testing each expert against
// k ids cost more instructions than everything else).
template <int NV>
__global__ void __launch_bounds__(kGradWarps * 32) router_grad_kernel(const GradParams p) {
  extern __shared__ float spread[];                // [kGradWarps, E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, k = p.k;
  float* mine = spread + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0.f;
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  const long long first = ((long long)blockIdx.x * kGradWarps + warp) * p.rows_per_warp;
  if (first >= p.T) return;
  const int r0 = (int)first, r1 = (int)min(first + p.rows_per_warp, (long long)p.T);
  int b = seq_of_row(p.off, p.B, p.T, r0);
  if (b >= p.B) return;
  int start = seq_start(p.off, b, p.T), end = seq_start(p.off, b + 1, p.T);
  bool fresh = true;
  float f[NV], next[NV], gain = 0.f, next_v = 0.f;
  int next_id = -1;
  auto load = [&](int row) {
    if (row >= r1) return;
    const float* src = p.logits + (size_t)row * E + lane;
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i] = lane + 32 * i < E ? src[32 * i] : -INFINITY;
    if (lane < k && p.d_weights) {
      next_id = p.ids[(size_t)row * k + lane];
      next_v = p.d_weights[(size_t)row * k + lane];
    }
  };
  load(r0);
  for (int row = r0; row < r1; ++row) {
    while (row >= end) {                       // the next sequence that holds rows behind this one
      if (++b >= p.B) return;
      start = end;
      end = max(end, seq_start(p.off, b + 1, p.T));
      fresh = true;
    }
    float l[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = next[i];
    const bool chosen = next_id >= 0 && next_id < E;
    const int id = chosen ? next_id : -1;
    const float v = chosen ? next_v : 0.f;
    load(row + 1);
    if (row < start) continue;                 // before the first sequence: left as it was
    if (fresh) {
      fresh = false;
      const float n = (float)(end - start);
      gain = p.d_loss ? p.d_loss[b] * p.coef / n : 0.f;
      const float fs = (float)E / ((float)k * n);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        f[i] = p.d_loss && lane + 32 * i < E ? (float)p.counts[(size_t)b * E + lane + 32 * i] * fs : 0.f;
    }
    if (p.d_weights) {
      // a chosen score again from its logit (the row is in L1)
      const float sc = id >= 0 ? score_of(p.logits[(size_t)row * E + id]) : 0.f;
      const float c = warp_sum(sc);
      const float ic = c == 0.f ? 0.f : 1.0f / c;
      const float m = warp_sum(v * sc) * ic;
      const float d = p.rsf * ic * (v - m);
      // an expert named in several slots gets their sum, in slot order, from its first
      float sum = 0.f;
      bool lead = id >= 0;
      for (int j = 0; j < k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, id, j);
        const float dj = __shfl_sync(0xffffffffu, d, j);
        sum += ej == id ? dj : 0.f;
        lead = lead && !(ej == id && j < lane);
      }
      if (lead) mine[id] = sum;
      __syncwarp();
    }
    float ds[NV], total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float e, r;
      exp_parts(l[i], e, r);
      const float s = l[i] >= 0.f ? r : e * r;
      ds[i] = e * r * r;
      total += s;
      dot = fmaf(f[i], s, dot);
    }
    total = warp_sum(total);
    dot = warp_sum(dot);
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    const float mean = dot * inv, scale = gain * inv;
    float* dst = p.d_logits + (size_t)row * E + lane;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < E) dst[32 * i] = (scale * (f[i] - mean) + mine[lane + 32 * i]) * ds[i];
    if (p.d_weights) {
      __syncwarp();
      if (id >= 0) mine[id] = 0.f;
      __syncwarp();
    }
  }
}

// Registers per lane for a row: the smallest instantiated count that holds E.
#define RNX_BY_ROW(E, CALL)          \
  do {                               \
    switch (((E) + 31) / 32) {       \
      case 1: CALL(1); break;        \
      case 2: CALL(2); break;        \
      case 3: CALL(3); break;        \
      case 4: CALL(4); break;        \
      case 5: CALL(5); break;        \
      case 6: CALL(6); break;        \
      case 7: CALL(7); break;        \
      case 8: CALL(8); break;        \
      case 9: CALL(9); break;        \
      case 10: CALL(10); break;      \
      case 11: case 12: CALL(12); break;                     \
      case 13: case 14: case 15: case 16: CALL(16); break;   \
      default: CALL(32); break;      \
    }                                \
  } while (0)

}  // namespace

int balance_rows_per_block(int T) {
  return max(kSumWarps, (T + kNumSMs - 1) / kNumSMs);      // one CTA per SM
}

int balance_blocks(int T) {
  if (T <= kBalanceSeqMaxT) return 0;
  const int r = balance_rows_per_block(T);
  return (T + r - 1) / r;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, int T, int E, int k, const int32_t* off,
                                int B, float coef, int32_t* counts, float* mean, float* loss, void* scratch,
                                cudaStream_t st) {
  BalanceParams p{logits, ids, off, T, E, k, B, balance_rows_per_block(T), coef, nullptr, nullptr, counts, mean, loss};
  const size_t smem = ((size_t)kSumWarps + 1) * E * 4;
  const int blocks = balance_blocks(T);
  cudaError_t err = cudaSuccess;
  if (blocks == 0) {
#define CALL(NV)                                                                                                  \
  do {                                                                                                            \
    if (smem > 48 * 1024) err = cudaFuncSetAttribute(balance_seq_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
    if (err == cudaSuccess) err = launch_pdl(balance_seq_kernel<NV>, dim3(B), dim3(kSumWarps * 32), smem, st, p);        \
  } while (0)
    RNX_BY_ROW(E, CALL);
#undef CALL
    return err;
  }
  p.psum = static_cast<float*>(scratch);
  p.pcnt = reinterpret_cast<int*>(p.psum + (size_t)(blocks + B) * E);
#define CALL(NV)                                                                                                  \
  do {                                                                                                            \
    if (smem > 48 * 1024) err = cudaFuncSetAttribute(balance_partial_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
    if (err == cudaSuccess) err = launch_pdl(balance_partial_kernel<NV>, dim3(blocks), dim3(kSumWarps * 32), smem, st, p); \
  } while (0)
  RNX_BY_ROW(E, CALL);
#undef CALL
  if (err != cudaSuccess) return err;
  // [parts, E] twice: parts * E <= kSumWarps * 32 + E at most
  const int parts = kSumWarps / ((E + 31) / 32);
  return launch_pdl(balance_join_kernel, dim3(B), dim3(kSumWarps * 32), (size_t)parts * E * 8, st, p);
}

cudaError_t launch_router_grad(const float* logits, const int32_t* ids, int T, int E, int k, const float* d_weights,
                               float rsf, const int32_t* off, int B, float coef, const int32_t* counts,
                               const float* d_loss, float* d_logits, cudaStream_t st) {
  GradParams p{logits, ids, d_weights, off, counts, d_loss, d_logits, T, E, k, B, 1, coef, rsf};
  // one wave: 32 resident warps per SM at 64 registers (E <= 288), 24 above;
  // beyond that each warp takes a run of rows
  const int warps = kNumSMs * (E <= 288 ? 32 : 24);
  p.rows_per_warp = max(1, (T + warps - 1) / warps);
  const int rows_per_cta = kGradWarps * p.rows_per_warp;
  const int blocks = (T + rows_per_cta - 1) / rows_per_cta;
  cudaError_t err = cudaSuccess;
#define CALL(NV) err = launch_pdl(router_grad_kernel<NV>, dim3(blocks), dim3(kGradWarps * 32), (size_t)kGradWarps * E * 4, st, p)
  RNX_BY_ROW(E, CALL);
#undef CALL
  return err;
}

}  // namespace rnx
