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
// slots with an id in [0, E) (one dropped after the weights were normalised
// keeps its id and has v = 0), and upstream v_j = d w_j
//   d s_(id_j) += rsf / C (v_j - sum_i v_i s_i / C)
// and d l = d s * s (1 - s).
//
// Both directions are streams over the logits [T, E] (4 T E bytes forward, 8 T
// E backward). A row is held in registers by G lanes (4 up to E = 32, 8 up to 320),
// four consecutive logits each, so a warp works on 32 / G rows at a time and
// at E = 288 the row's sums cost 3 shuffles for four rows: with a whole warp per row the
// shuffles, the slot loop and the bookkeeping of each row took as many issue
// slots as its 288 logits (42 us forward at 131072 x 288, 46 us backward at
// 65536 x 288).

#include "common.cuh"
#include "kernels.h"

namespace rnx {

namespace {

constexpr int kMaxK = 16;
// Sixteen warps per SM: one CTA forward, two backward. (Twelve with rings of
// three rows instead of two: 39.6 against 38.2 us forward at 131072 x 288.)
constexpr int kSumWarps = 16, kGradWarps = 8;
constexpr int kJoinWarps = 32;
// Up to these many tokens a whole warp takes a row: 2.8 against 3.5 us forward
// at one token of 288 experts, 3.8 against 5.7 us backward at 1024 (one row per
// resident warp); above, 4.2 against 4.0 us at 32 and 6.4 against 5.9 us at 3000.
constexpr int kSumWideT = 16, kGradWideT = kNumSMs * 2 * kGradWarps;

// s = 1 / (1 + E) and 1 - s = E s with E = exp(-l), on the two function units'
// approximations (within 2^-22; the product l log2 e adds |l| 2^-24 relative):
// four instructions a score, relative accuracy in both tails, and a score
// below 2^-126 is 0. With expf and a division the sums took 2.5 times the HBM
// time at 131072 x 288.
RNX_DEVICE float score_of(float l, float& E) {
  float s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(E) : "f"(-1.4426950408889634f * l));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + E));
  return s;
}

// s (1 - s); the minimum puts 1 - s = 1 where E is infinite (and s is 0).
RNX_DEVICE float slope_of(float s, float E) { return fminf(E * s, 1.f) * s; }

// Start of sequence b, clamped into [0, T] so that a wrong offset never leads
// outside the rows (offsets NULL: one sequence of T rows).
RNX_DEVICE int seq_start(const int32_t* off, int b, int T) {
  if (!off) return b > 0 ? T : 0;
  return min(max(*(off + b), 0), T);
}

// First sequence that ends behind `row` (B if none), found by a whole warp (row
// the same in all lanes): 32 probes at a time, so that up to 32 sequences take
// one load's latency and 1024 two.
RNX_DEVICE int seq_of_row(const int32_t* off, int B, int T, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;                              // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;   // the last of the lane's run
    const bool behind = at >= hi || seq_start(off, at + 1, T) > row;
    const unsigned hit = __ballot_sync(0xffffffffu, behind);
    if (hit == 0) return hi;
    const int i = __ffs(hit) - 1;
    hi = min(hi, lo + (i + 1) * step - 1);
    lo += i * step;
  }
  return lo;
}

// Sum over the G lanes of a row.
template <int G>
RNX_DEVICE float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows reach the registers through a ring of slots in shared memory, filled by
// cp.async DEPTH - 1 rows ahead (74 KB in flight per SM at E = 288, which
// covers the HBM latency; a second set of registers for the next row spilled).
// A slot is E logits rounded up to 4, then 16 ids and, backward, 16
// routing-weight gradients. Lane g of a row takes logits 4 (g + G q) + i; those behind the
// last expert (in the last quad alone, 4 G (NQ - 1) < E) are masked.
RNX_DEVICE void cp_async16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
RNX_DEVICE void cp_async4(float* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
RNX_DEVICE void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
RNX_DEVICE void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__host__ __device__ constexpr int padded(int E) { return (E + 3) / 4 * 4; }
__host__ __device__ constexpr int slot_floats(int E, bool weights) { return padded(E) + (weights ? 2 : 1) * kMaxK; }
template <int G, int NQ>
__host__ __device__ constexpr int ring_depth() { return NQ > 5 ? 2 : G == 4 ? 3 : 4; }

// Where lane g reads its quad q of a slot: the last quad's lanes behind the
// last expert read the row's last four again, so that no read leaves the slot.
template <int G, int NQ>
RNX_DEVICE int cell(int q, int g, int E) {
  const int c = 4 * (g + G * q);
  return q == NQ - 1 ? min(c, padded(E) - 4) : c;
}

template <int G, int NQ>
RNX_DEVICE void fill_slot(float* slot, const float* logits, const int32_t* ids, const float* weights, int E, int k,
                          int row, int g) {
  const float* src = logits + (size_t)row * E;
  if (E % 4 == 0) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int c = 4 * (g + G * q);
      if (q < NQ - 1 || c < E) cp_async16(slot + c, src + c);
    }
  } else {
    for (int c = g; c < E; c += G) cp_async4(slot + c, src + c);
  }
  float* tail = slot + padded(E);
  for (int j = g; j < k; j += G) {
    if (ids) cp_async4(tail + j, ids + (size_t)row * k + j);
    if (weights) cp_async4(tail + kMaxK + j, weights + (size_t)row * k + j);
  }
}

// A CTA's consecutive rows on their way through its rings: lane group j of warp
// w takes rows first + (w + 16 n) 32 / G + j. It runs on from one sequence to the
// next (starting anew at each cost 1 to 3 us of latency).
template <int G, int NQ>
struct RowStream {
  static constexpr int R = 32 / G, STEP = kSumWarps * R, DEPTH = ring_depth<G, NQ>();
  const float* logits;
  const int32_t* ids;
  float* ring;
  int E, k, end, base, at;    // base: first row of the warp's present group (warp-uniform), in slot `at`
  bool landed;

  RNX_DEVICE void fill(int d, int first) {
    const int lane = threadIdx.x & 31;
    // a lane group without a row left reads the last one again and adds nothing
    if (first < end) fill_slot<G, NQ>(ring + d * slot_floats(E, false), logits, ids, nullptr, E, k, min(first + lane / G, end - 1), lane % G);
    cp_commit();
  }
  RNX_DEVICE void start(const float* logits_, const int32_t* ids_, int E_, int k_, int first, int end_, float* rings) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    logits = logits_, ids = ids_, E = E_, k = k_, end = end_;
    ring = rings + (size_t)(warp * R + lane / G) * DEPTH * slot_floats(E, false);
    base = first + warp * R;
    at = 0;
    landed = false;
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d) fill(d, base + d * STEP);
  }
};

// Sums of the rows [lo, hi) of a stream by the whole CTA: normalised scores into
// sums[0 .. E) (fixed order: rows within a lane group, then the groups of a
// warp, then the warps) and assignment counts added to hist[0 .. E), which is
// zero and published before. warp_sums: kSumWarps * E floats. All threads call
// it; behind it thread t owns columns t + 512 i of both.
template <int G, int NQ>
RNX_DEVICE void sum_rows(RowStream<G, NQ>& st, int lo, int hi, float* warp_sums, int* hist) {
  constexpr int R = 32 / G, STEP = kSumWarps * R, DEPTH = ring_depth<G, NQ>();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane % G;
  const int E = st.E, k = st.k, slot = slot_floats(E, false), mine = lane / G;
  float acc[4 * NQ];
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) acc[i] = 0.f;
  while (st.base < hi) {
    if (!st.landed) {
      __syncwarp();                                      // the slot filled now was read one row ago
      st.fill(st.at == 0 ? DEPTH - 1 : st.at - 1, st.base + (DEPTH - 1) * STEP);
      cp_wait<DEPTH - 1>();
      __syncwarp();
    }
    const float* src = st.ring + st.at * slot;
    float s[4 * NQ], total = 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(src + cell<G, NQ>(q, g, E));
      const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float unused;
        float x = score_of(l[i], unused);
        if (q == NQ - 1 && 4 * (g + G * q) + i >= E) x = 0.f;
        s[4 * q + i] = x;
        total += x;
      }
    }
    total = row_sum<G>(total);
    const int row = st.base + mine;
    const bool exists = row >= lo && row < hi;
    if (st.base < lo || st.base + R > hi) {              // warp-uniform: rows of another sequence, NaN included
      if (!exists) {
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) s[i] = 0.f;
      }
    }
    const float inv = total == 0.f || !exists ? 0.f : 1.0f / total;      // a row of zero scores has no shares
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
    for (int j = g; j < k; j += G) {
      const int id = __float_as_int(src[padded(E) + j]);
      if (exists && id >= 0 && id < E) atomicAdd(hist + id, 1);          // integer: the order does not matter
    }
    st.landed = st.base + R > hi && hi < st.end;         // the next sequence takes the rest of this group
    if (st.landed) break;
    st.base += STEP;
    st.at = st.at == DEPTH - 1 ? 0 : st.at + 1;
  }
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    const int c = 4 * (g + G * (i / 4)) + i % 4;
    if (lane < G && c < E) warp_sums[warp * E + c] = acc[i];
  }
  __syncthreads();
  for (int e = tid; e < E; e += kSumWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) v += warp_sums[w * E + e];
    warp_sums[e] = v;                                    // only this thread reads or writes column e
  }
}
RNX_DEVICE void clear_counts(int* hist, int E) {
  for (int e = threadIdx.x; e < E; e += kSumWarps * 32) hist[e] = 0;
  __syncthreads();
}

// Shared memory of a summing CTA: rings, the warps' sums, the counts.
template <int G, int NQ>
__host__ __device__ constexpr size_t sum_ring_floats(int E) {
  return (size_t)kSumWarps * (32 / G) * ring_depth<G, NQ>() * slot_floats(E, false);
}
template <int G, int NQ>
constexpr size_t sum_smem(int E) { return 4 * (sum_ring_floats<G, NQ>(E) + ((size_t)kSumWarps + 1) * E); }

// One sequence's results from its column sums and counts (published in shared
// memory). n = T_b. red: 32 floats.
RNX_DEVICE void finish_sequence(const float* sums, const int* hist, int E, int k, int n, float coef, int32_t* counts,
                                float* mean, float* loss, float* red) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  const float fs = n > 0 ? (float)E / ((float)k * (float)n) : 0.f;
  float part = 0.f;
  for (int e = tid; e < E; e += blockDim.x) {
    const float p = sums[e] * inv_n;
    counts[e] = hist[e];
    mean[e] = p;
    part = fmaf((float)hist[e] * fs, p, part);
  }
  part = warp_sum(part);
  if (lane == 0) red[warp] = part;
  __syncthreads();
  if (warp == 0) {
    const float v = warp_sum(lane < (int)blockDim.x / 32 ? red[lane] : 0.f);
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
template <int G, int NQ>
__global__ void __launch_bounds__(kSumWarps * 32, 1) balance_seq_kernel(const BalanceParams p) {
  extern __shared__ __align__(16) float dyn[];
  __shared__ float red[32];
  float* warp_sums = dyn + sum_ring_floats<G, NQ>(p.E);
  int* hist = reinterpret_cast<int*>(warp_sums + (size_t)kSumWarps * p.E);
  const int b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int lo = seq_start(p.off, b, p.T), hi = max(lo, seq_start(p.off, b + 1, p.T));
  RowStream<G, NQ> rows;
  rows.start(p.logits, p.ids, p.E, p.k, lo, hi, dyn);
  clear_counts(hist, p.E);
  sum_rows(rows, lo, hi, warp_sums, hist);
  cp_wait<0>();
  __syncthreads();
  finish_sequence(warp_sums, hist, p.E, p.k, hi - lo, p.coef, p.counts + (size_t)b * p.E, p.mean + (size_t)b * p.E,
                  p.loss + b, red);
}

// Many tokens, step 1: CTA i sums rows [i R, (i + 1) R). It may meet several
// sequences; its part of sequence b goes to slot i + b, which is its own since
// both only grow.
template <int G, int NQ>
__global__ void __launch_bounds__(kSumWarps * 32, 1) balance_partial_kernel(const BalanceParams p) {
  extern __shared__ __align__(16) float dyn[];
  float* warp_sums = dyn + sum_ring_floats<G, NQ>(p.E);
  int* hist = reinterpret_cast<int*>(warp_sums + (size_t)kSumWarps * p.E);
  pdl_wait();
  pdl_trigger();
  const int r0 = (int)min((long long)blockIdx.x * p.rows_per_block, (long long)p.T);
  const int r1 = (int)min((long long)r0 + p.rows_per_block, (long long)p.T);
  RowStream<G, NQ> rows;
  rows.start(p.logits, p.ids, p.E, p.k, r0, r1, dyn);      // its latency beside the search
  clear_counts(hist, p.E);
  for (int b = seq_of_row(p.off, p.B, p.T, r0); b < p.B; ++b) {
    const int start = seq_start(p.off, b, p.T);
    if (start >= r1) break;
    const int lo = max(r0, start), hi = min(r1, seq_start(p.off, b + 1, p.T));
    if (lo >= hi) continue;
    sum_rows(rows, lo, hi, warp_sums, hist);
    const size_t slot = (size_t)(blockIdx.x + b) * p.E;
    for (int e = threadIdx.x; e < p.E; e += kSumWarps * 32) {   // as sum_rows left them to the threads
      p.psum[slot + e] = warp_sums[e];
      p.pcnt[slot + e] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
  }
  cp_wait<0>();
}

// Step 2: one CTA per sequence adds its slots in order. Warps split the slots
// into `parts` interleaved runs per group of 32 experts.
__global__ void __launch_bounds__(kJoinWarps * 32, 1) balance_join_kernel(const BalanceParams p) {
  extern __shared__ float dyn[];
  __shared__ float red[32];
  const int E = p.E, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (E + 31) / 32, parts = kJoinWarps / groups;   // E <= 1024: at least one part
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
  for (int x = tid; x < E; x += kJoinWarps * 32) {
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

// Both means are sums of products with scores that may be as small as 2^-126,
// divided by a sum of such scores: the other factor is raised for the sum by a
// power of two, and lowered again behind the division. Gradients of the weights
// are raised by 2^40 (from 2^-40 to 2^87 they keep their accuracy beside any
// score); loads f, at least 2^-22, by 2^24, which the balance loss's factor takes
// back (from 2^-102 on it is exact). Every gradient is formed as (slope / sum of
// scores) (upstream times difference): the first factor is at most 1, while the
// sum's reciprocal alone reaches 2^126.
constexpr float kRaise = 1099511627776.f, kLower = 1.f / kRaise;
constexpr float kRaiseLoad = 16777216.f, kLowerGain = 1.f / kRaiseLoad;

// G lanes per row, each warp a run of consecutive rows, so that the loads f of
// its sequence stay in registers. The routing weights' part of a row is k
// values: the row without them goes back to its slot, the slots' lanes add
// theirs, and the row is stored from there (testing each expert against k ids
// cost more instructions than everything else).
template <int G, int NQ>
__global__ void __launch_bounds__(kGradWarps * 32, 2) router_grad_kernel(const GradParams p) {
  constexpr int R = 32 / G, DEPTH = ring_depth<G, NQ>();
  constexpr int SL = G >= kMaxK ? 1 : kMaxK / G; // slots per lane: slot j + G h of lane j
  extern __shared__ __align__(16) float dyn[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G;
  const int E = p.E, k = p.k, slot = slot_floats(p.E, true), tail = padded(p.E);
  const bool vec = E % 4 == 0;
  float* ring = dyn + (size_t)(warp * R + lane / G) * DEPTH * slot;
  pdl_wait();
  pdl_trigger();
  const long long first = ((long long)blockIdx.x * kGradWarps + warp) * p.rows_per_warp;
  if (first >= p.T) return;
  const int r0 = (int)first, r1 = (int)min(first + p.rows_per_warp, (long long)p.T);
  const int32_t* ids = p.d_weights ? p.ids : nullptr;
  int base = r0;                                 // the warp's first row (warp-uniform)
  const int mine = lane / G;
  auto fill = [&](int d, int from) {
    if (from < r1) fill_slot<G, NQ>(ring + d * slot, p.logits, ids, p.d_weights, E, k, min(from + mine, r1 - 1), g);
    cp_commit();
  };
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fill(d, base + d * R);
  // this lane group's sequence [start, end), from the warp's first on; the
  // groups of a warp may be in different ones
  int b = seq_of_row(p.off, p.B, p.T, base);
  int start = b < p.B ? seq_start(p.off, b, p.T) : p.T, end = b < p.B ? seq_start(p.off, b + 1, p.T) : p.T;
  bool fresh = true;
  float f[4 * NQ], gain = 0.f;                   // f times 2^24, gain times 2^-24
#pragma unroll
  for (int i = 0; i < 4 * NQ; ++i) f[i] = 0.f;
  for (int at = 0; base < r1; base += R, at = at == DEPTH - 1 ? 0 : at + 1) {
    __syncwarp();                                // the slot filled now was read one row ago
    fill(at == 0 ? DEPTH - 1 : at - 1, base + (DEPTH - 1) * R);
    const int row = base + mine;
    while (b < p.B && row >= end) {              // the next sequence that holds rows behind this one
      ++b;
      start = end;
      if (b < p.B) end = max(end, seq_start(p.off, b + 1, p.T));
      fresh = true;
    }
    const bool inside = row < r1 && b < p.B && row >= start;   // others are left as they were
    if (inside && fresh && p.d_loss) {
      fresh = false;
      const float n = (float)(end - start);
      gain = p.d_loss[b] * p.coef / n * kLowerGain;
      const float fs = kRaiseLoad * ((float)E / ((float)k * n));
      const int32_t* count = p.counts + (size_t)b * E;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int c = 4 * (g + G * q);
        int4 v = make_int4(0, 0, 0, 0);
        if (vec) {
          if (q < NQ - 1 || c < E) v = *reinterpret_cast<const int4*>(count + c);
        } else {
          if (q < NQ - 1 || c < E) v.x = count[c];
          if (q < NQ - 1 || c + 1 < E) v.y = count[c + 1];
          if (q < NQ - 1 || c + 2 < E) v.z = count[c + 2];
          if (q < NQ - 1 || c + 3 < E) v.w = count[c + 3];
        }
        f[4 * q] = (float)v.x * fs, f[4 * q + 1] = (float)v.y * fs, f[4 * q + 2] = (float)v.z * fs, f[4 * q + 3] = (float)v.w * fs;
      }
    }
    cp_wait<DEPTH - 1>();
    __syncwarp();
    float* src = ring + at * slot;
    int id[SL];
    float d[SL];                                 // a slot's part of d logits
    if (p.d_weights) {
      float sc[SL], slope[SL], v[SL], c = 0.f, m = 0.f;
#pragma unroll
      for (int h = 0; h < SL; ++h) {
        const int j = g + G * h;
        const int e = inside && j < k ? __float_as_int(src[tail + j]) : -1;
        id[h] = e >= 0 && e < E ? e : -1;
        float ex;
        sc[h] = id[h] >= 0 ? score_of(src[id[h]], ex) : 0.f;
        slope[h] = id[h] >= 0 ? slope_of(sc[h], ex) : 0.f;
        v[h] = id[h] >= 0 ? src[tail + kMaxK + j] : 0.f;
        c += sc[h];
        m = fmaf(v[h], sc[h] * kRaise, m);
      }
      c = row_sum<G>(c);
      m = row_sum<G>(m);
      const float ic = c == 0.f ? 0.f : 1.0f / c;
      m *= ic * kLower;
#pragma unroll
      for (int h = 0; h < SL; ++h) d[h] = slope[h] * ic * (p.rsf * (v[h] - m));
      // An expert named in several slots gets their sum, in slot order, from
      // its first. Hardly ever: k ids in k lanes are compared with one match.
      bool twice = k > G;
      if (!twice) {
        const unsigned same = __match_any_sync(0xffffffffu, id[0] >= 0 ? mine << 16 | id[0] : -1 - lane);
        twice = __any_sync(0xffffffffu, same & (same - 1));
      }
      if (twice) {
        float sum[SL];
        bool lead[SL];
#pragma unroll
        for (int h = 0; h < SL; ++h) sum[h] = 0.f, lead[h] = true;
        for (int j = 0; j < k; ++j) {
          int ej = id[0];
          float dj = d[0];
#pragma unroll
          for (int h = 1; h < SL; ++h)
            if (j / G == h) ej = id[h], dj = d[h];
          ej = __shfl_sync(0xffffffffu, ej, j % G, G);
          dj = __shfl_sync(0xffffffffu, dj, j % G, G);
#pragma unroll
          for (int h = 0; h < SL; ++h) {
            sum[h] += ej == id[h] ? dj : 0.f;
            lead[h] = lead[h] && !(ej == id[h] && j < g + G * h);
          }
        }
#pragma unroll
        for (int h = 0; h < SL; ++h) {
          d[h] = sum[h];
          if (!lead[h]) id[h] = -1;
        }
      }
    }
    float l[4 * NQ], total = 0.f, dot = 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(src + cell<G, NQ>(q, g, E));
      l[4 * q] = v.x, l[4 * q + 1] = v.y, l[4 * q + 2] = v.z, l[4 * q + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) {
      float ex, s = score_of(l[i], ex);
      if (i >= 4 * NQ - 4 && 4 * (g + G * (NQ - 1)) + i % 4 >= E) s = 0.f;
      l[i] = slope_of(s, ex);
      total += s;
      dot = fmaf(f[i], s, dot);
    }
    total = row_sum<G>(total);
    dot = row_sum<G>(dot);
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    const float mean = dot * inv;
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) l[i] = l[i] * inv * (gain * (f[i] - mean));
    if (p.d_weights) {
      __syncwarp();                              // the slot's logits have been read
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int c = 4 * (g + G * q);
        if (q < NQ - 1 || c < E) *reinterpret_cast<float4*>(src + c) = make_float4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < SL; ++h)
        if (id[h] >= 0) src[id[h]] += d[h];
      __syncwarp();
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const float4 v = *reinterpret_cast<const float4*>(src + cell<G, NQ>(q, g, E));
        l[4 * q] = v.x, l[4 * q + 1] = v.y, l[4 * q + 2] = v.z, l[4 * q + 3] = v.w;
      }
    }
    if (inside) {
      float* dst = p.d_logits + (size_t)row * E;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int c = 4 * (g + G * q);
        if (q == NQ - 1 && c >= E) break;
        if (vec) {
          *reinterpret_cast<float4*>(dst + c) = make_float4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
        } else {
          dst[c] = l[4 * q];
          if (q < NQ - 1 || c + 1 < E) dst[c + 1] = l[4 * q + 1];
          if (q < NQ - 1 || c + 2 < E) dst[c + 2] = l[4 * q + 2];
          if (q < NQ - 1 || c + 3 < E) dst[c + 3] = l[4 * q + 3];
        }
      }
    }
  }
  cp_wait<0>();
}

// Lanes per row and quads per lane for E <= 1024 experts: at most 10 quads (40
// registers a row); `wide` asks for a warp per row, the shortest chain where
// there are no more rows than warps.
#define RNX_CASE(X, CALL, G, NQ) case X: CALL(G, NQ); break
#define RNX_BY_ROW(E, wide, CALL)                                \
  do {                                                           \
    if ((wide) || (E) > 640) {                                   \
      switch (((E) + 127) / 128) {                               \
        RNX_CASE(1, CALL, 32, 1);                                \
        RNX_CASE(2, CALL, 32, 2);                                \
        RNX_CASE(3, CALL, 32, 3);                                \
        RNX_CASE(4, CALL, 32, 4);                                \
        RNX_CASE(5, CALL, 32, 5);                                \
        RNX_CASE(6, CALL, 32, 6);                                \
        RNX_CASE(7, CALL, 32, 7);                                \
        default: CALL(32, 8);                                    \
      }                                                          \
    } else if ((E) > 320) {                                      \
      switch (((E) + 63) / 64) {                                 \
        RNX_CASE(6, CALL, 16, 6);                                \
        RNX_CASE(7, CALL, 16, 7);                                \
        RNX_CASE(8, CALL, 16, 8);                                \
        RNX_CASE(9, CALL, 16, 9);                                \
        default: CALL(16, 10);                                   \
      }                                                          \
    } else if ((E) <= 32) {                                      \
      switch (((E) + 15) / 16) {                                 \
        RNX_CASE(1, CALL, 4, 1);                                 \
        default: CALL(4, 2);                                     \
      }                                                          \
    } else {                                                     \
      switch (((E) + 31) / 32) {                                 \
        RNX_CASE(2, CALL, 8, 2);                                 \
        RNX_CASE(3, CALL, 8, 3);                                 \
        RNX_CASE(4, CALL, 8, 4);                                 \
        RNX_CASE(5, CALL, 8, 5);                                 \
        RNX_CASE(6, CALL, 8, 6);                                 \
        RNX_CASE(7, CALL, 8, 7);                                 \
        RNX_CASE(8, CALL, 8, 8);                                 \
        RNX_CASE(9, CALL, 8, 9);                                 \
        default: CALL(8, 10);                                    \
      }                                                          \
    }                                                            \
  } while (0)

template <int G, int NQ>
cudaError_t launch_sums(const BalanceParams& p, int blocks, cudaStream_t st) {
  static std::atomic<uint64_t> done[2];
  static_assert(sum_smem<G, NQ>(4 * G * NQ) <= kMaxDynamicSmem, "shared memory");
  const size_t smem = sum_smem<G, NQ>(p.E);
  auto kern = blocks ? balance_partial_kernel<G, NQ> : balance_seq_kernel<G, NQ>;
  const cudaError_t e = smem > 48 * 1024 ? allow_smem(kern, done[blocks > 0]) : cudaSuccess;
  return e != cudaSuccess ? e : launch_pdl(kern, dim3(blocks ? blocks : p.B), dim3(kSumWarps * 32), smem, st, p);
}

template <int G, int NQ>
cudaError_t launch_grad(GradParams p, cudaStream_t st) {
  constexpr int R = 32 / G;
  // one wave of 16 warps per SM; beyond that each warp takes a run of rows
  const int groups = (p.T + R - 1) / R, warps = kNumSMs * 2 * kGradWarps;
  p.rows_per_warp = R * max(1, (groups + warps - 1) / warps);
  const int rows = kGradWarps * p.rows_per_warp;
  const size_t smem = (size_t)kGradWarps * R * ring_depth<G, NQ>() * slot_floats(p.E, true) * 4;   // at most 102 KB
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = smem > 48 * 1024 ? allow_smem(router_grad_kernel<G, NQ>, done) : cudaSuccess;
  return e != cudaSuccess ? e : launch_pdl(router_grad_kernel<G, NQ>, dim3((p.T + rows - 1) / rows), dim3(kGradWarps * 32), smem, st, p);
}

}  // namespace

// One CTA per SM; at least a row per warp.
int balance_rows_per_block(int T) {
  return max(kSumWarps, (T + kNumSMs - 1) / kNumSMs);
}

int balance_blocks(int T, int E) {
  if (balance_one_launch(T, E)) return 0;
  const int r = balance_rows_per_block(T);
  return (T + r - 1) / r;
}

int balance_scratch_blocks(int T, int E) {
  return balance_one_launch(T, E) ? 0 : min(kNumSMs, (T + kSumWarps - 1) / kSumWarps);
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, int T, int E, int k, const int32_t* off,
                                int B, float coef, int32_t* counts, float* mean, float* loss, void* scratch,
                                cudaStream_t st) {
  const int blocks = balance_by_sequence(T, E, B) ? 0 : balance_blocks(T, E);
  float* psum = static_cast<float*>(scratch);
  BalanceParams p{logits, ids, off, T, E, k, B, balance_rows_per_block(T), coef, psum,
                  reinterpret_cast<int*>(psum + (size_t)(blocks + B) * E), counts, mean, loss};
  cudaError_t err = cudaSuccess;
#define CALL(G, NQ) err = launch_sums<G, NQ>(p, blocks, st)
  RNX_BY_ROW(E, T <= kSumWideT, CALL);
#undef CALL
  if (err != cudaSuccess || blocks == 0) return err;
  const int parts = kJoinWarps / ((E + 31) / 32);
  return launch_pdl(balance_join_kernel, dim3(B), dim3(kJoinWarps * 32), (size_t)parts * E * 8, st, p);
}

cudaError_t launch_router_grad(const float* logits, const int32_t* ids, int T, int E, int k, const float* d_weights,
                               float rsf, const int32_t* off, int B, float coef, const int32_t* counts,
                               const float* d_loss, float* d_logits, cudaStream_t st) {
  const GradParams p{logits, ids, d_weights, off, counts, d_loss, d_logits, T, E, k, B, 1, coef, rsf};
  cudaError_t err = cudaSuccess;
#define CALL(G, NQ) err = launch_grad<G, NQ>(p, st)
  RNX_BY_ROW(E, T <= kGradWideT, CALL);
#undef CALL
  return err;
}

}  // namespace rnx
