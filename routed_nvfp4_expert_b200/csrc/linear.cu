// BF16 linear layer with a fused epilogue, and its backward pass, on the
// 5th-generation tensor cores (tcgen05.mma kind::f16, fp32 accumulators in
// tensor memory).
//
//   z = x W^T + b,  y = act(z) + residual           x [T, K], W [N, K]
//   dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum_t dz
//
// All three products are D[m, j] = sum_r A[m, r] B[j, r]. An operand whose
// rows are contiguous along r is read K-major, one whose rows are contiguous
// along m (or j) MN-major; the shared-memory descriptors and two bits of the
// instruction descriptor say which, so no operand is ever transposed in
// memory:
//   forward  m = n (W, K-major),   j = t (x, K-major),   r = k
//   dx       m = k (W, MN-major),  j = t (dz, K-major),  r = n
//   dW       m = k (x, MN-major),  j = n (dz, MN-major), r = t
//
// dz is rounded to bf16, the tensor cores' operand type (half a step, at most 2^-8
// of each element; y, z, dx and dW take the same one rounding); db is summed in
// fp32 from the unrounded dz.

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tensor_map.h"

namespace rnx {

namespace {

// ---------------------------------------------------------------- activations

// The forward's epilogue evaluates 2^15 of these per CTA and tile beside the
// next tile's products, and the dz pass as many as it streams, so their
// instruction count matters: with normcdff, tanhf, expf and full divisions the
// epilogue took longer than the products (60% of the tensor pipe at 4096 x 4096
// x 12288, 83% now) and the dz pass of 4096 x 12288 was bound by them (now 50 to 56
// us for 46 us of HBM traffic). Everything is put on one power of two and one
// reciprocal (within 2^-22 each); GELU's normal tail is a fit of this file
// (normal_cdf). All values and slopes stay within 2^-20 of 1 + |z|, and the values
// within 2^-13 of themselves while Phi(z) or 1 / (1 + E) is above 2^-126, a
// sixteenth of bf16's half step or less (below that, from z = -13 in GELU, -10 in
// its tanh form and -87 in SiLU, they are 0). With E = 2^(-v log2 e) and s = 1 /
// (1 + E), 1 - s = E s; the minimum puts it to 1 where E is infinite and s is 0
// (another keeps z^2 finite beside a factor of 0).

RNX_DEVICE float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
RNX_DEVICE float recip(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
RNX_DEVICE void l2_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Two values rounded to bf16 in one instruction (lo in the low half).
RNX_DEVICE uint32_t pack2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Phi(z), with g = exp(-z^2 / 2): Phi(-|z|) = g t P(t), t = 1 / (1 + 0.29 |z|).
// P is the polynomial of degree 5 whose largest error over 0 <= |z| <= 14 is
// least, by linear programming on 800 Chebyshev points, where an error of Phi
// counts as twice itself or, where that is more, as a thousandth of its share of
// Phi: 4.5e-8 in all, 9e-5 of Phi in the tail. (Approximations of erfc that bound
// the error alone, 7.5e-8 with a polynomial shorter by one, are off by 1% of y at
// z = -8.)
RNX_DEVICE float normal_cdf(float z, float& g) {
  const float t = recip(fmaf(0.29f, fabsf(z), 1.f));
  float poly = fmaf(t, -0.088841276f, 0.284976389f);
  poly = fmaf(t, poly, -0.093334857f);
  poly = fmaf(t, poly, 0.179639302f);
  poly = fmaf(t, poly, 0.100685080f);
  poly = t * fmaf(t, poly, 0.116875408f);
  g = pow2(-0.72134752f * z * z);
  const float tail = poly * g;
  return z > 0.f ? 1.f - tail : tail;
}

template <int ACT>
RNX_DEVICE float act_of(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (ACT == MOE_ACT_GELU) {
    float g;
    return z * normal_cdf(z, g);
  }
  // (1 + tanh u) / 2 = 1 / (1 + e^-2u), 2 u log2 e = z (2.3022082 + 0.10294325 z^2)
  if (ACT == MOE_ACT_GELU_TANH) return z * recip(1.f + pow2(z * fmaf(-0.10294325f * z, z, -2.3022082f)));
  if (ACT == MOE_ACT_SILU) return z * recip(1.f + pow2(-1.442695041f * z));
  return z;
}

template <int ACT>
RNX_DEVICE float act_grad(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if (ACT == MOE_ACT_GELU) {                               // Phi(z) + z phi(z)
    float g;
    const float cdf = normal_cdf(z, g);
    return fmaf(z * 0.3989422804014327f, g, cdf);
  }
  if (ACT == MOE_ACT_GELU_TANH) {
    const float z2 = fminf(z * z, 1e30f), E = pow2(z * fmaf(-0.10294325f, z2, -2.3022082f)), s = recip(1.f + E);
    return fmaf(z * s * fminf(E * s, 1.f), fmaf(0.21406445f, z2, 1.5957691f), s);
  }
  if (ACT == MOE_ACT_SILU) {
    const float E = pow2(-1.442695041f * z), s = recip(1.f + E);
    return fmaf(z * s, fminf(E * s, 1.f), s);
  }
  return 1.f;
}

// ---------------------------------------------------------------- shared pieces

constexpr int kStepK = 64;                 // reduction elements per stage: 128 bytes per row (one swizzle span)
constexpr int kTileM = 128;
constexpr int kABytes = kTileM * 128;      // 16 KB; K-major: 128 rows; MN-major: two 64-wide blocks of 64 rows
constexpr int kMnBlock = 64 * 128;         // one MN-major block: 64 r rows of 128 bytes

// Position in a ring of stages: slot and the parity of its current pass.
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  RNX_DEVICE void next(int stages) {
    if (++slot == stages) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Bounded wait of a whole warp. A producer's loop is part of a stage's round
// trip (slot freed, copy issued, data, products, slot freed), and the ring
// just covers that trip, so the common case is one try and one vote; the abort
// flag is read only when the slot was not ready. limit_ns 0 gives up on a slot
// that is not ready at once (a try may hold the thread until it is).
RNX_DEVICE bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit_ns) {
  if (__all_sync(0xffffffffu, limit_ns ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_poll(bar, parity, limit_ns) && !*abort_flag);
}

// Waits (bounded) until the last `issued` copies of a producer that stopped at
// `at` have landed: one pass over the slots it filled.
RNX_DEVICE void ring_drain(uint64_t* full_bar, Ring at, int issued, int stages, uint32_t* status, int lane) {
  const int n = min(issued, stages);
  for (int i = 0; i < n; ++i) {
    if (--at.slot < 0) {
      at.slot = stages - 1;
      at.parity ^= 1u;
    }
    if (!mbar_wait(&full_bar[at.slot], at.parity) && lane == 0) set_status(status, kDevErrTimeout);
  }
}

// ---------------------------------------------------------------- unaligned rows
// Eight elements at p, of which `valid` belong to the row, by 16-byte loads.
// ANY: p on any element; the one or two aligned pieces that hold the elements
// are loaded here and shifted together in finish8. No piece is read that runs
// past `end`, the matrix's end: there load8 returns false and finish8 takes the
// elements one by one, as load8 without ANY does at a row's ragged end.
struct Load8 {
  uint4 lo, hi;
};
RNX_DEVICE uint4 load8_elements(const uint16_t* p, int valid) {
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < valid ? p[i] : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
template <bool ANY>
RNX_DEVICE bool load8(Load8& v, const uint16_t* p, int valid, const uint16_t* end) {
  if (!ANY) {
    if (valid >= 8) v.lo = *reinterpret_cast<const uint4*>(p);
    else v.lo = load8_elements(p, valid);
    return true;
  }
  if (valid <= 0) return false;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
  const bool two = (reinterpret_cast<uintptr_t>(p) & 15) + 2 * min(valid, 8) > 16;
  if (at + (two ? 32 : 16) > reinterpret_cast<uintptr_t>(end)) return false;
  v.lo = *reinterpret_cast<const uint4*>(at);
  v.hi = two ? *reinterpret_cast<const uint4*>(at + 16) : make_uint4(0u, 0u, 0u, 0u);
  return true;
}
// 16 of the 32 bytes lo, hi, from byte `shift` (even, below 16).
RNX_DEVICE uint4 shift16(const uint4& lo, const uint4& hi, uint32_t shift) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t a[6], b[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) a[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) b[i] = shift & 4 ? a[i + 1] : a[i];
  const uint32_t bits = 8 * (shift & 2);
  return make_uint4(__funnelshift_r(b[0], b[1], bits), __funnelshift_r(b[1], b[2], bits),
                    __funnelshift_r(b[2], b[3], bits), __funnelshift_r(b[3], b[4], bits));
}
template <bool ANY>
RNX_DEVICE uint4 finish8(const Load8& v, const uint16_t* p, int valid, bool loaded) {
  if (!ANY) return v.lo;
  if (!loaded) return load8_elements(p, valid);
  return shift16(v.lo, v.hi, (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15));
}

struct Epilogue {
  const uint16_t* bias;       // per output feature, nullable
  const uint16_t* residual;   // nullable
  uint16_t* z;                // pre-activation, nullable
  uint16_t* out;
  long long ldr, ldz, ldo;
  int vec;                    // rows of residual, z and out all start on 16-byte boundaries
};

// db from the column sums of the row chunks, by `units` warps: four lanes per
// column take every fourth chunk in order, then add theirs; a warp has four
// columns per lane group at work (eight columns in all left 7872 columns to 20
// rounds of memory latency in a launch of few CTAs: 10 us).
struct DbJoin {
  const float* part;          // [chunks, n]
  float* db;                  // nullable
  int chunks, n;
};
RNX_DEVICE void join_db(const DbJoin& d, int unit, int units, int lane) {
  if (!d.db) return;
  for (int c0 = unit * 32; c0 < d.n; c0 += units * 32) {    // warp-uniform
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const int c = c0 + lane / 4;
#pragma unroll 4
    for (int i = lane % 4; i < d.chunks; i += 4) {
      const float* src = d.part + (size_t)i * d.n + c;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (c + 8 * s < d.n) v[s] += src[8 * s];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v[s] += __shfl_xor_sync(0xffffffffu, v[s], 1);
      v[s] += __shfl_xor_sync(0xffffffffu, v[s], 2);
      if (c + 8 * s < d.n && lane % 4 == 0) d.db[c + 8 * s] = v[s];
    }
  }
}

// ---------------------------------------------------------------- split kernel
// One 128 x bn tile of D by a cluster of S CTAs that divide the reduction
// between them: few rows leave few tiles, and the weights' bytes should come
// in through every SM. Each CTA accumulates its part in tensor memory; CTA s
// then adds the S parts of its share of the j rows in rank order (so the result
// does not depend on timing), applies the epilogue and stores rows of out[j, m],
// 128 consecutive features per warp. Narrow tiles send their rows to the CTAs
// that finish them, as asynchronous stores counted on a barrier there, once all
// of the cluster have finished their products (a barrier without memory
// ordering); tiles above kPushColumns leave the part in their own shared memory
// for the others to read after an ordering barrier. (1 x 1024 x 1024: 3.8 us
// sent, 4.3 us read; 128 x 4096 x 4096, 128 columns: 16.2 us sent, 13.3 us
// read.) A barrier that each thread arrives at behind its last store, and waits
// for at its end, keeps every CTA until no peer has anything left to send it.
// Up to two products share a launch (dx and dW of few tokens); a reduction of
// fewer steps than S leaves the last ranks without a part of their own.
// Warps: 0 = TMA producer, 1 = MMA issuer, 2 = TMEM allocator, 3-7 = db join,
// 4-7 = TMEM readers; all eight reduce and store. Every wait is bounded; a
// timeout sets the status word, and the CTA still sends its (unspecified) part
// and meets its cluster's barriers.

constexpr int kSplitThreads = 256;
constexpr int kSplitMaxStages = 10;
constexpr int kMaxSplit = 8;               // the portable cluster size
constexpr int kPushColumns = 32;

struct SplitProblem {
  CUtensorMap tma_a, tma_b;
  Epilogue ep;
  int M, J;                   // D's extents
  int ksteps;                 // 64-element steps of the whole reduction
  int bn, stages;
  int mt, tiles;
  int a_mn, b_mn;
};
struct SplitParams {
  SplitProblem prob[2];
  DbJoin db;
  uint32_t* status;
  int tiles;                  // of all products
  int S, tmem_cols;
  int clear;
  unsigned long long wait_ns; // with LIMIT, of the ring's waits (the others keep the default)
};

// LIMIT: for a test's limit on the waits, which is in the way of every step as a
// parameter (T 777, 1000 -> 515 backward: 14.2 against 13.9 us).
template <int ACT, bool LIMIT>
__global__ void __launch_bounds__(kSplitThreads, 2) linear_split_kernel(const __grid_constant__ SplitParams p) {
  const unsigned long long wait_ns = LIMIT ? p.wait_ns : kWaitLimitNs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full_bar[kSplitMaxStages], empty_bar[kSplitMaxStages], mma_done, parts_bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.S, rank = (int)(blockIdx.x % (unsigned)S);
  int tile = (int)(blockIdx.x / (unsigned)S);
  const bool second = tile >= p.prob[0].tiles;
  const SplitProblem& q = p.prob[second];
  if (second) tile -= p.prob[0].tiles;
  const int jt = tile / q.mt, m0 = (tile - jt * q.mt) * kTileM, j0 = jt * q.bn;
  const int bn = q.bn, stages = q.stages;
  const int parts = min(S, q.ksteps);
  const bool push = bn <= kPushColumns;
  const int k_lo = rank < parts ? (int)((long long)q.ksteps * rank / parts) : 0;
  const int k_hi = rank < parts ? (int)((long long)q.ksteps * (rank + 1) / parts) : 0;
  const int stage_bytes = kABytes + bn * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&mma_done, 1);
    mbar_init(&parts_bar, 1);
    abort_flag = 0;
    fence_barrier_init();
    // the rows that this CTA finishes, from every part
    const int nj = min(bn, q.J - j0), per = (nj + S - 1) / S;
    const int rows = push ? max(0, min(nj, (rank + 1) * per) - rank * per) : 0;
    mbar_arrive_expect_tx(&parts_bar, (uint32_t)(parts * rows * kTileM * 4));
  }
  if (warp == 2) {
    tmem_alloc(&s_tmem, (uint32_t)p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();
  // the call's first launch clears the status word: its first CTA, and a wait
  // of another CTA that could set it runs out two seconds later at the earliest
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;

  if (warp == 0) {
    Ring r;
    int issued = 0;
    bool ok = true;
    for (int ks = k_lo; ks < k_hi; ++ks, ++issued, r.next(stages)) {
      if (!(ok = ring_wait(&empty_bar[r.slot], r.parity ^ 1u, &abort_flag, wait_ns))) break;
      if (elect_one()) {
        uint8_t* sA = smem + (size_t)r.slot * stage_bytes;
        uint8_t* sB = sA + kABytes;
        uint64_t* bar = &full_bar[r.slot];
        mbar_arrive_expect_tx(bar, (uint32_t)stage_bytes);
        if (q.a_mn) {
          tma_load_2d(sA, &q.tma_a, m0, ks * kStepK, bar);
          tma_load_2d(sA + kMnBlock, &q.tma_a, m0 + 64, ks * kStepK, bar);
        } else {
          tma_load_2d(sA, &q.tma_a, ks * kStepK, m0, bar);
        }
        if (q.b_mn) {
          for (int c = 0; c < bn; c += 64) tma_load_2d(sB + c * 128, &q.tma_b, j0 + c, ks * kStepK, bar);
        } else {
          tma_load_2d(sB, &q.tma_b, ks * kStepK, j0, bar);
        }
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      set_status(p.status, kDevErrTimeout);
      abort_flag = 1;
    }
    ring_drain(full_bar, r, issued, stages, p.status, lane);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_major(kTileM, bn, q.a_mn, q.b_mn);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t dA0 = q.a_mn ? sdesc_mn_sw128(s0, kMnBlock) : sdesc_k_sw128(s0);
    const uint64_t dB0 = q.b_mn ? sdesc_mn_sw128(s0 + kABytes, kMnBlock) : sdesc_k_sw128(s0 + kABytes);
    const uint64_t stepA = q.a_mn ? 2048 >> 4 : 32 >> 4, stepB = q.b_mn ? 2048 >> 4 : 32 >> 4;   // K = 16
    Ring r;
    bool ok = true;
    for (int ks = k_lo; ks < k_hi; ++ks, r.next(stages)) {
      if (!(ok = ring_wait(&full_bar[r.slot], r.parity, &abort_flag, wait_ns))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t so = (uint64_t)((uint32_t)(r.slot * stage_bytes) >> 4);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          mma_bf16(tmem, dA0 + so + kb * stepA, dB0 + so + kb * stepB, idesc, (ks > k_lo || kb > 0) ? 1u : 0u);
        mma_commit(&empty_bar[r.slot]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      set_status(p.status, kDevErrTimeout);
      abort_flag = 1;
    }
    if (elect_one()) mma_commit(&mma_done);
    __syncwarp();
    if (!mbar_wait_poll(&mma_done, 0) && lane == 0) set_status(p.status, kDevErrTimeout);
  } else if (warp >= 3) {
    join_db(p.db, (int)blockIdx.x * 5 + warp - 3, (int)gridDim.x * 5, lane);
  }

  // the producer and the issuer are through: every copy has been seen to land
  // and every MMA to end, on their barriers, so the stages may hold parts. No
  // peer stores into them before this CTA's threads, behind those waits, have
  // arrived at the cluster's barrier; it need not order memory, since what the
  // stores overwrite is complete.
  const int nj = min(bn, q.J - j0), per = (nj + S - 1) / S;
  float* part = reinterpret_cast<float*>(smem);            // push: [parts][per][128], else [nj][128]
  __syncthreads();
  if (push && S > 1) cluster_sync_relaxed();
  if (warp >= 4 && rank < parts) {
    tc_fence_after();
    const int qd = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(qd * 32) << 16);
    const uint32_t mine = smem_u32(part) + 4u * (uint32_t)(rank * per * kTileM + qd * 32 + lane);
    const uint32_t bar = smem_u32(&parts_bar);
    int to = 0, row = 0;                                   // destination of column j: row of CTA `to`
    for (int c = 0; c < nj; c += 16) {
      uint32_t v[16];
      tmem_ld16(tq + c, v);
      tmem_ld_wait();
      if (push) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i < nj) st_async(mapa_shared(mine + (uint32_t)(row * kTileM * 4), (uint32_t)to), v[i], mapa_shared(bar, (uint32_t)to));
          if (++row == per) row = 0, ++to;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kTileM + qd * 32 + lane] = __uint_as_float(v[i]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
  }
  __syncwarp();
  bool complete = true;
  if (push) {
    if (S > 1) cluster_arrive_relaxed();                   // this thread has nothing left to send
    complete = __all_sync(0xffffffffu, mbar_wait_cluster(&parts_bar, 0));
    if (!complete && lane == 0) set_status(p.status, kDevErrTimeout);
  } else if (S > 1) {
    cluster_sync_all();
  }

  // ---------------------------------------------------------------- join and epilogue
  // lane: four consecutive features where every row of z, residual and out
  // starts on 8 bytes, else features lane + 32 i (2-byte accesses that fill
  // whole sectors)
  const Epilogue& ep = q.ep;
  const int j_lo = rank * per, j_hi = min(nj, j_lo + per);
  const bool vec = ep.vec && m0 + kTileM <= q.M;
  const int first = vec ? 4 * lane : lane, step = vec ? 1 : 32;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (ep.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + first + step * i < q.M) bias[i] = bf16_bits_to_f32(ep.bias[m0 + first + step * i]);
#pragma unroll 2
  for (int j = j_lo + warp; j < j_hi; j += kSplitThreads / 32) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t at = smem_u32(part) + 4u * (uint32_t)((push ? j - j_lo : j) * kTileM + first);
    const long long row = j0 + j;
    const int m = m0 + first;
    uint32_t res[4] = {0u, 0u, 0u, 0u};                     // the residual's latency beside the parts'
    if (ep.residual) {
      const uint16_t* src = ep.residual + row * ep.ldr + m;
      if (vec) {
        const uint2 r = *reinterpret_cast<const uint2*>(src);
        res[0] = r.x << 16, res[1] = r.x & 0xFFFF0000u, res[2] = r.y << 16, res[3] = r.y & 0xFFFF0000u;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m + 32 * i < q.M) res[i] = (uint32_t)src[32 * i] << 16;
      }
    }
    float4 f[kMaxSplit];
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s) {                   // all in flight together
      if (s >= parts) continue;
      const uint32_t src = push || S == 1 ? at + (uint32_t)(s * per * kTileM * 4) : mapa_shared(at, (uint32_t)s);
      f[s] = vec ? ld_cluster_f4(src)
                 : make_float4(ld_cluster_f1(src), ld_cluster_f1(src + 128), ld_cluster_f1(src + 256), ld_cluster_f1(src + 384));
    }
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s)
      if (s < parts) v[0] += f[s].x, v[1] += f[s].y, v[2] += f[s].z, v[3] += f[s].w;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bias[i];
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = act_of<ACT>(v[i]);
    if (ep.residual)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += __uint_as_float(res[i]);
    if (vec) {
      if (ep.z) *reinterpret_cast<uint2*>(ep.z + row * ep.ldz + m) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
      *reinterpret_cast<uint2*>(ep.out + row * ep.ldo + m) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = m + 32 * i;
        if (c >= q.M) break;
        if (ep.z) ep.z[row * ep.ldz + c] = f32_to_bf16_bits(v[i]);
        ep.out[row * ep.ldo + c] = f32_to_bf16_bits(y[i]);
      }
    }
  }
  __syncwarp();
  if (S > 1) {   // no CTA leaves while a peer may still read its part, or send it one
    if (!push) cluster_arrive_relaxed();
    cluster_wait();
  }
  // what was sent by then is on its way at most
  if (!complete && !mbar_wait_cluster(&parts_bar, 0)) set_status(p.status, kDevErrTimeout);
}

// ---------------------------------------------------------------- pair kernel
// Many rows: 256 x bn tiles (bn = 256 or 128) on CTA pairs, out[m, n] with the
// token (or dW's row) on the accumulator's lanes. One persistent pair per two
// SMs walks the tiles; the even CTA issues M = 256 MMAs (cta_group::2) on
// operands both CTAs load, so each CTA brings its 128 rows of A and half of B.
// Two accumulators of 256 columns fill the tensor memory, so that one tile's
// epilogue runs beside the next tile's products.
//
// Up to two products share a launch: dx and dW depend on dz alone, and their
// tiles in one list leave one ragged last round instead of two.
// Warps: 0 and 3 = TMA producers of A and of B, 1 = MMA issuer (even CTA), 2 =
// TMEM allocator, then db join, 4-11 = epilogue (lane quadrant w % 4, half of the columns each):
// 64 columns at a time go through a swizzled 32-row box in shared memory, from
// which one tensor store writes them (the lanes' own stores where the pitch or N
// is no multiple of 8 elements).
// Every wait is bounded. No TMA load uses cluster multicast.

constexpr int kPairM = 256;
constexpr int kPairStages = 6;
constexpr int kPairBBytes = 128 * 128;                       // half of B's 256 rows
constexpr int kPairStageBytes = kABytes + kPairBBytes;       // 32 KB
constexpr int kFirstEpiWarp = 4, kEpiWarps = 8;
constexpr int kPairThreads = (kFirstEpiWarp + kEpiWarps) * 32;
constexpr int kEpiBox = 32 * 128;
constexpr int kPairSmem = kPairStages * kPairStageBytes + kEpiWarps * kEpiBox + 1024;
constexpr uint32_t kPairTmemCols = 512;
constexpr int kRaster = 16;                                  // m tiles per raster group
static_assert(kPairSmem <= kMaxDynamicSmem, "shared memory");

struct PairProblem {
  CUtensorMap tma_a, tma_b;
  CUtensorMap tma_out, tma_z;  // of the output and z where rows and N allow it (ep.vec): box 64 x 32 rows
  Epilogue ep;
  int M, N;
  int ksteps;
  int a_mn, b_mn;
  int mt, nt;                 // tiles
};
struct PairParams {
  PairProblem prob[2];
  DbJoin db;
  uint32_t* status;
  int bn;
  int tiles0, tiles1;         // tiles of the two products (0: absent)
  int rounds1;                // rounds of the second product in which every pair takes a tile; behind them
                              // only pairs with fewer tiles of the first do (pairs >= first_light)
  int first_light;
  int clear;
  unsigned long long wait_ns; // with LIMIT, of the main-loop waits (the others keep the default)
};

// The i-th tile of a pair: first the first product's, round robin, then the
// second's. Returns false behind the last.
struct PairTile {
  int which, index;
};
RNX_DEVICE bool pair_tile(const PairParams& p, int pair, int n_pairs, int i, PairTile& t) {
  const int n0 = pair < p.tiles0 ? (p.tiles0 - pair + n_pairs - 1) / n_pairs : 0;
  if (i < n0) {
    t.which = 0;
    t.index = pair + i * n_pairs;
    return true;
  }
  const int r = i - n0;
  t.which = 1;
  if (r < p.rounds1) {
    t.index = r * n_pairs + pair;
  } else {
    if (pair < p.first_light) return false;
    t.index = p.rounds1 * n_pairs + (r - p.rounds1) * (n_pairs - p.first_light) + pair - p.first_light;
  }
  return t.index < p.tiles1;
}

// Groups of kRaster m tiles, n across: the tiles at work at any time share a
// few rows of A and of B, which then come from L2.
RNX_DEVICE void pair_tile_coords(const PairProblem& q, int index, int& mt, int& nt) {
  const int per = kRaster * q.nt;
  const int g = index / per, in = index - g * per;
  const int rows = min(kRaster, q.mt - g * kRaster);
  nt = in / rows;
  mt = g * kRaster + (in - nt * rows);
}

// A warp's box of 32 rows x 64 bf16: 16-byte chunk c of row r at position
// c ^ (r & 7), so that a lane walking its own row and eight lanes walking one
// row both reach all banks.
RNX_DEVICE uint8_t* box_at(uint8_t* box, int row, int chunk) { return box + row * 128 + ((chunk ^ (row & 7)) << 4); }

RNX_DEVICE uint16_t* box_elem(uint8_t* box, int row, int col) {
  return reinterpret_cast<uint16_t*>(box_at(box, row, col >> 3)) + (col & 7);
}

// A box to rows that no tensor map describes: eight lanes per row, the aligned
// 16-byte pieces inside it, then the elements before the first (up to 7) and
// behind the last. (4096 x 640 -> 4691 with residual: 215 us by elements, 58 us
// by pieces; words of two columns, for even pitches, gain 5% without a residual
// and lose 11% with one.)
template <int UNROLL>
RNX_DEVICE void box_store_pieces(uint8_t* box, uint16_t* out, long long ld, int rows, int cols, int lane) {
  const int l = lane & 7;
  uint16_t* p = out + (lane >> 3) * ld;
#pragma unroll UNROLL
  for (int r = lane >> 3; r < rows; r += 4, p += 4 * ld) {
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / 2, from = head + 8 * l;
    const int tail = (cols < head ? cols : head + ((cols - head) & ~7)) + l;
    const uint4 piece = shift16(*reinterpret_cast<const uint4*>(box_at(box, r, l)),
                                *reinterpret_cast<const uint4*>(box_at(box, r, (l + 1) & 7)), 2 * head);
    const uint16_t before = *box_elem(box, r, l), behind = *box_elem(box, r, min(tail, 63));
    if (from + 8 <= cols) *reinterpret_cast<uint4*>(p + from) = piece;
    if (l < head && l < cols) p[l] = before;
    if (tail < cols) p[tail] = behind;
  }
}

// The box to global memory at column col0, row row0 (whole warp): one tensor
// store, which ends at the tensor's edges by itself, or rows x cols elements
// where the pitch rules a tensor map out. Before the box is written again:
// box_free().
template <int UNROLL>
RNX_DEVICE void box_store(uint8_t* box, const CUtensorMap* map, uint16_t* out, long long ld, int row0, int col0, int rows,
                          int cols, int vec, int lane) {
  if (vec) {
    fence_proxy_async_smem();                 // the lanes' writes, visible to the tensor store
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, col0, row0, box);
      bulk_commit_group();
    }
  } else {
    __syncwarp();
    box_store_pieces<UNROLL>(box, out + row0 * ld + col0, ld, rows, cols, lane);
  }
}
RNX_DEVICE void box_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}

// The residual's box, in flight in registers (vec) while the accumulator is
// waited for.
struct BoxLoad {
  uint4 v[8];
};
RNX_DEVICE void box_issue(BoxLoad& b, const uint16_t* src, long long ld, int rows, int cols, int lane) {
  const int c = lane & 7, left = cols - 8 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    b.v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && left > 0) b.v[i] = *reinterpret_cast<const uint4*>(src + r * ld + 8 * c);
  }
}
RNX_DEVICE void box_land(const BoxLoad& b, uint8_t* box, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(box_at(box, 4 * i + (lane >> 3), lane & 7)) = b.v[i];
  __syncwarp();
}
// The same from rows on any element, straight into the box. `end`: the matrix's.
constexpr int kBoxRows = 2, kBoxUnroll = 2;
RNX_DEVICE void box_load_any(uint8_t* box, const uint16_t* src, long long ld, int rows, int cols, const uint16_t* end,
                             int lane) {
  const int c = lane & 7;
#pragma unroll 1
  for (int r0 = lane >> 3; r0 < 32; r0 += 4 * kBoxRows) {
    Load8 v[kBoxRows];
    bool loaded[kBoxRows];
#pragma unroll
    for (int i = 0; i < kBoxRows; ++i) {
      const int r = r0 + 4 * i;
      loaded[i] = load8<true>(v[i], src + r * ld + 8 * c, r < rows ? cols - 8 * c : 0, end);
    }
#pragma unroll
    for (int i = 0; i < kBoxRows; ++i) {
      const int r = r0 + 4 * i;
      *reinterpret_cast<uint4*>(box_at(box, r, c)) =
          finish8<true>(v[i], src + r * ld + 8 * c, r < rows ? cols - 8 * c : 0, loaded[i]);
    }
  }
  __syncwarp();
}

template <int ACT, bool LIMIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairParams p) {
  const unsigned long long wait_ns = LIMIT ? p.wait_ns : kWaitLimitNs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full_bar[kPairStages], empty_bar[kPairStages];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int abort_flag;              // of both CTAs: set in each by whoever stops
  __shared__ volatile int s_issued[4];             // steps by A and B of the even, then of the odd CTA

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int half = p.bn / 2;                       // this CTA's rows of B

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&mma_done, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(&s_tmem, kPairTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;   // as in the split kernel

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ TMA producers (both CTAs)
    const bool is_a = warp == 0;
    Ring r;
    int issued = 0;
    bool ok = true;
    PairTile t;
    for (int i = 0; ok && pair_tile(p, pair, n_pairs, i, t); ++i) {
      const PairProblem& q = p.prob[t.which];
      int mt, nt;
      pair_tile_coords(q, t.index, mt, nt);
      const CUtensorMap* map = is_a ? &q.tma_a : &q.tma_b;
      const int first = is_a ? mt * kPairM + 128 * (int)rank : nt * p.bn + half * (int)rank;   // row of the operand
      const int ksteps = q.ksteps;
      const bool mn = is_a ? q.a_mn : q.b_mn;
      const bool two = is_a || half > 64;          // MN-major blocks are 64 wide
      const bool expects = is_a && rank == 0;
      for (int ks = 0; ks < ksteps; ++ks, ++issued, r.next(kPairStages)) {
        if (!(ok = ring_wait(&empty_bar[r.slot], r.parity ^ 1u, &abort_flag, wait_ns))) break;
        if (elect_one()) {
          uint8_t* dst = smem + r.slot * kPairStageBytes + (is_a ? 0 : kABytes);
          const uint32_t bar = mapa_shared(smem_u32(&full_bar[r.slot]), 0);
          if (expects) mbar_arrive_expect_tx(&full_bar[r.slot], 2u * (uint32_t)(kABytes + half * 128));
          if (mn) {
            tma_load_2d_pair(dst, map, first, ks * kStepK, bar);
            if (two) tma_load_2d_pair(dst + kMnBlock, map, first + 64, ks * kStepK, bar);
          } else {
            tma_load_2d_pair(dst, map, ks * kStepK, first, bar);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) stop_pair(p.status, &abort_flag);
      s_issued[2 * rank + !is_a] = issued;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0) {
      const uint32_t s0 = smem_u32(smem);
      Ring r;
      int tc = 0;
      bool ok = true;
      PairTile t;
      for (int i = 0; ok && pair_tile(p, pair, n_pairs, i, t); ++i, ++tc) {
        const PairProblem& q = p.prob[t.which];
        const uint32_t idesc = idesc_bf16_major(kPairM, p.bn, q.a_mn, q.b_mn);
        const uint64_t dA0 = q.a_mn ? sdesc_mn_sw128(s0, kMnBlock) : sdesc_k_sw128(s0);
        const uint64_t dB0 = q.b_mn ? sdesc_mn_sw128(s0 + kABytes, kMnBlock) : sdesc_k_sw128(s0 + kABytes);
        const uint64_t stepA = q.a_mn ? 2048 >> 4 : 32 >> 4, stepB = q.b_mn ? 2048 >> 4 : 32 >> 4;
        const int b = tc & 1, ksteps = q.ksteps;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[b], ((uint32_t)(tc >> 1) & 1u) ^ 1u, wait_ns)))) break;
        tc_fence_after();
        const uint32_t acc = tmem + 256u * b;
        for (int ks = 0; ks < ksteps; ++ks, r.next(kPairStages)) {
          if (!(ok = ring_wait(&full_bar[r.slot], r.parity, &abort_flag, wait_ns))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t so = (uint64_t)((uint32_t)(r.slot * kPairStageBytes) >> 4);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
              mma_bf16_pair(acc, dA0 + so + kb * stepA, dB0 + so + kb * stepB, idesc, (ks > 0 || kb > 0) ? 1u : 0u);
            mma_commit_pair_mc(&empty_bar[r.slot], 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair_mc(&acc_full[b], 0x3);
        __syncwarp();
      }
      if (!ok && lane == 0) stop_pair(p.status, &abort_flag);
      if (elect_one()) mma_commit_pair_mc(&mma_done, 0x1);
      __syncwarp();
      if (!mbar_wait(&mma_done, 0) && lane == 0) set_status(p.status, kDevErrTimeout);
    }
  } else if (warp == 2) {
    join_db(p.db, blockIdx.x, gridDim.x, lane);
  } else if (warp >= kFirstEpiWarp) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int qd = warp & 3, ch = (warp - kFirstEpiWarp) >> 2;
    const uint32_t acc_empty_even[2] = {mapa_shared(smem_u32(&acc_empty[0]), 0), mapa_shared(smem_u32(&acc_empty[1]), 0)};
    uint8_t* box = smem + (size_t)kPairStages * kPairStageBytes + (size_t)(warp - kFirstEpiWarp) * kEpiBox;
    const int chunks = half / 64;                  // 64-column chunks of this warp
    int tc = 0;
    PairTile t;
    for (int i = 0; pair_tile(p, pair, n_pairs, i, t); ++i, ++tc) {
      const PairProblem& q = p.prob[t.which];
      const Epilogue& ep = q.ep;
      int mt, nt;
      pair_tile_coords(q, t.index, mt, nt);
      const int b = tc & 1;
      const int row0 = mt * kPairM + 128 * (int)rank + qd * 32;
      const int rows = min(32, q.M - row0);        // <= 0: none of this warp's rows exist
      bool gone = false;
      if (ep.residual && !ep.vec && lane < rows) { // loaded late, in batches: into L2 beside the products
        const uint16_t* r = ep.residual + (row0 + lane) * ep.ldr;
        const int c0 = nt * p.bn + half * ch, c1 = min(q.N, c0 + half);
        for (int c = c0; c < c1; c += 64) l2_prefetch(r + c);
        if (c0 < c1) l2_prefetch(r + c1 - 1);
      }
      for (int c = 0; c < chunks; ++c) {
        const int col0 = nt * p.bn + half * ch + 64 * c, cols = min(64, q.N - col0);
        BoxLoad res;
        const uint16_t* res_src = ep.residual ? ep.residual + row0 * ep.ldr + col0 : nullptr;
        if (res_src && ep.vec) box_issue(res, res_src, ep.ldr, rows, cols, lane);
        if (c == 0) {
          if (__any_sync(0xffffffffu, !mbar_wait_poll(&acc_full[b], (uint32_t)(tc >> 1) & 1u, wait_ns) || abort_flag)) {
            gone = true;
            break;
          }
          tc_fence_after();
        }
        uint32_t v[64];
        const uint32_t tq = tmem + 256u * b + ((uint32_t)(qd * 32) << 16) + half * ch + 64 * c;
        tmem_ld32(tq, v);
        tmem_ld32(tq + 32, v + 32);
        tmem_ld_wait();
        if (c == chunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_even[b]);
        }
        if (rows <= 0 || cols <= 0) continue;
        if (ep.bias) {
#pragma unroll
          for (int j = 0; j < 64; j += 8) {        // the same 16 bytes for every lane
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (j + 8 <= cols) {
              const uint4 u = *reinterpret_cast<const uint4*>(ep.bias + col0 + j);
              w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (j + e < cols) w[e >> 1] |= (uint32_t)ep.bias[col0 + j + e] << (16 * (e & 1));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = bf16x2_to_f32x2(w[e]);
              v[j + 2 * e] = __float_as_uint(__uint_as_float(v[j + 2 * e]) + f.x);
              v[j + 2 * e + 1] = __float_as_uint(__uint_as_float(v[j + 2 * e + 1]) + f.y);
            }
          }
        }
        box_free(lane);                            // the previous chunk's store has read the box
        if (ep.z) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(box_at(box, lane, j)) =
                make_uint4(pack2(__uint_as_float(v[8 * j]), __uint_as_float(v[8 * j + 1])),
                           pack2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3])),
                           pack2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5])),
                           pack2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7])));
          box_store<1>(box, &q.tma_z, ep.z, ep.ldz, row0, col0, rows, cols, ep.vec, lane);
          box_free(lane);
        }
        if (res_src) {
          if (ep.vec) box_land(res, box, lane);
          else box_load_any(box, res_src, ep.ldr, rows, cols, ep.residual + (q.M - 1) * ep.ldr + q.N, lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4* at = reinterpret_cast<uint4*>(box_at(box, lane, j));
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = act_of<ACT>(__uint_as_float(v[8 * j + e]));
          if (res_src) {
            const uint4 u = *at;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = bf16x2_to_f32x2(w[e]);
              y[2 * e] += f.x, y[2 * e + 1] += f.y;
            }
          }
          *at = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]),
                           pack2(y[6], y[7]));
        }
        box_store<kBoxUnroll>(box, &q.tma_out, ep.out, ep.ldo, row0, col0, rows, cols, ep.vec, lane);
      }
      if (gone) {
        if (lane == 0) stop_pair(p.status, &abort_flag);
        break;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  // no CTA leaves (or frees TMEM) while the pair's MMAs or copies may still
  // touch its shared or tensor memory; without an abort the products have
  // consumed every copy
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (abort_flag) {                                // the same in all threads of both CTAs
    const uint32_t b_bytes = (uint32_t)half * 128u, bytes[4] = {kABytes, b_bytes, kABytes, b_bytes};
    pair_drain<4, kPairStages>(rank, full_bar, s_issued, bytes, p.status);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmemCols);
  }
}

// ---------------------------------------------------------------- row pitch
// Rows whose pitch is not a multiple of 16 bytes cannot be a TMA operand; they
// are copied to a pitch that is (columns behind the last are never read: the
// tensor map ends at `cols`). Up to two operands in one launch: the forward's
// first, or CTAs behind those of the backward's dz pass.
struct PackJob {
  const uint16_t* src;
  uint16_t* dst;
  long long ld_src, ld_dst;
  int rows, cols;
  unsigned items;      // 256-column pieces, set by launch_pack
};
struct PackParams {
  PackJob job[2];
  int n;
  uint32_t* clear;     // status word (the pack is the call's first launch)
};
// A warp per 256 columns of a row (fewer than 2^31 of those fit the device),
// two such pieces in flight; CTAs of eight warps.
constexpr int kPackItems = 2;
RNX_DEVICE void pack_rows(const PackParams& p, unsigned cta, unsigned ctas) {
  const int lane = threadIdx.x & 31;
  const unsigned first = p.job[0].items, items = first + p.job[1].items, step = ctas * 8;
  for (unsigned at = cta * 8 + (threadIdx.x >> 5); at < items; at += kPackItems * step) {
    Load8 v[kPackItems];
    const uint16_t* s[kPackItems];
    uint16_t* d[kPackItems];
    int valid[kPackItems];
    bool loaded[kPackItems];
#pragma unroll
    for (int k = 0; k < kPackItems; ++k) {
      const unsigned it = at + k * step;
      valid[k] = 0;
      if (it >= items) continue;
      const PackJob& j = p.job[it >= first];
      const unsigned i = it >= first ? it - first : it, chunks = (j.cols + 255) / 256, r = i / chunks;
      const int c = 256 * (int)(i - r * chunks) + 8 * lane;
      s[k] = j.src + r * j.ld_src + c;
      d[k] = j.dst + r * j.ld_dst + c;
      valid[k] = j.cols - c;
      loaded[k] = load8<true>(v[k], s[k], valid[k], j.src + (j.rows - 1) * j.ld_src + j.cols);
    }
#pragma unroll
    for (int k = 0; k < kPackItems; ++k)
      if (valid[k] > 0) *reinterpret_cast<uint4*>(d[k]) = finish8<true>(v[k], s[k], valid[k], loaded[k]);
  }
}
__global__ void __launch_bounds__(256) pack_rows_kernel(const __grid_constant__ PackParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0u;
  pack_rows(p, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- dz and db
// dz = dy act'(z) in bf16 and the column sums of each chunk of rows in fp32
// (rows of a warp in order, then the warps). A CTA owns 256 columns of one
// chunk, eight consecutive ones per lane; a warp has four rows' loads in flight
// together (ANY, rows off 16 bytes: two rows of twice the loads). HBM-bound:
// 6 T N bytes (dy, z, dz). The CTAs behind `strips` x chunks copy operands.
constexpr int kDzRows = 4;

RNX_DEVICE void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = bf16x2_to_f32x2(w[i]);
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}

template <int ACT, bool ANY>
__global__ void __launch_bounds__(256, ANY ? 3 : 4) linear_dz_kernel(const uint16_t* dy, long long lddy, const uint16_t* z,
                                                        long long ldz, int T, int N, int rows_per_cta, uint16_t* dz,
                                                        long long lddz, float* db_part, uint32_t* clear,
                                                        unsigned strips, unsigned ctas,
                                                        const __grid_constant__ PackParams pk) {
  constexpr int kRows = ANY ? kDzRows / 2 : kDzRows;
  __shared__ float red[8][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned chunk = blockIdx.x / strips, strip = blockIdx.x - chunk * strips;
  const int c0 = strip * 256 + 8 * lane, valid = N - c0;
  const int r0 = chunk * rows_per_cta, r1 = min(T, r0 + rows_per_cta);
  const uint16_t *dy_end = dy + (T - 1) * lddy + N, *z_end = z + (T - 1) * ldz + N;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  pdl_wait();
  pdl_trigger();
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0u;
  if (blockIdx.x >= ctas) {
    pack_rows(pk, blockIdx.x - ctas, gridDim.x - ctas);
    return;
  }
  for (int base = r0 + warp; valid > 0 && base < r1; base += 8 * kRows) {
    Load8 u[kRows], uz[kRows];
    bool got[kRows], got_z[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = base + 8 * k;
      if (r >= r1) continue;
      got[k] = load8<ANY>(u[k], dy + r * lddy + c0, valid, dy_end);
      if (ACT != MOE_ACT_NONE) got_z[k] = load8<ANY>(uz[k], z + r * ldz + c0, valid, z_end);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = base + 8 * k;
      if (r >= r1) break;
      float g[8], a[8];
      unpack8(finish8<ANY>(u[k], dy + r * lddy + c0, valid, got[k]), g);
      if (ACT != MOE_ACT_NONE) unpack8(finish8<ANY>(uz[k], z + r * ldz + c0, valid, got_z[k]), a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (ACT != MOE_ACT_NONE) g[i] *= act_grad<ACT>(a[i]);
        acc[i] += g[i];
      }
      // whole pieces: dz's rows are padded to them, and the padding is never read
      if (dz)
        *reinterpret_cast<uint4*>(dz + r * lddz + c0) = make_uint4(pack2(g[0], g[1]), pack2(g[2], g[3]),
                                                                   pack2(g[4], g[5]), pack2(g[6], g[7]));
    }
  }
  if (!db_part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[warp][8 * lane + i] = acc[i];
  __syncthreads();
  const int c = strip * 256 + threadIdx.x;
  if (c < N) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][threadIdx.x];
    db_part[(size_t)chunk * N + c] = v;
  }
}

// db of a call that wants nothing else.
__global__ void __launch_bounds__(32) linear_db_kernel(const DbJoin d) {
  pdl_wait();
  pdl_trigger();
  join_db(d, blockIdx.x, gridDim.x, threadIdx.x);
}

// ---------------------------------------------------------------- host side

// One operand of a product: `rows` x `red` elements (red = the reduction).
// mn: memory is [red, rows] with pitch ld, else [rows, red].
struct Operand {
  const uint16_t* p;
  long long ld;
  int rows;
  bool mn;
};

bool operand_map(CUtensorMap* m, const Operand& o, int red, int box_rows) {
  const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (o.mn)
    return make_tensor_map_2d(m, o.p, t, 2, (uint64_t)o.rows, (uint64_t)red, 64, kStepK, CU_TENSOR_MAP_SWIZZLE_128B,
                              (uint64_t)o.ld);
  return make_tensor_map_2d(m, o.p, t, 2, (uint64_t)red, (uint64_t)o.rows, kStepK, (uint32_t)box_rows,
                            CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)o.ld);
}

// One product out[m, n] = epilogue(sum_r A[m, r] B[n, r]), row m of the output
// contiguous along n.
struct Product {
  Operand a, b;
  int red;
  Epilogue ep;
};

template <int ACT, bool LIMIT = false>
cudaError_t launch_split_act(const SplitParams& p, int smem, cudaStream_t st) {
  if (!LIMIT && p.wait_ns != kWaitLimitNs) return launch_split_act<ACT, true>(p, smem, st);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_split_kernel<ACT, LIMIT>, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.S * p.tiles));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePriority;
  attr[1].val.priority = launch_priority_high();
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = p.S;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<ACT, LIMIT>, p);
}

// ---------------------------------------------------------------- choice of kernel and tiles
// Estimated times in microseconds at 1.9 GHz, fitted to 90 measured
// combinations of shape (1 to 5000 tokens, 256 to 12288 features), tile width
// and split. On 32 random shapes of up to 3000 tokens the choices by them took
// 1.5% longer on average, 24% at most, than the best of the forms measured.
// What they weigh: narrow tiles and deep splits use more SMs but stream A more
// often and fill more than one wave; the pair kernel reads least and overlaps
// its epilogue but needs many tiles.

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

struct SplitPlan {
  double us;
  int S;
  int bn[2];
};

// CTAs of clusters of S that are resident together, for tiles of up to 64
// columns (two CTAs per SM) or wider.
int split_capacity(bool two, int S) {
  return two ? (S <= 2 ? 296 : S == 4 ? 264 : 256) : (S <= 2 ? 148 : S == 4 ? 136 : 112);
}

int tile_width(const Product& q, int most) {
  const int J = q.a.rows, unit = q.a.mn ? 64 : 16;           // MN-major blocks are 64 wide
  const long long jt = ceil_div(J, most);
  return (int)(ceil_div(ceil_div(J, jt), unit) * unit);
}

SplitPlan plan_split(const Product* prod, int n) {
  SplitPlan best{};
  best.us = -1;
  for (int most = 256; most >= 16; most /= 2) {
    if (most < 64 && (prod[0].a.mn || (n > 1 && prod[1].a.mn))) break;
    if (most < 32 && prod[0].a.rows > 16) break;
    int bn[2] = {0, 0}, widest = 0;
    long long tiles = 0;
    for (int i = 0; i < n; ++i) {
      bn[i] = tile_width(prod[i], most);
      widest = std::max(widest, bn[i]);
      tiles += ceil_div(prod[i].b.rows, kTileM) * ceil_div(prod[i].a.rows, bn[i]);
    }
    const bool two = widest <= 64;
    for (int S = 1; S <= kMaxSplit; S *= 2) {
      const int cap = split_capacity(two, S);
      const bool shared = two && tiles * S > kNumSMs;        // two CTAs share an SM's bandwidth
      const double busy = std::min(1.0, (double)tiles * S / kNumSMs);
      const double kb_us = two ? (shared ? 0.0225 : 0.0126) : 0.0085 + 0.0021 * busy;
      double longest = 0, sum = 0;
      for (int i = 0; i < n; ++i) {
        const long long t = ceil_div(prod[i].b.rows, kTileM) * ceil_div(prod[i].a.rows, bn[i]);
        const double kb = 16 + bn[i] / 8.0, steps = (double)ceil_div(ceil_div(prod[i].red, kStepK), S);
        const double us = steps * kb * kb_us + 0.0196 * bn[i] + 0.0197 * bn[i] / S + 2.85;
        longest = std::max(longest, us);
        sum += us * t / tiles;
      }
      const long long waves = ceil_div(tiles * S, cap);
      const double us = 0.9 + (waves == 1 ? longest : std::max(longest, waves * sum));
      if (best.us < 0 || us < best.us) best = SplitPlan{us, S, {bn[0], bn[1]}};
    }
  }
  return best;
}

// How the pairs share two products' tiles: each pair takes `rounds1` tiles of
// the second behind its own of the first, then those with a tile less of the
// first (from first_light on) go on alone. cost: of a tile; `end` in its units.
struct PairSchedule {
  double end;
  int rounds1, first_light;
};
PairSchedule schedule_pairs(const long long* tiles, const double* cost, int pairs) {
  const long long each = tiles[0] / pairs, heavy = tiles[0] % pairs, light = pairs - heavy;
  PairSchedule best{-1, 0, (int)heavy};
  auto end_of = [&](long long q) {
    const long long rest = std::max<long long>(0, tiles[1] - q * pairs);
    return std::max((each + (heavy > 0)) * cost[0] + q * cost[1],
                    each * cost[0] + (q + ceil_div(rest, light)) * cost[1]);
  };
  // all end together at about this q: light pairs make up for a tile of the first
  const long long most = ceil_div(tiles[1], pairs);
  const double at = cost[1] > 0 ? ((double)tiles[1] - light * cost[0] / cost[1]) / pairs : 0;
  const long long mid = at <= 0 ? 0 : std::min(most, (long long)at);
  for (long long q = std::max<long long>(0, mid - 2); q <= std::min(most, mid + 2); ++q) {
    const double end = end_of(q);
    if (best.end < 0 || end < best.end) best.end = end, best.rounds1 = (int)q;
  }
  return best;
}

// Pairs at work on two products' tiles: one for each tile of either, up to one
// per two SMs.
int pair_count(const long long* tiles) { return (int)std::min<long long>(kNumSMs / 2, tiles[0] + tiles[1]); }

// A tile of the pair kernel: its products (a step takes longer the more pairs
// are at work: L2 and power) and its epilogue, which run beside each other.
struct PairTileUs {
  double mma, all;
};
PairTileUs pair_tile_us(const Product& q, int bn, double busy) {
  const double step_us = bn == 256 ? 0.28 + 0.09 * busy : 0.215 + 0.05 * busy;
  const bool maps = q.ep.vec && q.b.rows % 8 == 0;           // stored by tensor maps
  const double mma = ceil_div(q.red, kStepK) * step_us + 0.5;
  return {mma, std::max(mma, bn == 256 ? (maps ? 2.5 : 4.5) : (maps ? 1.5 : 2.5))};
}
double pair_us(const Product* prod, int n, int bn) {
  long long tiles[2] = {0, 0}, steps = 0;
  for (int i = 0; i < n; ++i) {
    tiles[i] = ceil_div(prod[i].a.rows, kPairM) * ceil_div(prod[i].b.rows, bn);
    steps = std::max(steps, ceil_div(prod[i].red, kStepK));
  }
  const long long all = tiles[0] + tiles[1];
  const int pairs = pair_count(tiles);
  const double busy = (double)all / (ceil_div(all, kNumSMs / 2) * (kNumSMs / 2));
  double mma[2] = {0, 0}, cost[2] = {0, 0};
  for (int i = 0; i < n; ++i) {
    const PairTileUs t = pair_tile_us(prod[i], bn, busy);
    mma[i] = t.mma, cost[i] = t.all;
  }
  // filling and draining the pipeline costs less where a tile is a step or two
  const double ends = std::min(bn == 256 ? 7.6 : 6.0, 3.0 + 1.7 * steps);
  return std::max(ends + schedule_pairs(tiles, mma, pairs).end, 3.0 + schedule_pairs(tiles, cost, pairs).end);
}

struct Choice {
  double us;
  int width;           // of the pair kernel's tiles, 0 for the split kernel
  SplitPlan split;
};
Choice choose(const Product* prod, int n) {
  Choice c{0, 0, plan_split(prod, n)};
  c.us = c.split.us;
  for (int bn = 128; bn <= 256; bn *= 2) {
    const double us = pair_us(prod, n, bn);
    if (us < c.us) c.us = us, c.width = bn;
  }
  return c;
}

// A kernel's first CTA clears the status word beside the others' work, which is
// early enough for waits of seconds alone: under a test's limit it is cleared before.
cudaError_t clear_ahead(bool& clear, uint32_t* status, cudaStream_t st) {
  if (!clear || test_wait_limit_ns() == kWaitLimitNs) return cudaSuccess;
  clear = false;
  return cudaMemsetAsync(status, 0, 4, st);
}

// The products' columns are the split kernel's m side, their rows its j side.
cudaError_t launch_split(int act, const Product* prod, int n, const SplitPlan& plan, const DbJoin& db,
                         uint32_t* status, bool clear, cudaStream_t st) {
  const cudaError_t cleared = clear_ahead(clear, status, st);
  if (cleared != cudaSuccess) return cleared;
  SplitParams p;
  memset(&p, 0, sizeof p);
  const int S = plan.S;
  const bool two = std::max(plan.bn[0], plan.bn[1]) <= 64;
  const int budget = two ? 100 * 1024 : 200 * 1024;
  long long tiles = 0;
  int smem = 0;
  p.tmem_cols = 32;
  for (int i = 0; i < n; ++i) {
    SplitProblem& q = p.prob[i];
    const Operand &a = prod[i].b, &b = prod[i].a;
    q.M = a.rows;
    q.J = b.rows;
    q.bn = plan.bn[i];
    q.ksteps = (prod[i].red + kStepK - 1) / kStepK;
    q.mt = (q.M + kTileM - 1) / kTileM;
    const long long t = (long long)q.mt * ((q.J + q.bn - 1) / q.bn);
    tiles += t;
    if (tiles > 1 << 27) return cudaErrorInvalidValue;
    q.tiles = (int)t;
    q.a_mn = a.mn;
    q.b_mn = b.mn;
    q.ep = prod[i].ep;
    const int stage = kABytes + q.bn * 128, steps = (q.ksteps + S - 1) / S;
    const int hold = ((q.bn + S) * kTileM * 4 + stage - 1) / stage;    // stages that the parts take
    q.stages = std::max(hold, std::min({budget / stage, steps, kSplitMaxStages}));
    smem = std::max(smem, q.stages * stage + 1024);
    while (p.tmem_cols < q.bn) p.tmem_cols *= 2;
    if (!operand_map(&q.tma_a, a, prod[i].red, kTileM) || !operand_map(&q.tma_b, b, prod[i].red, q.bn))
      return cudaErrorInvalidValue;
  }
  p.S = S;
  p.wait_ns = test_wait_limit_ns();
  p.tiles = (int)tiles;
  p.db = db;
  p.status = status;
  p.clear = clear;
  switch (act) {
    case MOE_ACT_NONE: return launch_split_act<MOE_ACT_NONE>(p, smem, st);
    case MOE_ACT_RELU: return launch_split_act<MOE_ACT_RELU>(p, smem, st);
    case MOE_ACT_GELU: return launch_split_act<MOE_ACT_GELU>(p, smem, st);
    case MOE_ACT_GELU_TANH: return launch_split_act<MOE_ACT_GELU_TANH>(p, smem, st);
    case MOE_ACT_SILU: return launch_split_act<MOE_ACT_SILU>(p, smem, st);
  }
  return cudaErrorInvalidValue;
}

template <int ACT, bool LIMIT = false>
cudaError_t launch_pair_act(const PairParams& p, int pairs, cudaStream_t st) {
  if (!LIMIT && p.wait_ns != kWaitLimitNs) return launch_pair_act<ACT, true>(p, pairs, st);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_pair_kernel<ACT, LIMIT>, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(linear_pair_kernel<ACT, LIMIT>, dim3(2 * pairs), dim3(kPairThreads), kPairSmem, st, p);
}

cudaError_t launch_pair(int act, const Product* prod, int n, int bn, const DbJoin& db, uint32_t* status, bool clear,
                        cudaStream_t st) {
  const cudaError_t cleared = clear_ahead(clear, status, st);
  if (cleared != cudaSuccess) return cleared;
  PairParams p;
  memset(&p, 0, sizeof p);
  long long tiles[2] = {0, 0};
  for (int i = 0; i < n; ++i) {
    PairProblem& q = p.prob[i];
    q.M = prod[i].a.rows;
    q.N = prod[i].b.rows;
    q.ksteps = (prod[i].red + kStepK - 1) / kStepK;
    q.a_mn = prod[i].a.mn;
    q.b_mn = prod[i].b.mn;
    q.mt = (q.M + kPairM - 1) / kPairM;
    q.nt = (q.N + bn - 1) / bn;
    q.ep = prod[i].ep;
    // a tensor store writes whole 16-byte pieces: past the last column of an N
    // that is no multiple of 8 it left its box's values in the row's padding
    q.ep.vec = q.ep.vec && q.N % 8 == 0;
    tiles[i] = (long long)q.mt * q.nt;
    if (tiles[i] > 1 << 30) return cudaErrorInvalidValue;
    if (!operand_map(&q.tma_a, prod[i].a, prod[i].red, kTileM) || !operand_map(&q.tma_b, prod[i].b, prod[i].red, bn / 2))
      return cudaErrorInvalidValue;
    auto out_map = [&](CUtensorMap* m, const uint16_t* out, long long ld) {
      return make_tensor_map_2d(m, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)q.N, (uint64_t)q.M, 64, 32,
                                CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)ld);
    };
    if (q.ep.vec && (!out_map(&q.tma_out, q.ep.out, q.ep.ldo) || (q.ep.z && !out_map(&q.tma_z, q.ep.z, q.ep.ldz))))
      return cudaErrorInvalidValue;
  }
  p.tiles0 = (int)tiles[0];
  p.tiles1 = (int)tiles[1];
  p.wait_ns = test_wait_limit_ns();
  p.bn = bn;
  p.db = db;
  p.status = status;
  p.clear = clear;
  const int pairs = pair_count(tiles);
  double cost[2] = {0, 0};
  for (int i = 0; i < n; ++i) cost[i] = pair_tile_us(prod[i], bn, 1).all;
  const PairSchedule plan = schedule_pairs(tiles, cost, pairs);
  p.rounds1 = plan.rounds1;
  p.first_light = plan.first_light;
  switch (act) {
    case MOE_ACT_NONE: return launch_pair_act<MOE_ACT_NONE>(p, pairs, st);
    case MOE_ACT_RELU: return launch_pair_act<MOE_ACT_RELU>(p, pairs, st);
    case MOE_ACT_GELU: return launch_pair_act<MOE_ACT_GELU>(p, pairs, st);
    case MOE_ACT_GELU_TANH: return launch_pair_act<MOE_ACT_GELU_TANH>(p, pairs, st);
    case MOE_ACT_SILU: return launch_pair_act<MOE_ACT_SILU>(p, pairs, st);
  }
  return cudaErrorInvalidValue;
}

bool vec_ok(const Epilogue& e) {
  return e.ldo % 8 == 0 && (!e.residual || e.ldr % 8 == 0) && (!e.z || e.ldz % 8 == 0);
}

long long up8(long long v) { return (v + 7) / 8 * 8; }

// Row pitch of a copied operand and of dz: whole 128-byte lines.
long long copy_pitch(long long cols) { return (cols + 63) / 64 * 64; }

// A single row's pitch is of no account.
bool needs_copy(int rows, long long ld) { return rows > 1 && ld % 8; }
long long operand_pitch(int rows, long long ld) { return rows > 1 ? ld : up8(ld); }

// Counts the jobs' items; CTAs for them in `grid`.
bool plan_pack(PackParams& p, unsigned& grid) {
  long long items = 0;
  for (int i = 0; i < p.n; ++i) {
    const long long n = p.job[i].rows * ceil_div(p.job[i].cols, 256);
    p.job[i].items = (unsigned)n;
    items += n;
  }
  grid = (unsigned)std::min<long long>((items + 7) / 8, 16 * kNumSMs);
  return items <= 1ll << 31;
}

cudaError_t launch_pack(PackParams p, cudaStream_t st) {
  if (p.n == 0) return cudaSuccess;
  unsigned grid;
  if (!plan_pack(p, grid)) return cudaErrorInvalidValue;
  return launch_pdl(pack_rows_kernel, dim3(grid), dim3(256), 0, st, p);
}

template <int ACT>
cudaError_t launch_dz(bool any, cudaStream_t st, const uint16_t* dy, long long lddy, const uint16_t* z, long long ldz,
                      int T, int N, int rows, uint16_t* dz, long long lddz, float* part, uint32_t* clear, PackParams pk) {
  unsigned more;
  if (!plan_pack(pk, more)) return cudaErrorInvalidValue;
  const unsigned strips = (unsigned)ceil_div(N, 256), ctas = strips * (unsigned)ceil_div(T, rows);
  return launch_pdl(any ? linear_dz_kernel<ACT, true> : linear_dz_kernel<ACT, false>, dim3(ctas + more), dim3(256), 0, st,
                    dy, lddy, z, ldz, T, N, rows, dz, lddz, part, clear, strips, ctas, pk);
}

// Rows per CTA of the dz pass: one round of loads, more where that gives over
// eight CTAs per SM or more than 128 chunks for db's join.
int dz_rows(int T, int N) {
  const long long round = 8 * kDzRows, strips = (N + 255) / 256, all = (T + round - 1) / round;
  const long long rounds = std::max((all * strips + 8 * kNumSMs - 1) / (8 * kNumSMs), (all + 127) / 128);
  return (int)(round * rounds);
}

// The most chunks that dz_rows makes of any up to T rows: the chunks themselves
// get fewer where T passes a limit (128 at T 4096, 65 at 4097), and a workspace
// for T tokens has to do for fewer.
size_t most_dz_chunks(int T) { return std::min<size_t>(128, (T + 8 * kDzRows - 1) / (8 * kDzRows)); }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

LinearLayout linear_layout(int T, int K, int N, long long ldx, long long ldw) {
  LinearLayout L{};
  size_t o = 256;                                             // status word
  L.x = o;
  if (needs_copy(T, ldx)) o = up256(o + 2 * (size_t)T * copy_pitch(K));
  L.w = o;
  if (needs_copy(N, ldw)) o = up256(o + 2 * (size_t)N * copy_pitch(K));
  L.dz = L.part = L.bytes = o;
  return L;
}

LinearLayout linear_backward_layout(int T, int K, int N, long long ldx, long long ldw) {
  LinearLayout L = linear_layout(T, K, N, ldx, ldw);
  size_t o = L.bytes;
  L.dz = o;
  o = up256(o + 2 * (size_t)T * copy_pitch(N));
  L.part = o;
  o = up256(o + 4 * (size_t)N * most_dz_chunks(T));
  L.bytes = o;
  return L;
}

cudaError_t launch_linear(int act, const LinearArgs& a, void* ws, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  const LinearLayout L = linear_layout(a.T, a.K, a.N, a.ldx, a.ldw);
  Operand x{a.x, operand_pitch(a.T, a.ldx), a.T, false}, w{a.w, operand_pitch(a.N, a.ldw), a.N, false};
  PackParams pk{};
  if (needs_copy(a.T, a.ldx)) {
    x = Operand{reinterpret_cast<uint16_t*>(base + L.x), copy_pitch(a.K), a.T, false};
    pk.job[pk.n++] = PackJob{a.x, reinterpret_cast<uint16_t*>(base + L.x), a.ldx, x.ld, a.T, a.K};
  }
  if (needs_copy(a.N, a.ldw)) {
    w = Operand{reinterpret_cast<uint16_t*>(base + L.w), copy_pitch(a.K), a.N, false};
    pk.job[pk.n++] = PackJob{a.w, reinterpret_cast<uint16_t*>(base + L.w), a.ldw, w.ld, a.N, a.K};
  }
  Epilogue ep{a.bias, a.residual, a.z, a.y, a.ldr, a.ldz, a.ldy, 0};
  ep.vec = vec_ok(ep);
  const Product prod{x, w, a.K, ep};
  uint32_t* status = reinterpret_cast<uint32_t*>(base);
  const Choice c = choose(&prod, 1);
  if (pk.n) {
    pk.clear = status;
    const cudaError_t e = launch_pack(pk, st);
    if (e != cudaSuccess) return e;
  }
  if (c.width) return launch_pair(act, &prod, 1, c.width, DbJoin{}, status, pk.n == 0, st);
  return launch_split(act, &prod, 1, c.split, DbJoin{}, status, pk.n == 0, st);
}

cudaError_t launch_linear_backward(int act, const LinearBackwardArgs& a, void* ws, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(base);
  const LinearLayout L = linear_backward_layout(a.T, a.K, a.N, a.ldx, a.ldw);
  cudaError_t e;
  PackParams pk{};
  const uint16_t *x = a.x, *w = a.w;
  long long ldx = operand_pitch(a.T, a.ldx), ldw = operand_pitch(a.N, a.ldw);
  if (a.dw && needs_copy(a.T, a.ldx)) {
    x = reinterpret_cast<uint16_t*>(base + L.x);
    ldx = copy_pitch(a.K);
    pk.job[pk.n++] = PackJob{a.x, reinterpret_cast<uint16_t*>(base + L.x), a.ldx, ldx, a.T, a.K};
  }
  if (a.dx && needs_copy(a.N, a.ldw)) {
    w = reinterpret_cast<uint16_t*>(base + L.w);
    ldw = copy_pitch(a.K);
    pk.job[pk.n++] = PackJob{a.w, reinterpret_cast<uint16_t*>(base + L.w), a.ldw, ldw, a.N, a.K};
  }
  bool clear = true;                   // for the call's first launch

  // dz: dy itself where the layer has no activation and dy can be an operand
  const bool products = a.dx || a.dw, write_dz = products && (act != MOE_ACT_NONE || needs_copy(a.T, a.lddy));
  const uint16_t* dz = a.dy;
  long long lddz = operand_pitch(a.T, a.lddy);
  DbJoin db{};
  if (write_dz || a.db) {
    uint16_t* dst = write_dz ? reinterpret_cast<uint16_t*>(base + L.dz) : nullptr;
    const long long pitch = copy_pitch(a.N);
    const int rows = dz_rows(a.T, a.N), chunks = (a.T + rows - 1) / rows;
    float* part = a.db ? reinterpret_cast<float*>(base + L.part) : nullptr;
    const bool any = a.lddy % 8 || (act != MOE_ACT_NONE && a.ldz % 8);
    switch (act) {
#define RNX_DZ(A) case A: e = launch_dz<A>(any, st, a.dy, a.lddy, a.z, a.ldz, a.T, a.N, rows, dst, pitch, part, status, pk); break
      RNX_DZ(MOE_ACT_NONE);
      RNX_DZ(MOE_ACT_RELU);
      RNX_DZ(MOE_ACT_GELU);
      RNX_DZ(MOE_ACT_GELU_TANH);
      RNX_DZ(MOE_ACT_SILU);
#undef RNX_DZ
      default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    clear = false;
    if (write_dz) {
      dz = dst;
      lddz = pitch;
    }
    if (a.db) db = DbJoin{part, a.db, chunks, a.N};
  } else if (pk.n) {
    pk.clear = status;
    if ((e = launch_pack(pk, st)) != cudaSuccess) return e;
    clear = false;
  }
  Product prod[2];
  int n = 0;
  auto take = [&](uint16_t* out, long long ldo, const Operand& rows, const Operand& cols, int red) {
    Epilogue ep{nullptr, nullptr, nullptr, out, 0, 0, ldo, 0};
    ep.vec = vec_ok(ep);
    prod[n++] = Product{rows, cols, red, ep};
  };
  // dx[t, k] = sum_n dz[t, n] w[n, k];  dw[n, k] = sum_t dz[t, n] x[t, k]
  if (a.dx) take(a.dx, a.lddx, Operand{dz, lddz, a.T, false}, Operand{w, ldw, a.K, true}, a.N);
  if (a.dw) take(a.dw, a.lddw, Operand{dz, lddz, a.N, true}, Operand{x, ldx, a.K, true}, a.T);
  if (n == 2 && prod[0].red < prod[1].red) std::swap(prod[0], prod[1]);   // the longer tiles first
  auto launch = [&](const Product* q, int count, const Choice& c) {
    const cudaError_t err = c.width ? launch_pair(MOE_ACT_NONE, q, count, c.width, db, status, clear, st)
                                    : launch_split(MOE_ACT_NONE, q, count, c.split, db, status, clear, st);
    db = DbJoin{};
    clear = false;
    return err;
  };
  if (n) {
    // both in one launch, or one launch each where that is estimated a quarter
    // shorter (the second waits for the first's end): a single form of tiles and
    // splits does not fit every pair of reductions. T 1, 1472 -> 5760: 40 us in
    // one launch, 19 in two; T 64, 4096 -> 4096: 30 and 36.
    const Choice both = choose(prod, n);
    if (n == 2) {
      const Choice first = choose(prod, 1), second = choose(prod + 1, 1);
      if (1.25 * (first.us + second.us) < both.us) {
        if ((e = launch(prod, 1, first)) != cudaSuccess) return e;
        if ((e = launch(prod + 1, 1, second)) != cudaSuccess) return e;
        n = 0;
      }
    }
    if (n && (e = launch(prod, n, both)) != cudaSuccess) return e;
  }
  if (db.db) return launch_pdl(linear_db_kernel, dim3((a.N + 31) / 32), dim3(32), 0, st, db);
  return cudaSuccess;
}

}  // namespace rnx
