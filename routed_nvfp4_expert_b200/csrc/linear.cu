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
// dz is rounded to bf16, the tensor cores' operand type (half a step, 2^-9 of
// each element; y, z, dx and dW take the same one rounding); db is summed in
// fp32 from the unrounded dz.

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tensor_map.h"

namespace rnx {

namespace {

// ---------------------------------------------------------------- activations

template <int ACT>
RNX_DEVICE float act_of(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (ACT == MOE_ACT_GELU) return z * normcdff(z);
  if (ACT == MOE_ACT_GELU_TANH) {
    const float u = 0.7978845608028654f * fmaf(0.044715f * z * z, z, z);
    return 0.5f * z * (1.f + tanhf(u));
  }
  if (ACT == MOE_ACT_SILU) return z / (1.f + expf(-z));
  return z;
}

template <int ACT>
RNX_DEVICE float act_grad(float z) {
  if (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if (ACT == MOE_ACT_GELU) return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
  if (ACT == MOE_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float t = tanhf(0.7978845608028654f * fmaf(0.044715f * z2, z, z));
    return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * 0.7978845608028654f * fmaf(3.f * 0.044715f, z2, 1.f);
  }
  if (ACT == MOE_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

// ---------------------------------------------------------------- shared pieces

constexpr int kStepK = 64;                 // reduction elements per stage: 128 bytes per row (one swizzle span)
constexpr int kTileM = 128;
constexpr int kABytes = kTileM * 128;      // 16 KB; K-major: 128 rows; MN-major: two 64-wide blocks of 64 rows
constexpr int kMnBlock = 64 * 128;         // one MN-major block: 64 r rows of 128 bytes

struct Epilogue {
  const uint16_t* bias;       // per output feature, nullable
  const uint16_t* residual;   // nullable
  uint16_t* z;                // pre-activation, nullable
  uint16_t* out;
  long long ldr, ldz, ldo;
  int vec;                    // rows of residual, z and out all start on 16-byte boundaries
};

// db from the column sums of the row chunks, in chunk order, by one warp per CTA.
struct DbJoin {
  const float* part;          // [chunks, n]
  float* db;                  // nullable
  int chunks, n;
};
RNX_DEVICE void join_db(const DbJoin& d, int cta, int ctas, int lane) {
  if (!d.db) return;
  for (int c = cta * 32 + lane; c < d.n; c += ctas * 32) {
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < d.chunks; ++i) v += d.part[(size_t)i * d.n + c];
    d.db[c] = v;
  }
}

// ---------------------------------------------------------------- split kernel
// One 128 x bn tile of D by a cluster of S CTAs that divide the reduction
// between them: few rows leave few tiles, and the weights' bytes should come
// in through every SM. Each CTA accumulates its part in tensor memory and
// leaves it in its shared memory as fp32 [bn][128]; after a cluster barrier
// CTA s adds the S parts of its share of the j rows in rank order (so the
// result does not depend on timing), applies the epilogue and stores rows of
// out[j, m], 128 consecutive features per warp.
// Warps: 0 = TMA producer, 1 = MMA issuer, 2 = TMEM allocator, 3 = db join,
// 4-7 = TMEM readers; all eight reduce and store. Every wait is bounded; a
// timeout sets the status word, and the CTA still meets its cluster's barriers.

constexpr int kSplitThreads = 256;
constexpr int kSplitMaxStages = 10;

struct SplitParams {
  CUtensorMap tma_a, tma_b;
  Epilogue ep;
  DbJoin db;
  uint32_t* status;
  int M, J;                   // D's extents
  int ksteps;                 // 64-element steps of the whole reduction
  int bn, stages, tmem_cols;
  int a_mn, b_mn;
  int clear;
};

template <int ACT>
__global__ void __launch_bounds__(kSplitThreads, 2) linear_split_kernel(const __grid_constant__ SplitParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full_bar[kSplitMaxStages], empty_bar[kSplitMaxStages], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = gridDim.x, rank = blockIdx.x;
  const int m0 = blockIdx.y * kTileM, j0 = blockIdx.z * p.bn;
  const int k_lo = (int)((long long)p.ksteps * rank / S), k_hi = (int)((long long)p.ksteps * (rank + 1) / S);
  const int stage_bytes = kABytes + p.bn * 128;
  const int cta = (blockIdx.z * gridDim.y + blockIdx.y) * S + rank;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&mma_done, 1);
    abort_flag = 0;
    fence_barrier_init();
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
  if (p.clear && cta == 0 && threadIdx.x == 0) *p.status = 0u;

  if (warp == 0) {
    int it = 0;
    bool ok = true;
    for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
      const int s = it % p.stages;
      const uint32_t ph = (uint32_t)(it / p.stages) & 1u;
      if (__any_sync(0xffffffffu, !mbar_wait_poll(&empty_bar[s], ph ^ 1u) || abort_flag)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        uint8_t* sA = smem + (size_t)s * stage_bytes;
        uint8_t* sB = sA + kABytes;
        mbar_arrive_expect_tx(&full_bar[s], (uint32_t)stage_bytes);
        if (p.a_mn) {
          tma_load_2d(sA, &p.tma_a, m0, ks * kStepK, &full_bar[s]);
          tma_load_2d(sA + kMnBlock, &p.tma_a, m0 + 64, ks * kStepK, &full_bar[s]);
        } else {
          tma_load_2d(sA, &p.tma_a, ks * kStepK, m0, &full_bar[s]);
        }
        if (p.b_mn) {
          for (int c = 0; c < p.bn; c += 64)
            tma_load_2d(sB + c * 128, &p.tma_b, j0 + c, ks * kStepK, &full_bar[s]);
        } else {
          tma_load_2d(sB, &p.tma_b, ks * kStepK, j0, &full_bar[s]);
        }
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      set_status(p.status, kDevErrTimeout);
      abort_flag = 1;
    }
    for (int j = max(0, it - p.stages); j < it; ++j)      // every copy issued must have landed
      if (!mbar_wait(&full_bar[j % p.stages], (uint32_t)(j / p.stages) & 1u) && lane == 0)
        set_status(p.status, kDevErrTimeout);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_major(kTileM, p.bn, p.a_mn, p.b_mn);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t dA0 = p.a_mn ? sdesc_mn_sw128(s0, kMnBlock) : sdesc_k_sw128(s0);
    const uint64_t dB0 = p.b_mn ? sdesc_mn_sw128(s0 + kABytes, kMnBlock) : sdesc_k_sw128(s0 + kABytes);
    const uint64_t stepA = p.a_mn ? 2048 >> 4 : 32 >> 4, stepB = p.b_mn ? 2048 >> 4 : 32 >> 4;   // K = 16
    int it = 0;
    bool ok = true;
    for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
      const int s = it % p.stages;
      const uint32_t ph = (uint32_t)(it / p.stages) & 1u;
      if (__any_sync(0xffffffffu, !mbar_wait_poll(&full_bar[s], ph) || abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t so = (uint64_t)((uint32_t)(s * stage_bytes) >> 4);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          mma_bf16(tmem, dA0 + so + kb * stepA, dB0 + so + kb * stepB, idesc, (it > 0 || kb > 0) ? 1u : 0u);
        mma_commit(&empty_bar[s]);
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
  } else if (warp == 3) {
    join_db(p.db, cta, S * gridDim.y * gridDim.z, lane);
  }

  // the producer and the issuer are through: every copy has landed and every
  // MMA is done, so the stages may hold the accumulator's fp32 values
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);            // [bn][128]
  if (warp >= 4) {
    tc_fence_after();
    const int q = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    for (int c = 0; c < p.bn; c += 16) {
      uint32_t v[16];
      tmem_ld16(tq + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * kTileM + q * 32 + lane] = __uint_as_float(v[i]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (S > 1) cluster_sync_all();

  // ---------------------------------------------------------------- join and epilogue
  const int nj = min(p.bn, p.J - j0), per = (nj + S - 1) / S;
  const int j_lo = rank * per, j_hi = min(nj, j_lo + per);
  const int m = m0 + 4 * lane;
  const bool whole = p.ep.vec && m + 4 <= p.M;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.ep.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m + i < p.M) bias[i] = bf16_bits_to_f32(p.ep.bias[m + i]);
  const uint32_t part_addr = smem_u32(part) + 16 * lane;
  for (int j = j_lo + warp; j < j_hi; j += kSplitThreads / 32) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (S == 1) {
      const float4 f = *reinterpret_cast<const float4*>(part + (size_t)j * kTileM + 4 * lane);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll 8
      for (int s = 0; s < S; ++s) {
        const float4 f = ld_cluster_f4(mapa_shared(part_addr + j * kTileM * 4, (uint32_t)s));
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
    }
    const long long row = j0 + j;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bias[i];
    if (whole) {
      if (p.ep.z)
        *reinterpret_cast<uint2*>(p.ep.z + row * p.ep.ldz + m) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = act_of<ACT>(v[i]);
      if (p.ep.residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(p.ep.residual + row * p.ep.ldr + m);
        const float2 a = bf16x2_to_f32x2(r.x), b = bf16x2_to_f32x2(r.y);
        v[0] += a.x, v[1] += a.y, v[2] += b.x, v[3] += b.y;
      }
      *reinterpret_cast<uint2*>(p.ep.out + row * p.ep.ldo + m) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m + i >= p.M) break;
        if (p.ep.z) p.ep.z[row * p.ep.ldz + m + i] = f32_to_bf16_bits(v[i]);
        float y = act_of<ACT>(v[i]);
        if (p.ep.residual) y += bf16_bits_to_f32(p.ep.residual[row * p.ep.ldr + m + i]);
        p.ep.out[row * p.ep.ldo + m + i] = f32_to_bf16_bits(y);
      }
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync_all();      // no CTA leaves while a peer may still read its part
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
  }
}

// ---------------------------------------------------------------- dz and db
// dz = dy act'(z) in bf16 and the column sums of each chunk of rows in fp32
// (rows of a warp in order, then the warps). A CTA owns 256 columns of one
// chunk. VEC: 16-byte loads, eight consecutive columns per lane; otherwise
// columns lane + 32 i. HBM-bound: 6 T N bytes (dy, z, dz).
template <int ACT, bool VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(const uint16_t* dy, long long lddy, const uint16_t* z,
                                                        long long ldz, int T, int N, int rows_per_cta, uint16_t* dz,
                                                        long long lddz, float* db_part, uint32_t* clear) {
  __shared__ float red[8][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * 256 + (VEC ? 8 * lane : lane);
  constexpr int kStep = VEC ? 1 : 32;
  const int r0 = blockIdx.y * rows_per_cta, r1 = min(T, r0 + rows_per_cta);
  const bool whole = VEC && c0 + 8 <= N;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  pdl_wait();
  pdl_trigger();
  if (clear && blockIdx.x + blockIdx.y == 0 && threadIdx.x == 0) *clear = 0u;
#pragma unroll 2
  for (int r = r0 + warp; r < r1; r += 8) {
    float g[8], a[8];
    const uint16_t* py = dy + r * lddy;
    const uint16_t* pz = z + r * ldz;
    if (whole) {
      const uint4 u = *reinterpret_cast<const uint4*>(py + c0);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_f32x2(w[i]);
        g[2 * i] = f.x, g[2 * i + 1] = f.y;
      }
      if (ACT != MOE_ACT_NONE) {
        const uint4 uz = *reinterpret_cast<const uint4*>(pz + c0);
        const uint32_t wz[4] = {uz.x, uz.y, uz.z, uz.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_f32x2(wz[i]);
          a[2 * i] = f.x, a[2 * i + 1] = f.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + kStep * i;
        g[i] = c < N ? bf16_bits_to_f32(py[c]) : 0.f;
        a[i] = ACT != MOE_ACT_NONE && c < N ? bf16_bits_to_f32(pz[c]) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ACT != MOE_ACT_NONE) g[i] *= act_grad<ACT>(a[i]);
      acc[i] += g[i];
    }
    if (dz) {
      uint16_t* pd = dz + r * lddz;
      if (whole) {
        *reinterpret_cast<uint4*>(pd + c0) = make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                                                        pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + kStep * i < N) pd[c0 + kStep * i] = f32_to_bf16_bits(g[i]);
      }
    }
  }
  if (!db_part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[warp][(VEC ? 8 * lane : lane) + kStep * i] = acc[i];
  __syncthreads();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < N) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][threadIdx.x];
    db_part[(size_t)blockIdx.y * N + c] = v;
  }
}

// db of a call that wants nothing else.
__global__ void __launch_bounds__(32) linear_db_kernel(const DbJoin d) {
  pdl_wait();
  pdl_trigger();
  join_db(d, blockIdx.x, gridDim.x, threadIdx.x);
}

// ---------------------------------------------------------------- row pitch
// Rows whose pitch is not a multiple of 16 bytes cannot be a TMA operand; they
// are copied to a pitch that is (columns behind the last are never read: the
// tensor map ends at `cols`). Up to two operands in one launch.
struct PackJob {
  const uint16_t* src;
  uint16_t* dst;
  long long ld_src, ld_dst;
  int rows, cols;
};
struct PackParams {
  PackJob job[2];
  int n;
  uint32_t* clear;     // status word (the pack is the call's first launch)
};
__global__ void __launch_bounds__(256) pack_rows_kernel(const PackParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.clear = 0u;
  for (int q = 0; q < p.n; ++q) {
    const PackJob& d = p.job[q];
    const int groups = (d.cols + 7) / 8;
    const long long items = (long long)d.rows * groups;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
      const long long r = i / groups;
      const int c = 8 * (int)(i - r * groups);
      const uint16_t* s = d.src + r * d.ld_src + c;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = c + 2 * k < d.cols ? s[2 * k] : 0u, hi = c + 2 * k + 1 < d.cols ? s[2 * k + 1] : 0u;
        w[k] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(d.dst + r * d.ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------- host side

// Opt-in shared memory of a kernel, once per device.
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinearMaxSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

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

template <int ACT>
cudaError_t launch_split_act(const SplitParams& p, int S, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_split_kernel<ACT>, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, (p.M + kTileM - 1) / kTileM, (p.J + p.bn - 1) / p.bn);
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePriority;
  attr[1].val.priority = launch_priority_high();
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = S;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<ACT>, p);
}

// out[j, m] = epilogue(sum_r A[m, r] B[j, r])
cudaError_t launch_split(int act, const Operand& a, const Operand& b, int red, const Epilogue& ep, const DbJoin& db,
                         uint32_t* status, bool clear, cudaStream_t st) {
  SplitParams p;
  memset(&p, 0, sizeof p);
  const int J = b.rows, unit = b.mn ? 64 : 16;            // MN-major blocks are 64 wide
  const int jt = (J + 255) / 256;
  p.bn = ((J + jt - 1) / jt + unit - 1) / unit * unit;
  p.M = a.rows;
  p.J = J;
  p.ksteps = (red + kStepK - 1) / kStepK;
  const int mt = (p.M + kTileM - 1) / kTileM, tiles = mt * ((J + p.bn - 1) / p.bn);
  const int stage = kABytes + p.bn * 128;
  // narrow tiles keep two CTAs per SM (one's epilogue beside the other's
  // stream), wide ones need the shared memory for their stages
  const bool two = p.bn <= 64;
  const int budget = two ? 100 * 1024 : 200 * 1024;
  int S = 1;
  while (S < 8 && tiles * S * 2 <= (two ? 2 : 1) * kNumSMs && S * 2 <= p.ksteps) S *= 2;
  const int steps = (p.ksteps + S - 1) / S;
  const int hold = (p.bn * kTileM * 4 + stage - 1) / stage;          // stages that the fp32 tile takes
  p.stages = std::max(hold, std::min({budget / stage, steps, kSplitMaxStages}));
  p.tmem_cols = 32;
  while (p.tmem_cols < p.bn) p.tmem_cols *= 2;
  p.a_mn = a.mn;
  p.b_mn = b.mn;
  p.ep = ep;
  p.db = db;
  p.status = status;
  p.clear = clear;
  if (mt > 65535 || (J + p.bn - 1) / p.bn > 65535) return cudaErrorInvalidValue;
  if (!operand_map(&p.tma_a, a, red, kTileM) || !operand_map(&p.tma_b, b, red, p.bn)) return cudaErrorInvalidValue;
  const int smem = p.stages * stage + 1024;
  switch (act) {
    case MOE_ACT_NONE: return launch_split_act<MOE_ACT_NONE>(p, S, smem, st);
    case MOE_ACT_RELU: return launch_split_act<MOE_ACT_RELU>(p, S, smem, st);
    case MOE_ACT_GELU: return launch_split_act<MOE_ACT_GELU>(p, S, smem, st);
    case MOE_ACT_GELU_TANH: return launch_split_act<MOE_ACT_GELU_TANH>(p, S, smem, st);
    case MOE_ACT_SILU: return launch_split_act<MOE_ACT_SILU>(p, S, smem, st);
  }
  return cudaErrorInvalidValue;
}

bool vec_ok(const Epilogue& e) {
  return e.ldo % 8 == 0 && (!e.residual || e.ldr % 8 == 0) && (!e.z || e.ldz % 8 == 0);
}

long long up8(long long v) { return (v + 7) / 8 * 8; }

// A single row's pitch is of no account.
bool needs_copy(int rows, long long ld) { return rows > 1 && ld % 8; }
long long operand_pitch(int rows, long long ld) { return rows > 1 ? ld : up8(ld); }

cudaError_t launch_pack(const PackParams& p, cudaStream_t st) {
  if (p.n == 0) return cudaSuccess;
  long long items = 0;
  for (int i = 0; i < p.n; ++i) items = std::max(items, (long long)p.job[i].rows * ((p.job[i].cols + 7) / 8));
  const int grid = (int)std::min<long long>((items + 255) / 256, 8 * kNumSMs);
  return launch_pdl(pack_rows_kernel, dim3(grid), dim3(256), 0, st, p);
}

template <int ACT>
cudaError_t launch_dz(bool vec, dim3 grid, cudaStream_t st, const uint16_t* dy, long long lddy, const uint16_t* z,
                      long long ldz, int T, int N, int rows, uint16_t* dz, long long lddz, float* part, uint32_t* clear) {
  if (vec) return launch_pdl(linear_dz_kernel<ACT, true>, grid, dim3(256), 0, st, dy, lddy, z, ldz, T, N, rows, dz, lddz, part,
                             clear);
  return launch_pdl(linear_dz_kernel<ACT, false>, grid, dim3(256), 0, st, dy, lddy, z, ldz, T, N, rows, dz, lddz, part,
                    clear);
}

// Row chunks of the dz pass: enough CTAs to fill the GPU a few times over.
int dz_rows(int T, int N) {
  const long long strips = (N + 255) / 256;
  const long long chunks = std::max<long long>(1, std::min<long long>((T + 31) / 32, (8 * kNumSMs + strips - 1) / strips));
  return (int)((T + chunks - 1) / chunks);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

LinearLayout linear_layout(int T, int K, int N, long long ldx, long long ldw) {
  LinearLayout L{};
  size_t o = 256;                                             // status word
  L.x = o;
  if (needs_copy(T, ldx)) o = up256(o + 2 * (size_t)T * up8(K));
  L.w = o;
  if (needs_copy(N, ldw)) o = up256(o + 2 * (size_t)N * up8(K));
  L.dz = L.part = L.bytes = o;
  return L;
}

LinearLayout linear_backward_layout(int T, int K, int N, long long ldx, long long ldw) {
  LinearLayout L = linear_layout(T, K, N, ldx, ldw);
  size_t o = L.bytes;
  L.dz = o;
  o = up256(o + 2 * (size_t)T * up8(N));
  L.part = o;
  if (T > 0) o = up256(o + 4 * (size_t)N * ((T + dz_rows(T, N) - 1) / dz_rows(T, N)));
  L.bytes = o;
  return L;
}

cudaError_t launch_linear(int act, const LinearArgs& a, void* ws, cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  const LinearLayout L = linear_layout(a.T, a.K, a.N, a.ldx, a.ldw);
  Operand x{a.x, operand_pitch(a.T, a.ldx), a.T, false}, w{a.w, operand_pitch(a.N, a.ldw), a.N, false};
  PackParams pk{};
  if (needs_copy(a.T, a.ldx)) {
    x = Operand{reinterpret_cast<uint16_t*>(base + L.x), up8(a.K), a.T, false};
    pk.job[pk.n++] = PackJob{a.x, reinterpret_cast<uint16_t*>(base + L.x), a.ldx, x.ld, a.T, a.K};
  }
  if (needs_copy(a.N, a.ldw)) {
    w = Operand{reinterpret_cast<uint16_t*>(base + L.w), up8(a.K), a.N, false};
    pk.job[pk.n++] = PackJob{a.w, reinterpret_cast<uint16_t*>(base + L.w), a.ldw, w.ld, a.N, a.K};
  }
  pk.clear = reinterpret_cast<uint32_t*>(base);
  cudaError_t e = launch_pack(pk, st);
  if (e != cudaSuccess) return e;
  Epilogue ep{a.bias, a.residual, a.z, a.y, a.ldr, a.ldz, a.ldy, 0};
  ep.vec = vec_ok(ep);
  return launch_split(act, w, x, a.K, ep, DbJoin{}, reinterpret_cast<uint32_t*>(base), pk.n == 0, st);
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
    ldx = up8(a.K);
    pk.job[pk.n++] = PackJob{a.x, reinterpret_cast<uint16_t*>(base + L.x), a.ldx, ldx, a.T, a.K};
  }
  if (a.dx && needs_copy(a.N, a.ldw)) {
    w = reinterpret_cast<uint16_t*>(base + L.w);
    ldw = up8(a.K);
    pk.job[pk.n++] = PackJob{a.w, reinterpret_cast<uint16_t*>(base + L.w), a.ldw, ldw, a.N, a.K};
  }
  pk.clear = status;
  if ((e = launch_pack(pk, st)) != cudaSuccess) return e;
  bool clear = pk.n == 0;              // for the call's first launch

  // dz: dy itself where the layer has no activation and dy can be an operand
  const bool products = a.dx || a.dw, write_dz = products && (act != MOE_ACT_NONE || needs_copy(a.T, a.lddy));
  const uint16_t* dz = a.dy;
  long long lddz = operand_pitch(a.T, a.lddy);
  DbJoin db{};
  if (write_dz || a.db) {
    uint16_t* dst = write_dz ? reinterpret_cast<uint16_t*>(base + L.dz) : nullptr;
    const long long pitch = up8(a.N);
    const int rows = dz_rows(a.T, a.N), chunks = (a.T + rows - 1) / rows;
    float* part = a.db ? reinterpret_cast<float*>(base + L.part) : nullptr;
    const dim3 grid((a.N + 255) / 256, chunks);
    const bool vec = a.lddy % 8 == 0 && (act == MOE_ACT_NONE || a.ldz % 8 == 0);
    switch (act) {
#define RNX_DZ(A) case A: e = launch_dz<A>(vec, grid, st, a.dy, a.lddy, a.z, a.ldz, a.T, a.N, rows, dst, pitch, part, clear ? status : nullptr); break
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
  }
  if (a.dx) {
    Epilogue ep{nullptr, nullptr, nullptr, a.dx, 0, 0, a.lddx, 0};
    ep.vec = vec_ok(ep);
    e = launch_split(MOE_ACT_NONE, Operand{w, ldw, a.K, true}, Operand{dz, lddz, a.T, false}, a.N, ep, db, status,
                     clear, st);
    if (e != cudaSuccess) return e;
    db = DbJoin{};
    clear = false;
  }
  if (a.dw) {
    Epilogue ep{nullptr, nullptr, nullptr, a.dw, 0, 0, a.lddw, 0};
    ep.vec = vec_ok(ep);
    e = launch_split(MOE_ACT_NONE, Operand{x, ldx, a.K, true}, Operand{dz, lddz, a.N, true}, a.T, ep, db, status,
                     clear, st);
    if (e != cudaSuccess) return e;
    db = DbJoin{};
  }
  if (db.db) return launch_pdl(linear_db_kernel, dim3((a.N + 31) / 32), dim3(32), 0, st, db);
  return cudaSuccess;
}

}  // namespace rnx
