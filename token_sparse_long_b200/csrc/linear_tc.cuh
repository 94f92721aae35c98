// tcgen05 matrix products of the linear layer (sm_100a), on CTA pairs.
//
//   D[R, C] = sum_k A[R, k] B[C, k]        bf16 in, fp32 accumulate
//
// Three products share the kernel; an operand whose reduction index is its slow (row) index in
// memory is taken MN-major, straight from the row-major matrix (no transposed copy):
//   forward   y  = x w^T    A = x  [M, K]  K-major,   B = w [N, K]  K-major
//   dx        dx = dz w     A = dz [M, N]  K-major,   B = w [N, K]  MN-major (reduction N)
//   dw        dw = dz^T x   A = dz [M, N]  MN-major,  B = x [M, K]  MN-major (reduction M)
//
// A cluster of two CTAs owns a 256 x BN tile: each CTA stages its 128 rows of A and half of
// B's rows per 64-deep k-block, and one tcgen05.mma (cta_group::2, M 256) issued by the
// leader reads both CTAs' shared memory, so each SM moves half of the B tile it would alone.
// Accumulators (128 lanes x BN columns per CTA) are double buffered in tensor memory.
// With few rows of x (SWAP) the operands change places -- the weights are the 256-row side,
// A = w or w^T, and x or dz the narrow one -- so that the weights, which are all the traffic,
// spread over every SM; and a product with few tiles splits its reduction (ksplit) into fp32
// partial products that linear_finish adds in order.
// 320 threads per CTA (352 for tiles up to 128 wide):
//   warp 0      TMA producer (both CTAs; completion counted on the leader's full barrier)
//   warp 1      allocates tensor memory; in the leader one lane issues the MMAs and commits
//               (multicast to both CTAs' barriers)
//   warps 2..9  epilogue: two warps per TMEM lane quarter, half of the columns each
//   warp 10     in the leader, the MMAs of every other k-block of a narrow tile, into an
//               accumulator of its own that the epilogue adds: a warp issues an MMA only
//               every 116 clocks or so, which is more than a tile of 128 columns needs.  The
//               k-blocks alternate over the whole launch, not within a tile: a ring of an even
//               number of stages then keeps each stage with one of the two warps.  (Taken by a
//               warp that had not seen the stage's last phase, a wait by parity passes while that
//               phase is still open.)
// Persistent: one cluster per SM pair walks the tiles in bands of 8 row tiles (row tile
// fastest), so that a wave's operands stay within L2.
#pragma once

#include "gemm_tc.cuh"
#include "rows.cuh"

namespace jenga {

constexpr int LT_BAND = 8;

enum LinMode : int {
  LIN_OUT = 0,   // out bf16 = act(acc + bias) (+ residual); pre bf16 = acc + bias
  LIN_GRAD = 1,  // out fp32 (+)= acc, the accumulator promoted every LT_CHUNK k-blocks
};

// k-blocks (of 64) that a tensor-memory accumulator sums before it is added into fp32
// registers.  The tensor core truncates when it adds into the accumulator: measured relative
// loss 5e-7 over 512 products, 4e-6 over 4096 and 3e-5 over 26240 (1e-4 for all-positive
// operands), growing with the length.  512 products at a time keep it at what fp32 sums lose
// anyway, whatever the number of rows, and the reads hide behind the next products.
constexpr int LT_CHUNK = 8;

struct LinArgs {
  int R, C, nkb;                  // rows, columns, k-blocks of one pass over the reduction
  int m;                          // host bound on the rows of x (R, or the reduction of LIN_GRAD)
  int ksplit;                     // ranges of k-blocks; above 1 the tiles go to `part`
  float* part;                    // [ksplit][rows of the result][columns] fp32
  int passes;                     // LIN_GRAD: 3 = A is held in three parts, one pass over the rows each
  const int32_t* n_kept;          // device count of valid blocks of x's rows (nullable)
  int blk;
  const void* bias;
  int bias_bf16, act;
  const bf16* residual;
  int64_t ldr;
  void* out;
  int64_t ldo;
  bf16* pre;
  int64_t ldp;
  int out_tma, pre_tma;           // the tensor maps of out / pre are valid
  int accumulate;                 // LIN_GRAD
  const float* db_part;           // LIN_GRAD: partial column sums of dz [db_chunks][R] (nullable), added
  int db_chunks;                  //   into db by the first column's tiles while their products run
  float* db;
  int tail;                       // LIN_GRAD: the last partial k-block comes from the tail copy of x
};

template <int BN>
constexpr int lin_mma_warps = BN <= 128 ? 2 : 1;
template <int BN>
constexpr int lin_threads = BN <= 128 ? 352 : 320;

template <int BN, bool SWAP>
struct LinSmem {
  // narrow tiles move little per k-block: more of them in flight (about 180 KB an SM)
  static constexpr int STAGES = SWAP ? (BN >= 128 ? 8 : 10) : (BN >= 256 ? 5 : 6);
  static constexpr int A_BYTES = 128 * 64 * 2;
  static constexpr int B_BYTES = BN / 2 * 64 * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STG_OFF = STAGES * STAGE_BYTES;
  static constexpr int STG_BYTES = SWAP ? 0 : 8 * 2 * 4096;  // two 32-row x 128-byte tiles per epilogue warp
  static constexpr int BIAS_OFF = STG_OFF + STG_BYTES;
  static constexpr int BIAS_BYTES = SWAP ? 0 : BN * 4;  // the tile's bias, fp32
  static constexpr int BAR_OFF = BIAS_OFF + BIAS_BYTES;
  static constexpr int TOTAL = BAR_OFF + 256 + 1024;
  static_assert(TOTAL <= 232448, "shared memory per CTA");
};

// ---- CTA-pair PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// shared::cluster address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// TMA tile load into this CTA's shared memory, completion counted on a barrier of the pair
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar_cluster, int x,
                                                 int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs once the MMAs issued so far are complete
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_holder, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_holder)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t phase) { return poll_wait(bar, phase, SITE_LINEAR); }

// ---- activations (fp32).  GELU takes the normal distribution's tail by itself: 1 + erf(z / sqrt 2) cancels
// for negative z (nothing of it is left below -5.5).  __expf is within 2 + 1.17 |x| ulp, at most
// 2^-16 relative: below a bf16 result's half step; the fp32 gradients dw and db carry it.
//
// P(Z > t) of a standard normal Z, t >= 0, and e = e^(-t^2/2): e times a polynomial of degree 9 in r =
// 1 / (1 + 0.34 t) without a constant term (the ratio falls like 1 / t), a Lawson IRLS minimax fit of
// its relative error on [0, 14], 3.2e-8; evaluated in fp32 with e within 0.7 (1.3 (1 + t^2) + 12)
// half steps.  (4096 x 4096 -> 11008 with GELU, pre-activation saved: 307 us, with erfcf 338.)
__device__ __forceinline__ float normal_tail(float t, float& e) {
  const float r = __fdividef(1.f, fmaf(0.34f, t, 1.f));
  float a = -0x1.abf520p-6f;
  a = fmaf(a, r, 0x1.1db1dcp-3f);
  a = fmaf(a, r, -0x1.17b00ep-2f);
  a = fmaf(a, r, 0x1.9e11d4p-3f);
  a = fmaf(a, r, -0x1.6e5512p-5f);
  a = fmaf(a, r, 0x1.d882c8p-4f);
  a = fmaf(a, r, 0x1.d7d984p-4f);
  a = fmaf(a, r, 0x1.16c1fep-3f);
  a = fmaf(a, r, 0x1.15c034p-3f);
  e = fast_exp2(t * t * -0.72134752044448170f);
  return a * r * e;
}
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == JENGA_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (act == JENGA_ACT_GELU) {
    float e;
    const float q = normal_tail(fabsf(z), e);
    return z * (z < 0.f ? q : 1.f - q);
  }
  if (act == JENGA_ACT_SILU) return z / (1.f + __expf(-z));
  return z;
}
template <int N>
__device__ __forceinline__ void act_values(float* v, int act) {
  if (act == JENGA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], JENGA_ACT_RELU);
  } else if (act == JENGA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], JENGA_ACT_GELU);
  } else if (act == JENGA_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], JENGA_ACT_SILU);
  }
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == JENGA_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  // a pre-activation beyond bf16's range is saved as an infinity: the slopes' limits
  if (act != JENGA_ACT_NONE && fabsf(z) == INFINITY) return z > 0.f ? 1.f : 0.f;
  if (act == JENGA_ACT_GELU) {
    float e;
    const float q = normal_tail(fabsf(z), e);
    return fmaf(z * 0.39894228040143268f, e, z < 0.f ? q : 1.f - q);
  }
  if (act == JENGA_ACT_SILU) {
    const float s = 1.f / (1.f + __expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// One output element from z = product + bias: pre, activation, residual, rounding.
__device__ __forceinline__ void lin_finish(const LinArgs& p, int m, int n, float z) {
  if (p.pre) p.pre[(int64_t)m * p.ldp + n] = __float2bfloat16_rn(z);
  z = act_value(z, p.act);
  if (p.residual) z += __bfloat162float(p.residual[(int64_t)m * p.ldr + n]);
  reinterpret_cast<bf16*>(p.out)[(int64_t)m * p.ldo + n] = __float2bfloat16_rn(z);
}

// out = the epilogue of the partial products added in order: V columns per thread (four when the
// partial rows are 16-byte aligned), row y of the grid.
template <int V>
__global__ void __launch_bounds__(128) linear_finish_kernel(LinArgs p, int N) {
  const int m = blockIdx.y, n = (blockIdx.x * 128 + threadIdx.x) * V;
  if (n >= N || m >= valid_rows(RowMap{nullptr, p.n_kept, p.blk, 0, p.m})) return;
  const float* q = p.part + (int64_t)m * N + n;
  float z[V];
#pragma unroll
  for (int e = 0; e < V; ++e) z[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.ksplit; ++s) {
    if constexpr (V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(q + (int64_t)s * p.m * N);
      z[0] += f.x;
      z[1] += f.y;
      z[2] += f.z;
      z[3] += f.w;
    } else {
      z[0] += q[(int64_t)s * p.m * N];
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (p.bias) {
      float b;
      load_params<1>(p.bias, p.bias_bf16, n + e, 0.f, &b);
      z[e] += b;
    }
    lin_finish(p, m, n + e, z[e]);
  }
}

template <int BN, bool AMN, bool BMN, int MODE, bool SWAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lin_threads<BN>, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                     const __grid_constant__ CUtensorMap tmA3, const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmTail, const __grid_constant__ CUtensorMap tmOut,
                     const __grid_constant__ CUtensorMap tmPre, LinArgs p) {
  using L = LinSmem<BN, SWAP>;
  static_assert(!(BMN && BN < 128), "an MN-major B half is at least one 64-wide box");
  constexpr int ST = L::STAGES, MW = lin_mma_warps<BN>, ACC = MW * BN;  // columns of an accumulator set
  static_assert(ST % MW == 0 && LT_CHUNK % MW == 0, "a ring stage belongs to one MMA warp");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* empty = full + ST;
  uint64_t* acc_full = empty + ST;     // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2], used in the leader
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  // LIN_OUT: the valid rows of x bound the row tiles (the column tiles with SWAP); LIN_GRAD: they
  // are the reduction
  const int valid = valid_rows(RowMap{nullptr, p.n_kept, p.blk, 0, p.m});
  const int rows = MODE == LIN_OUT && !SWAP ? valid : p.R;
  const int cols = SWAP ? valid : p.C;
  const int nkb1 = MODE == LIN_OUT ? p.nkb : (valid + 63) / 64;
  const int nkb_all = nkb1 * (MODE == LIN_GRAD ? p.passes : 1);
  const int ntr = (rows + 255) / 256, ntc = (cols + BN - 1) / BN;
  const int ksplit = p.ksplit;
  const int ntiles = ntr * ntc * ksplit;
  if (cluster >= ntiles) return;  // uniform over the cluster
  // work tile t: output tile t / ksplit, k-blocks [lo, hi) of range t % ksplit
  auto tile_at = [&](int t, int& r0, int& c0, int& lo, int& hi) {
    const int ks = t % ksplit;
    t /= ksplit;
    lo = (int)((int64_t)nkb_all * ks / ksplit);
    hi = (int)((int64_t)nkb_all * (ks + 1) / ksplit);
    const int band = t / (LT_BAND * ntc), rem = t - band * LT_BAND * ntc;
    const int gm = min(LT_BAND, ntr - band * LT_BAND);
    r0 = (band * LT_BAND + rem % gm) * 256;
    c0 = rem / gm * BN;
  };

  if (threadIdx.x == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], MW);
      mbar_init(&acc_empty[b], 16);
    }
    fence_barrier_init();
  }
  // The pair's barriers are ready after this cluster barrier.  Tensor memory is allocated
  // meanwhile: the warps that read it wait for that here, and the leader's MMAs for the first
  // arrivals on acc_empty, which come from both CTAs; the loads start 700 clocks sooner.
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  if (warp == 1) tmem_alloc_pair(tmem_holder, 2 * ACC);
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  uint32_t tmem = 0;
  if (warp != 0) {
    tc_fence_before();
    asm volatile("bar.sync 2, %0;" ::"n"(lin_threads<BN> - 32) : "memory");
    tc_fence_after();
    tmem = *tmem_holder;
  }

  if (warp == 0) {
    // ---------------- TMA producer (the warp stays converged and elects a lane to issue: from a
    // divergent lane each copy or MMA took about 100 clocks to issue, 700 per k-block for 530)
    int g = 0;
    bool ok = true;
    for (int t = cluster; ok && t < ntiles; t += nclusters) {
      int r0, c0, lo, hi;
      tile_at(t, r0, c0, lo, hi);
      r0 += rank * 128;
      c0 += rank * (BN / 2);
      for (int kb = lo; kb < hi; ++kb, ++g) {
        const int s = g % ST;
        if (g >= ST && !__all_sync(0xffffffffu, pair_wait(&empty[s], ((g / ST) - 1) & 1))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* sa = smem + s * L::STAGE_BYTES;
          uint8_t* sb = sa + L::A_BYTES;
          const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::STAGE_BYTES);
          const int pass = MODE == LIN_GRAD ? (kb >= 2 * nkb1 ? 2 : (kb >= nkb1 ? 1 : 0)) : 0;
          const int kk = kb - pass * nkb1;
          const CUtensorMap* ma = pass == 2 ? &tmA3 : (pass == 1 ? &tmA2 : &tmA);
          if (AMN) {
            tma_load_2d_pair(sa, ma, bar, r0, kk * 64);
            tma_load_2d_pair(sa + 8192, ma, bar, r0 + 64, kk * 64);
          } else {
            tma_load_2d_pair(sa, ma, bar, kk * 64, r0);
          }
          if (BMN) {
            const bool tl = MODE == LIN_GRAD && p.tail && (kk + 1) * 64 > valid;
            const CUtensorMap* mb = tl ? &tmTail : &tmB;
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_2d_pair(sb + j * 8192, mb, bar, c0 + j * 64, tl ? 0 : kk * 64);
          } else {
            tma_load_2d_pair(sb, &tmB, bar, kk * 64, c0);
          }
        }
        __syncwarp();
      }
    }
    // the pair's copies are complete before either CTA leaves (at once after a normal run: the
    // MMAs waited for the same phases)
    if (rank == 0)
      for (int i = g > ST ? g - ST : 0; i < g; ++i)
        if (!pair_wait(&full[i % ST], (i / ST) & 1)) break;
  } else if ((warp == 1 || warp == 10) && rank == 0) {
    // ---------------- MMA issuers (leader): warp mw takes every MW-th k-block of the launch, those
    // of a unit (a tile, or a chunk of LIN_GRAD) into the unit's accumulator mw
    const int mw = warp == 1 ? 0 : 1;
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
                           ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
    bool ok = true;
    int g = 0, it = 0;  // k-blocks before the tile; units so far
    for (int t = cluster; ok && t < ntiles; t += nclusters) {
      int r0, c0, lo, hi;
      tile_at(t, r0, c0, lo, hi);
      for (int u0 = lo; ok && u0 < hi; u0 += LT_CHUNK) {
        const int u1 = MODE == LIN_GRAD ? min(u0 + LT_CHUNK, hi) : hi;
        const int buf = it & 1;
        if (!__all_sync(0xffffffffu, pair_wait(&acc_empty[buf], (it >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + buf * ACC + mw * BN;
        const int kb0 = u0 + ((g + u0 - lo + mw) & (MW - 1));  // the warp's first of the unit
        for (int kb = kb0; kb < u1; kb += MW) {
          const int gk = g + kb - lo, s = gk % ST;
          if (!__all_sync(0xffffffffu, pair_wait(&full[s], (gk / ST) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * L::STAGE_BYTES);
          const uint32_t sb = sa + L::A_BYTES;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t da = AMN ? umma_desc_mn_sw128(sa + k * 2048, 8192) : umma_desc_k_sw128(sa + k * 32);
              const uint64_t db = BMN ? umma_desc_mn_sw128(sb + k * 2048, 8192) : umma_desc_k_sw128(sb + k * 32);
              umma_pair(acc, da, db, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
            }
            umma_commit_pair(&empty[s]);
          }
          __syncwarp();
        }
        if (ok && elect_one()) umma_commit_pair(&acc_full[buf]);  // without MMAs of its own: at once
        __syncwarp();
        ++it;
        if (MODE == LIN_OUT) break;
      }
      g += hi - lo;
    }
  } else if (warp >= 2 && warp < 10) {
    // ---------------- epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = smem + L::STG_OFF + (warp - 2) * 2 * 4096;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + half * (BN / 2);
    const uint32_t empty_leader[2] = {map_rank(smem_u32(&acc_empty[0]), 0), map_rank(smem_u32(&acc_empty[1]), 0)};
    float* s_bias = reinterpret_cast<float*>(smem + L::BIAS_OFF);
    if (lane == 0) {  // both accumulators are free at first: each CTA's is allocated
      mbar_arrive_cluster(empty_leader[0]);
      mbar_arrive_cluster(empty_leader[1]);
    }
    bool alive = true;
    int nst = 0;
    auto stage_wait = [&] {  // the store that last read staging tile nst & 1 is done
      if (lane == 0 && nst >= 2) bulk_wait_group_read<1>();
      __syncwarp();
    };
    auto stage_done = [&] {
      if (lane == 0) bulk_commit_group();
      ++nst;
    };
    int it = 0, g = 0;  // units and k-blocks before the tile
    for (int t = cluster; t < ntiles; t += nclusters) {
      int r0, c0, lo, hi;
      tile_at(t, r0, c0, lo, hi);
      // accumulator of the tile's (and of each of its chunks') first k-block, and the other one's offset
      const int acc1 = (g & (MW - 1)) * BN, acc2 = ACC - BN - acc1;
      g += hi - lo;
      const int rw = r0 + (int)rank * 128 + quarter * 32;  // the warp's first row
      const int r = rw + lane;
      const int cw = c0 + half * (BN / 2);                 // the warp's first column
      if (MODE == LIN_OUT) {
        const int buf = it & 1;
        if (!SWAP) {
          // the tile's bias goes through shared memory: read per row from global memory its 64
          // loads a chunk cost 25 us at the end of a product.  A warp that timed out takes the
          // others with it here (the barrier carries the AND of `alive`).
          __syncwarp();  // the last tile's stores branch by row
          if (!bar_and(alive, 1, 256)) break;
          const int q = (warp - 2) * 32 + lane;
          float bv = 0.f;
          if (q < BN) {
            if (p.bias && c0 + q < p.C) load_params<1>(p.bias, p.bias_bf16, c0 + q, 0.f, &bv);
            s_bias[q] = bv;
          }
          __syncwarp();
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        // the residual's first chunk is on its way before the product is ready
        const bool res_vec = !SWAP && p.residual && (p.ldr & 7) == 0 && aligned16_dev(p.residual);
        uint4 rq[8];
        auto fetch_res = [&](int n) {
          if (res_vec && r < rows && n + 64 <= p.C) {
            const uint4* q = reinterpret_cast<const uint4*>(p.residual + (int64_t)r * p.ldr + n);
#pragma unroll
            for (int i = 0; i < 8; ++i) rq[i] = q[i];
          }
        };
        if (!SWAP) fetch_res(cw);
        const bool ok = __all_sync(0xffffffffu, pair_wait(&acc_full[buf], (it >> 1) & 1));
        if (!ok) {
          if (SWAP) break;
          alive = false;
          continue;
        }
        tc_fence_after();
        if constexpr (SWAP) {
          // lane = row of w = column n of the output; the warp's tokens go by in steps of 16
#pragma unroll 1
          for (int cc = 0; cc < BN / 32; ++cc) {
            const int m0 = cw + cc * 16;
            uint32_t raw[16];
            __syncwarp();  // the load below is collective
            tmem_ld16_nowait(lane_base + buf * ACC + acc1 + cc * 16, raw);
            if (MW == 2 && hi - lo > 1) {  // the other warp's k-blocks
              uint32_t more[16];
              tmem_ld16_nowait(lane_base + buf * ACC + acc2 + cc * 16, more);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) + __uint_as_float(more[i]));
            } else {
              tmem_wait_ld();
            }
            if (cc == BN / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(empty_leader[buf]);
            }
            if (r >= rows) continue;
            if (ksplit > 1) {
              float* o = p.part + ((int64_t)(t % ksplit) * p.m + m0) * rows + r;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (m0 + i < cols) o[(int64_t)i * rows] = __uint_as_float(raw[i]);
              continue;
            }
            float b = 0.f, v[16];
            if (p.bias) load_params<1>(p.bias, p.bias_bf16, r, 0.f, &b);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(raw[i]) + b;
            if (p.pre) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (m0 + i < cols) p.pre[(int64_t)(m0 + i) * p.ldp + r] = __float2bfloat16_rn(v[i]);
            }
            act_values<16>(v, p.act);
            if (p.residual) {
              float e[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                e[i] = m0 + i < cols ? __bfloat162float(p.residual[(int64_t)(m0 + i) * p.ldr + r]) : 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += e[i];
            }
            bf16* o = reinterpret_cast<bf16*>(p.out) + (int64_t)m0 * p.ldo + r;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (m0 + i < cols) o[(int64_t)i * p.ldo] = __float2bfloat16_rn(v[i]);
          }
          ++it;
          continue;
        }
        const bool whole = rw + 32 <= rows;
#pragma unroll 1
        for (int cc = 0; cc < BN / 128; ++cc) {
          const int n = cw + cc * 64;
          uint32_t raw[64];
          __syncwarp();  // the loads below are collective
          tmem_ld32_nowait(lane_base + buf * ACC + acc1 + cc * 64, raw);
          tmem_ld32_nowait(lane_base + buf * ACC + acc1 + cc * 64 + 32, raw + 32);
          if (MW == 2 && hi - lo > 1) {  // the other warp's k-blocks
            uint32_t more[64];
            tmem_ld32_nowait(lane_base + buf * ACC + acc2 + cc * 64, more);
            tmem_ld32_nowait(lane_base + buf * ACC + acc2 + cc * 64 + 32, more + 32);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 64; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) + __uint_as_float(more[i]));
          } else {
            tmem_wait_ld();
          }
          if (cc == BN / 128 - 1) {  // the accumulator is read: release it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(empty_leader[buf]);
          }
          if (n >= p.C || rw >= rows) continue;
          const bool full_cols = n + 64 <= p.C;
          if (ksplit > 1 && whole && p.out_tma) {  // the map's rows: ksplit blocks of p.m
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (n + 32 * h >= p.C) continue;
              stage_wait();
              uint8_t* tb = stg + (nst & 1) * 4096;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(tb + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                    make_uint4(raw[32 * h + 4 * q], raw[32 * h + 4 * q + 1], raw[32 * h + 4 * q + 2], raw[32 * h + 4 * q + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) tma_store_2d(&tmOut, tb, n + 32 * h, t % ksplit * p.m + rw);
              stage_done();
            }
            continue;
          }
          if (ksplit > 1) {
            if (r < rows) {
              float* o = p.part + ((int64_t)(t % ksplit) * p.m + r) * p.C + n;
              if (full_cols && (p.C & 3) == 0) {
#pragma unroll
                for (int i = 0; i < 64; i += 4)
                  *reinterpret_cast<uint4*>(o + i) = make_uint4(raw[i], raw[i + 1], raw[i + 2], raw[i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                  if (n + i < p.C) o[i] = __uint_as_float(raw[i]);
              }
            }
            continue;
          }
          float v[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(raw[i]);
          if (p.bias) {
            const float4* bq = reinterpret_cast<const float4*>(s_bias + half * (BN / 2) + cc * 64);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 b = bq[i];
              v[4 * i] += b.x;
              v[4 * i + 1] += b.y;
              v[4 * i + 2] += b.z;
              v[4 * i + 3] += b.w;
            }
          }
          if (p.pre) {
            if (whole && p.pre_tma) {
              stage_wait();
              uint8_t* tb = stg + (nst & 1) * 4096;
              uint32_t w[16];
              pack32<false>(v, w);
              stage_row32(tb, lane, 0, w);
              pack32<false>(v + 32, w);
              stage_row32(tb, lane, 4, w);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) tma_store_2d(&tmPre, tb, n, rw);
              stage_done();
            } else if (r < rows) {
              bf16* o = p.pre + (int64_t)r * p.ldp + n;
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (n + i < p.C) o[i] = __float2bfloat16_rn(v[i]);
            }
          }
          act_values<64>(v, p.act);
          if (p.residual && r < rows) {
            if (res_vec && full_cols) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t w[4] = {rq[i].x, rq[i].y, rq[i].z, rq[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  v[8 * i + 2 * e] += __uint_as_float(w[e] << 16);
                  v[8 * i + 2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
                }
              }
            } else {
              const bf16* q = p.residual + (int64_t)r * p.ldr + n;
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (n + i < p.C) v[i] += __bfloat162float(q[i]);
            }
          }
          if (cc + 1 < BN / 128) fetch_res(n + 64);
          if (whole && p.out_tma) {
            stage_wait();
            uint8_t* tb = stg + (nst & 1) * 4096;
            uint32_t w[16];
            pack32<false>(v, w);
            stage_row32(tb, lane, 0, w);
            pack32<false>(v + 32, w);
            stage_row32(tb, lane, 4, w);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tma_store_2d(&tmOut, tb, n, rw);
            stage_done();
          } else if (r < rows) {
            bf16* o = reinterpret_cast<bf16*>(p.out) + (int64_t)r * p.ldo + n;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (n + i < p.C) o[i] = __float2bfloat16_rn(v[i]);
          }
        }
        ++it;
      } else {
        // LIN_GRAD: add the chunks in fp32 registers, then write the tile
        if (p.db_part && c0 == 0 && half == 0 && t % ksplit == 0 && r < rows) {
          float a = 0.f;
#pragma unroll 4
          for (int q = 0; q < p.db_chunks; ++q) a += p.db_part[(int64_t)q * p.R + r];
          p.db[r] = p.accumulate ? p.db[r] + a : a;
        }
        float acc[BN / 2];
#pragma unroll
        for (int i = 0; i < BN / 2; ++i) acc[i] = 0.f;
        bool ok = true;
        for (int kb = lo; kb < hi; kb += LT_CHUNK) {
          const int buf = it & 1;
          ok = __all_sync(0xffffffffu, pair_wait(&acc_full[buf], (it >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < BN / 64; ++c) {
            uint32_t raw[32];
            tmem_ld32_nowait(lane_base + buf * ACC + acc1 + c * 32, raw);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c * 32 + i] += __uint_as_float(raw[i]);
            if (MW == 2 && hi - kb > 1) {  // the other warp's k-blocks
              tmem_ld32_nowait(lane_base + buf * ACC + acc2 + c * 32, raw);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c * 32 + i] += __uint_as_float(raw[i]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(empty_leader[buf]);
          ++it;
        }
        if (!ok) break;
        const bool whole = rw + 32 <= rows;
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) {
          const int n = cw + c * 32;
          if (n >= p.C || rw >= rows) continue;
          const float* v = acc + c * 32;
          if (whole && p.out_tma) {
            stage_wait();
            uint8_t* tb = stg + (nst & 1) * 4096;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(tb + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (ksplit > 1)  // the map's rows: ksplit blocks of p.R
                tma_store_2d(&tmOut, tb, n, t % ksplit * p.R + rw);
              else if (p.accumulate)
                tma_reduce_add_2d(&tmOut, tb, n, rw);
              else
                tma_store_2d(&tmOut, tb, n, rw);
            }
            stage_done();
          } else if (r < rows && ksplit > 1) {
            float* o = p.part + ((int64_t)(t % ksplit) * p.R + r) * p.C + n;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n + i < p.C) o[i] = v[i];
          } else if (r < rows) {
            float* o = reinterpret_cast<float*>(p.out) + (int64_t)r * p.ldo + n;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n + i < p.C) o[i] = p.accumulate ? o[i] + v[i] : v[i];
          }
        }
      }
    }
    if (lane == 0 && nst > 0) bulk_wait_group_read<0>();  // staging outlives the stores' reads
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * ACC);
  }
}

}  // namespace jenga
