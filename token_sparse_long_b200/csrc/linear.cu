// Linear layer with bias, activation and residual in the product's epilogue, and its
// gradients: the dense pieces of an OPT-style feed-forward sub-block on retained rows (the
// Llama layer's projections are fused in layer.cu).
//
//   z = x w^T + bias,   y = act(z) + residual,   pre = z (kept for the backward, bf16)
//   dz = dy act'(pre),  dx = dz w,   dw (+)= dz^T x,   db (+)= sum_r dz
//
// bf16 operands, fp32 accumulation; z stays fp32 up to y's one rounding.  dz is rounded to bf16
// to be a tensor-core operand: exact for no activation and ReLU (dy or 0).  For GELU and SiLU the
// rounding (half a bf16 step, 2^-8 relative) is like that of the bf16 result in dx; the fp32 dw takes
// dz as three bf16 parts (24 bits, all of dz) in three passes over the rows -- with two parts dw
// was 4e-6 off, four times what fp32 sums lose.  db sums dz in fp32 before any rounding.
#include "linear_tc.cuh"

namespace jenga {

// dz = dy act'(pre) as bf16 (with PARTS = 3 also what the rounding left, twice), and partial
// column sums of dz: CTA (strip, chunk) takes 256 columns x the chunk's rows, eight columns per
// lane and four rows a step per warp (loads first: two matrices, one pass, bound by memory); the
// eight warps' sums are added in order, part[chunk][N].  Rows from the valid count up to the
// next multiple of 64 are written as zeros (the product over the rows reads whole 64-row
// blocks).  VEC: rows of dy and pre are whole 16-byte vectors.
template <bool VEC, bool WRITE, int PARTS>
__global__ void __launch_bounds__(256)
    linear_dz_kernel(const bf16* __restrict__ dy, int64_t ldy, const bf16* __restrict__ pre, int64_t ldp, int act,
                     int M, int N, const int32_t* n_kept, int blk, int rows_per, bf16* __restrict__ dz, int64_t ldz,
                     int64_t part_stride, float* __restrict__ part) {
  constexpr int STEP = 4, PER = VEC ? 8 : 1, NV = 8 / PER;  // unaligned: every 32nd column, element by element
  constexpr int CSTEP = VEC ? 8 : 32;
  __shared__ float s_sum[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int valid = valid_rows(RowMap{nullptr, n_kept, blk, 0, M});
  const int cl = VEC ? lane * 8 : lane, c = blockIdx.x * 256 + cl;  // first column in the strip and overall
  const int r_lo = blockIdx.y * rows_per;
  const int r_hi = min(min((valid + 63) / 64 * 64, M), r_lo + rows_per);
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  if (c < N) {
    for (int r0 = r_lo + warp; r0 < r_hi; r0 += 8 * STEP) {
      RowVec<bf16, PER> a[STEP][NV], b[STEP][NV];
#pragma unroll
      for (int u = 0; u < STEP; ++u) {
        const int r = r0 + u * 8;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          a[u][i].zero();
          b[u][i].zero();
          if (r < r_hi && r < valid && c + i * CSTEP < N) {
            a[u][i].load(dy + (int64_t)r * ldy + c + i * CSTEP);
            if (act != JENGA_ACT_NONE) b[u][i].load(pre + (int64_t)r * ldp + c + i * CSTEP);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < STEP; ++u) {
        const int r = r0 + u * 8;
        if (r >= r_hi) break;
        float d[8], z[8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          a[u][i].get(d + i * PER);
          b[u][i].get(z + i * PER);
        }
        if (act == JENGA_ACT_RELU) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = z[e] > 0.f ? d[e] : 0.f;
        } else if (act != JENGA_ACT_NONE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= act_slope(z[e], act);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += d[e];
        if (WRITE) {
          bf16* o = dz + (int64_t)r * ldz + c;
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (c + i * CSTEP < N) RowVec<bf16, PER>::store(o + q * part_stride + i * CSTEP, d + i * PER);
            if (q + 1 < PARTS) {  // what the rounding left; nothing of an infinity or a NaN
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float hi = __bfloat162float(__float2bfloat16_rn(d[e]));
                d[e] = fabsf(hi) < INFINITY ? d[e] - hi : 0.f;
              }
            }
          }
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < PER; ++e) s_sum[warp][cl + i * CSTEP + e] = sum[i * PER + e];
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < N) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a += s_sum[w][threadIdx.x];
    part[(int64_t)blockIdx.y * N + col] = a;
  }
}

// db[c] (+)= sum over the chunks, in order
__global__ void __launch_bounds__(128) linear_db_reduce_kernel(const float* __restrict__ part, int chunks, int N,
                                                               float* db, int accumulate) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= N) return;
  float a = 0.f;
  for (int p = 0; p < chunks; ++p) a += part[(int64_t)p * N + c];
  db[c] = accumulate ? db[c] + a : a;
}

// dw[r][c] (+)= the partial products added in order (row y of the grid)
__global__ void __launch_bounds__(256) linear_dw_sum_kernel(const float* __restrict__ part, int splits, int N, int K,
                                                            float* dw, int64_t ldw, int accumulate) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= K) return;
  const float* q = part + (int64_t)blockIdx.y * K + c;
  float a = 0.f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) a += q[(int64_t)s * N * K];
  float* o = dw + (int64_t)blockIdx.y * ldw + c;
  *o = accumulate ? *o + a : a;
}

// The rows of x past the last whole 64-row block, with zeros up to 64 rows (a device row count
// can end inside x, whose later rows may hold anything).
__global__ void __launch_bounds__(256) linear_tail_kernel(const bf16* __restrict__ x, int64_t ldx, int M, int K,
                                                          const int32_t* n_kept, int blk, bf16* __restrict__ tail,
                                                          int64_t ldt) {
  const int valid = valid_rows(RowMap{nullptr, n_kept, blk, 0, M});
  const int r0 = valid / 64 * 64, r = blockIdx.y;
  for (int c = blockIdx.x * 256 + threadIdx.x; c < K; c += gridDim.x * 256)
    tail[r * ldt + c] = r0 + r < valid ? x[(int64_t)(r0 + r) * ldx + c] : __float2bfloat16_rn(0.f);
}

// Forward for one or two rows of x: the weights are the whole traffic, read once.  Each CTA takes
// a consecutive share of w's rows and streams them through a ring of whole rows in shared memory
// (bulk copies by a warp of their own, up to 190 KB in flight an SM whatever the others do).
// A group of G warps takes a row: it holds its slice of x as fp32 pairs in registers (NV vectors
// of eight a thread), so a weight is read from shared memory once and used MT times, and with
// G = 1 eight rows are reduced side by side (all eight warps on one row: 400 clocks a row).  A
// warp needs about as long for a row as memory for eight, so its loads are issued eight at a
// time and vectors past the row's end are zeros, not branches (23 -> 21 us).  The sums of GV_BATCH
// rows at a time meet in shared memory, where the epilogue runs.  fp32 products and sums.  One
// row of 4096 into 32000: 46 us, 5.7 TB/s; into 11008: 21 us and into 4096: 10.6 us, of which
// 5.5 are the launch and the way to the first row (the tensor core kernel with its second launch:
// 27 and 17 us).  Four rows with G = 4 were slower than the tensor cores (63 against 50 us into
// 32000, 54 against 31 for 5120 into 13824).
constexpr int GV_BATCH = 64;
constexpr int GV_MAX_STAGES = 64;
template <int MT, int NV>
__global__ void __launch_bounds__(288, 1)
    linear_rows_kernel(const bf16* __restrict__ w, int64_t ldw, const bf16* __restrict__ x, int64_t ldx, int N, int K,
                       int G, int stages, LinArgs p) {
  constexpr int NB = NV < 8 ? NV : 8;  // vectors of a row in flight to registers
  static_assert(GV_BATCH * MT <= 256, "a thread finishes one value of a batch");
  extern __shared__ __align__(128) uint8_t s_w[];
  __shared__ uint64_t s_full[GV_MAX_STAGES], s_empty[GV_MAX_STAGES];
  __shared__ float s_part[2][GV_BATCH][MT][8];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int valid = valid_rows(RowMap{nullptr, p.n_kept, p.blk, 0, p.m});
  const int lo = (int)((int64_t)N * blockIdx.x / gridDim.x), hi = (int)((int64_t)N * (blockIdx.x + 1) / gridDim.x);
  const uint32_t row_bytes = (uint32_t)K * 2;
  if (valid == 0) return;
  if (warp == 8) {
    // ---------------- producer: its copies start before the others have come this far
    for (int i = lane; i < stages; i += 32) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], G);
    }
    fence_barrier_init();
    __syncwarp();
    asm volatile("bar.arrive 2, 288;" ::: "memory");
    int s = 0, ph = 1;  // the first lap finds every stage free
    for (int n = lo; n < hi; ++n) {
      if (!__all_sync(0xffffffffu, poll_wait(&s_empty[s], ph, SITE_LINEAR))) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(&s_full[s], row_bytes);
        bulk_load_1d(s_w + (size_t)s * row_bytes, w + (int64_t)n * ldw, row_bytes, &s_full[s]);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    return;
  }
  // ---------------- eight warps of dot products
  const int groups = 8 / G, grp = warp / G, gwarp = warp - grp * G;
  const int nvec = K / 8, v0 = gwarp * 32 + lane, step = G * 32;
  uint64_t xf[MT][NV][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < valid && v0 + i * step < nvec)
        v = *reinterpret_cast<const uint4*>(x + (int64_t)m * ldx + (int64_t)(v0 + i * step) * 8);
      vec_pairs<bf16>(v, xf[m][i]);
    }
  asm volatile("bar.sync 2, 288;" ::: "memory");  // the barriers are ready
  bool ok = true;
  int s = grp, ph = 0;  // the group's stage (stages is a multiple of groups)
  for (int b0 = lo, bi = 0; b0 < hi; b0 += GV_BATCH, bi ^= 1) {
    const int b1 = min(b0 + GV_BATCH, hi);
    // the value that this thread finishes below, and its bias
    const int fm = threadIdx.x / (b1 - b0), fq = threadIdx.x - fm * (b1 - b0);
    float bias = 0.f;
    if (fm < MT) load_params<1>(p.bias, p.bias_bf16, b0 + fq, 0.f, &bias);
    for (int n = b0 + grp; n < b1; n += groups) {
      ok = __all_sync(0xffffffffu, poll_wait(&s_full[s], ph, SITE_LINEAR));
      if (!ok) break;
      const uint8_t* row = s_w + (size_t)s * row_bytes + v0 * 16;
      uint64_t acc[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = 0;
#pragma unroll
      for (int i0 = 0; i0 < NV; i0 += NB) {
        uint4 raw[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          raw[i] = make_uint4(0, 0, 0, 0);
          if (v0 + (i0 + i) * step < nvec) raw[i] = *reinterpret_cast<const uint4*>(row + (i0 + i) * step * 16);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          uint64_t f[4];
          vec_pairs<bf16>(raw[i], f);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][e] = ffma2(f[e], xf[m][i0 + i][e], acc[m][e]);
        }
      }
      __syncwarp();  // every lane has read the row
      if (lane == 0) mbar_arrive(&s_empty[s]);
      float t[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        t[m] = pair_sum(fadd2(fadd2(acc[m][0], acc[m][1]), fadd2(acc[m][2], acc[m][3])));
      // lanes halve the rows of x among them as they add: after log2(MT) exchanges lanes
      // 32/MT m .. of row m hold one sum each
#pragma unroll
      for (int o = 16, c = MT / 2; o > 0; o >>= 1, c /= 2) {
        if (c > 0) {
          const bool up = lane & o;
#pragma unroll
          for (int m = 0; m < c; ++m) {
            const float give = up ? t[m] : t[m + c], keep = up ? t[m + c] : t[m];
            t[m] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        } else {
          t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
        }
      }
      if (lane % (32 / MT) == 0) s_part[bi][n - b0][lane / (32 / MT)][gwarp] = t[0];
      s += groups;
      if (s >= stages) {
        s -= stages;
        ph ^= 1;
      }
    }
    if (!bar_and(ok, 1, 256)) return;  // a warp that timed out takes the others with it
    if (fm < MT && fm < valid) {
      float z = 0.f;
      for (int k = 0; k < G; ++k) z += s_part[bi][fq][fm][k];
      lin_finish(p, fm, b0 + fq, z + bias);
    }
  }
}

// ------------------------------------------------------------------ host
struct LinMats {
  CUtensorMap a, a2, a3, b, tail, out, pre;
};

template <int BN, bool AMN, bool BMN, int MODE, bool SWAP>
static jenga_status linear_launch(const LinMats& m, const LinArgs& p, const char* name, cudaStream_t st) {
  using L = LinSmem<BN, SWAP>;
  auto kernel = linear_tc_kernel<BN, AMN, BMN, MODE, SWAP>;
  JENGA_CUDA_TRY(allow_smem((const void*)kernel, L::TOTAL));
  const int64_t tiles = (int64_t)((p.R + 255) / 256) * ((p.C + BN - 1) / BN) * p.ksplit;
  const int pairs = sm_count() / 2;
  const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
  const int ps = prof_begin(name, st);
  kernel<<<grid, lin_threads<BN>, L::TOTAL, st>>>(m.a, m.a2, m.a3, m.b, m.tail, m.out, m.pre, p);
  prof_end(ps, st);
  JENGA_LAUNCH_CHECK();
  return JENGA_OK;
}

// bf16 tensor map for an output of 32-row tiles; false when the matrix is not 16-byte aligned
static bool out_map(CUtensorMap* map, const void* base, int rows, int cols, int64_t ld) {
  return base && is16(base) && ld % 8 == 0 && make_tmap_bf16(map, base, rows, cols, ld, 32) == JENGA_OK;
}

// Shape of a forward or dx product [M, N] over `red`: operands swapped (and the narrow side's
// tile), tile width, ranges of the reduction.  Costs in k-blocks of a 256-wide tile (530 clocks
// measured; a narrower tile's take 215 to 250 with operands in L2, but about 400 when they come
// from HBM, which few rows make the rule: over M 16 to 4096 and seven pairs of N and K, 0.75 was
// never more than 3% behind 0.5 or 0.6 but at M 512 4096->1024, and up to 13% ahead of them).
// A further tile of a cluster costs its epilogue's start;
// a split adds the pass over the partial products: a launch, and 0.8 MB a k-block of time.
struct LinShape {
  bool swap;
  int bn, ksplit;
};
static LinShape lin_shape(int M, int N, int red) {
  const int pairs = sm_count() / 2, nkb = (red + 63) / 64;
  LinShape best{};
  double cost = 1e300;
  auto consider = [&](bool swap, int bn) {
    const int64_t tiles = (int64_t)(((swap ? N : M) + 255) / 256) * (((swap ? M : N) + bn - 1) / bn);
    const double per = swap || bn < 256 ? 0.75 : 1.0, fill = 1.5;
    for (int s = 1; s <= (M < 65536 ? 16 : 1) && s <= 1 + nkb / 8; ++s) {  // linear_finish: a grid row per row
      const double waves = (double)((tiles * s + pairs - 1) / pairs);
      double c = waves * (per * ((nkb + s - 1) / s) + fill);
      if (s > 1) c += 12.0 + (double)s * M * N * 8.0 / 0.8e6;
      if (c < cost * 0.97) {
        cost = c;
        best = LinShape{swap, bn, s};
      }
    }
  };
  if (M > 128 || N <= 128) {
    consider(false, 256);
    consider(false, 128);
  } else {
    consider(true, M <= 32 ? 32 : (M <= 64 ? 64 : 128));
  }
  return best;
}
static size_t lin_part_bytes(const LinShape& s, int M, int N) {
  return s.ksplit > 1 ? (size_t)s.ksplit * M * N * sizeof(float) + 256 : 0;
}

// Is the forward a pass over the rows of w (linear_rows)?  x as fp32 has to fit the registers of eight
// warps; rows of w are copied whole, in multiples of 16 bytes.
static bool lin_rows_ok(int M, int K) { return M <= 2 && K % 8 == 0 && K <= 16384; }

// Ring of the rows pass: 128 registers of x a thread at the most, as few warps a row as that
// allows, and a whole number of stages per group of warps, so that a stage always belongs to
// one group: a group that met a stage after another group's row would wait by parity for a phase two
// ahead, which passes at once while that row is still on its way.
constexpr int GV_ROOM = 192 * 1024;
struct LinRows {
  int G, nv, stages;
};
static LinRows lin_rows_shape(int M, int K) {
  LinRows r{1, 0, 0};
  while ((K / 8 + 32 * r.G - 1) / (32 * r.G) > 16 / M) r.G *= 2;
  r.nv = (K / 8 + 32 * r.G - 1) / (32 * r.G);
  r.stages = GV_ROOM / (K * 2);
  if (r.stages > GV_MAX_STAGES) r.stages = GV_MAX_STAGES;
  r.stages -= r.stages % (8 / r.G);
  return r;
}

// forward or dx: x side [M, red] (K-major), weight side [N, red] K-major or (WMN) [red, N]
template <bool WMN>
static jenga_status lin_out(const LinShape& s, const void* x, int64_t ldx, const void* w, int64_t ldw, int M, int N,
                            int red, LinArgs p, void* part, const char* name, cudaStream_t st) {
  LinMats m;
  p.m = M;
  p.nkb = (red + 63) / 64;
  p.passes = 1;
  p.ksplit = s.ksplit;
  p.part = (float*)(((uintptr_t)part + 255) & ~uintptr_t(255));
  const int wr = WMN ? red : N, wc = WMN ? N : red;  // the weight matrix in memory
  if (s.swap) {
    p.R = N;
    p.C = M;
    JENGA_TRY(make_tmap_bf16(&m.a, w, wr, wc, ldw, WMN ? 64 : 128));
    JENGA_TRY(make_tmap_bf16(&m.b, x, M, red, ldx, s.bn / 2));
    m.a2 = m.a3 = m.tail = m.out = m.pre = m.a;
    JENGA_TRY((s.bn == 32   ? linear_launch<32, WMN, false, LIN_OUT, true>(m, p, name, st)
               : s.bn == 64 ? linear_launch<64, WMN, false, LIN_OUT, true>(m, p, name, st)
                            : linear_launch<128, WMN, false, LIN_OUT, true>(m, p, name, st)));
  } else {
    p.R = M;
    p.C = N;
    JENGA_TRY(make_tmap_bf16(&m.a, x, M, red, ldx, 128));
    JENGA_TRY(make_tmap_bf16(&m.b, w, wr, wc, ldw, WMN ? 64 : s.bn / 2));
    m.a2 = m.a3 = m.tail = m.out = m.pre = m.a;
    if (s.ksplit == 1) {
      p.out_tma = out_map(&m.out, p.out, M, N, p.ldo);
      p.pre_tma = out_map(&m.pre, p.pre, M, N, p.ldp);
    } else {
      p.out_tma = N % 4 == 0 && make_tmap_f32(&m.out, p.part, (uint64_t)s.ksplit * M, N, N, 32) == JENGA_OK;
    }
    JENGA_TRY((s.bn == 256 ? linear_launch<256, false, WMN, LIN_OUT, false>(m, p, name, st)
                           : linear_launch<128, false, WMN, LIN_OUT, false>(m, p, name, st)));
  }
  if (s.ksplit > 1) {
    const int ps = prof_begin("linear_finish", st);
    if (N % 4 == 0)
      linear_finish_kernel<4><<<dim3((N + 511) / 512, M), 128, 0, st>>>(p, N);
    else
      linear_finish_kernel<1><<<dim3((N + 127) / 128, M), 128, 0, st>>>(p, N);
    prof_end(ps, st);
    JENGA_LAUNCH_CHECK();
  }
  return JENGA_OK;
}

static bool lin_operand_ok(const void* p, int64_t ld) { return is16(p) && ld % 8 == 0; }
// the pitch of x or w: a single row has none, whatever the caller's stride says
static int64_t lin_pitch(int64_t rows, int64_t ld) { return rows == 1 ? (ld + 7) / 8 * 8 : ld; }

static int dz_rows_per(int M, int N) {  // rows per chunk of linear_dz: about four CTAs an SM, whole steps of 32
  const int strips = (N + 255) / 256;
  int chunks = (4 * sm_count() + strips - 1) / strips;
  int per = (M + chunks - 1) / chunks;
  per = (per + 31) / 32 * 32;
  return per;
}

// parts that dz is held in: all of its 24 bits for dw after a smooth activation
static int dz_parts(int act) { return act == JENGA_ACT_GELU || act == JENGA_ACT_SILU ? 3 : 1; }

// ranges of dw's reduction when its tiles leave SM pairs idle (at least eight k-blocks each); the
// sum over them then takes a pass of its own over N x K values, at most 37 tiles of them
static int dw_splits(int M, int N, int K, int act) {
  const int pairs = sm_count() / 2, nkb = (M + 63) / 64 * dz_parts(act);
  const int64_t tiles = (int64_t)((N + 255) / 256) * ((K + 127) / 128);
  if (tiles * 2 > pairs || nkb < 32) return 1;
  int s = (int)(pairs / tiles);
  if (s > nkb / 8) s = nkb / 8;
  return s > 8 ? 8 : s;
}

struct LinBwdWs {
  bf16 *dz, *tail;  // dz: `parts` matrices [M, ldz]
  float *part, *dxpart, *dwpart;
  int64_t ldz, ldt, stride;
  size_t bytes;
};
static LinBwdWs lin_bwd_carve(void* ws, int M, int N, int K, int act) {
  LinBwdWs w;
  w.ldz = (N + 63) / 64 * 64;  // whole 128-byte lines: a box of other rows takes TMA 1.2 to 1.4 times as long
  w.ldt = (K + 63) / 64 * 64;
  w.stride = (int64_t)M * w.ldz;
  Carve c(ws);
  w.dz = c.take<bf16>((size_t)w.stride * dz_parts(act));
  w.tail = c.take<bf16>((size_t)64 * w.ldt);
  const int per = dz_rows_per(M, N);
  w.part = c.take<float>((size_t)((M + per - 1) / per) * N);
  w.dxpart = c.take<float>((lin_part_bytes(lin_shape(M, K, N), M, K) + 3) / 4);
  const int ks = dw_splits(M, N, K, act);
  w.dwpart = c.take<float>(ks > 1 ? (size_t)ks * N * K : 0);
  w.bytes = c.used();
  return w;
}

static bool lin_sizes_ok(int M, int N, int K) { return M <= (1 << 30) && N <= (1 << 24) && K <= (1 << 24); }
static jenga_status lin_check(const char* who, int M, int N, int K, const int32_t* n_kept, int blk, int act) {
  JENGA_CHECK_ARG(M >= 0 && N >= 1 && K >= 1 && blk >= 1, "%s: bad sizes M=%d N=%d K=%d blk=%d", who, M, N, K, blk);
  JENGA_CHECK_ARG(lin_sizes_ok(M, N, K), "%s: sizes too large M=%d N=%d K=%d", who, M, N, K);
  JENGA_CHECK_ARG(!n_kept || M % blk == 0, "%s: M (%d) must be whole blocks of %d", who, M, blk);
  JENGA_CHECK_ARG(act >= JENGA_ACT_NONE && act <= JENGA_ACT_SILU, "%s: activation %d", who, act);
  return JENGA_OK;
}

}  // namespace jenga

using namespace jenga;

extern "C" size_t jenga_linear_fwd_workspace_bytes(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || !lin_sizes_ok(M, N, K)) return 0;
  return lin_rows_ok(M, K) ? 0 : lin_part_bytes(lin_shape(M, N, K), M, N);
}

extern "C" jenga_status jenga_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                         jenga_dtype bias_dt, jenga_activation act, const void* residual, int64_t ldr,
                                         int M, int N, int K, const int32_t* n_kept, int blk, void* y, int64_t ldy,
                                         void* pre, int64_t ldp, void* ws, size_t ws_bytes, jenga_stream_t stream) {
  JENGA_TRY(lin_check("jenga_linear_fwd", M, N, K, n_kept, blk, act));
  JENGA_CHECK_ARG(bias_dt == JENGA_F32 || bias_dt == JENGA_BF16, "jenga_linear_fwd: bias dtype");
  JENGA_CHECK_ARG(ldx >= K && ldw >= K && ldy >= N && (!residual || ldr >= N) && (!pre || ldp >= N),
                  "jenga_linear_fwd: row pitch smaller than the row");
  if (M == 0) return JENGA_OK;
  JENGA_CHECK_ARG(x && w && y, "jenga_linear_fwd: null pointer");
  ldx = lin_pitch(M, ldx);
  ldw = lin_pitch(N, ldw);
  JENGA_CHECK_ARG(lin_operand_ok(x, ldx) && lin_operand_ok(w, ldw),
                  "jenga_linear_fwd: x and w need 16-byte aligned rows (pitch a multiple of 8)");
  const auto apart = [&](size_t ws_used) {
    return outputs_apart(
        {mat_span(y, M, N, ldy, 2), mat_span(pre, M, N, ldp, 2), vec_span(ws, ws_used, 1)},
        {mat_span(residual, M, N, ldr, 2, true), mat_span(x, M, K, ldx, 2), mat_span(w, N, K, ldw, 2),
         vec_span(bias, N, bias_dt == JENGA_F32 ? 4 : 2), vec_span(n_kept, 1, 4)});
  };
  const char* met = "jenga_linear_fwd: an output or the workspace overlaps an input or another output (allowed only for "
                    "y = residual, the same matrix)";
  JENGA_CHECK_ARG(apart(0), "%s", met);
  const LinShape shape = lin_shape(M, N, K);
  const size_t need = jenga_linear_fwd_workspace_bytes(M, N, K);
  if (need && (!ws || ws_bytes < need))
    return fail(JENGA_EWORKSPACE, "jenga_linear_fwd: workspace %zu < %zu", ws ? ws_bytes : (size_t)0, need);
  JENGA_CHECK_ARG(!need || apart(need), "%s", met);
  LinArgs p{};
  p.n_kept = n_kept;
  p.blk = blk;
  p.bias = bias;
  p.bias_bf16 = bias_dt == JENGA_BF16;
  p.act = act;
  p.residual = (const bf16*)residual;
  p.ldr = ldr;
  p.out = y;
  p.ldo = ldy;
  p.pre = (bf16*)pre;
  p.ldp = ldp;
  cudaStream_t st = (cudaStream_t)stream;
  if (lin_rows_ok(M, K)) {
    p.m = M;
    const LinRows r = lin_rows_shape(M, K);
    const unsigned grid = (unsigned)(N < sm_count() ? N : sm_count());
    const int ps = prof_begin("linear_rows", st);
    auto go = [&](auto kernel) {
      const cudaError_t e = allow_smem((const void*)kernel, GV_ROOM);
      if (e == cudaSuccess)
        kernel<<<grid, 288, (size_t)r.stages * K * 2, st>>>((const bf16*)w, ldw, (const bf16*)x, ldx, N, K, r.G, r.stages,
                                                            p);
      return e;
    };
    JENGA_CUDA_TRY(M == 1   ? (r.nv <= 4   ? go(linear_rows_kernel<1, 4>)
                               : r.nv <= 8 ? go(linear_rows_kernel<1, 8>)
                                           : go(linear_rows_kernel<1, 16>))
                            : (r.nv <= 4 ? go(linear_rows_kernel<2, 4>) : go(linear_rows_kernel<2, 8>)));
    prof_end(ps, st);
    JENGA_LAUNCH_CHECK();
    return JENGA_OK;
  }
  return lin_out<false>(shape, x, ldx, w, ldw, M, N, K, p, ws, "linear_fwd", st);
}

// Test hook: the rows pass's warps per row and ring stages for M rows of x of K columns.
extern "C" jenga_status jenga_test_linear_rows_shape(int M, int K, int* warps_per_row, int* stages) {
  JENGA_CHECK_ARG(warps_per_row && stages && M >= 1 && K >= 1 && lin_rows_ok(M, K),
                  "jenga_test_linear_rows_shape: M=%d K=%d", M, K);
  const LinRows r = lin_rows_shape(M, K);
  *warps_per_row = r.G;
  *stages = r.stages;
  return JENGA_OK;
}

extern "C" size_t jenga_linear_bwd_workspace_bytes(int M, int N, int K, jenga_activation act) {
  if (M < 1 || N < 1 || K < 1 || !lin_sizes_ok(M, N, K)) return 0;
  return lin_bwd_carve(nullptr, M, N, K, act).bytes;
}

extern "C" jenga_status jenga_linear_bwd(const void* dy, int64_t ldy, const void* x, int64_t ldx, const void* w,
                                         int64_t ldw, jenga_activation act, const void* pre, int64_t ldp, int M, int N,
                                         int K, const int32_t* n_kept, int blk, void* dx, int64_t ldd, float* dw,
                                         int64_t lddw, float* db, int accumulate, void* ws, size_t ws_bytes,
                                         jenga_stream_t stream) {
  JENGA_TRY(lin_check("jenga_linear_bwd", M, N, K, n_kept, blk, act));
  JENGA_CHECK_ARG(ldy >= N && (!dw || (ldx >= K && lddw >= K)) && (!dx || (ldw >= K && ldd >= K)) &&
                      (act == JENGA_ACT_NONE || ldp >= N),
                  "jenga_linear_bwd: row pitch smaller than the row");
  cudaStream_t st = (cudaStream_t)stream;
  if (M == 0) {  // empty sums
    if (!accumulate && dw)
      JENGA_CUDA_TRY(cudaMemset2DAsync(dw, (size_t)lddw * 4, 0, (size_t)K * 4, (size_t)N, st));
    if (!accumulate && db) JENGA_CUDA_TRY(cudaMemsetAsync(db, 0, (size_t)N * 4, st));
    return JENGA_OK;
  }
  JENGA_CHECK_ARG(dy && (act == JENGA_ACT_NONE || pre) && (!dw || x) && (!dx || w), "jenga_linear_bwd: null pointer");
  if (!dx && !dw && !db) return JENGA_OK;
  ldx = lin_pitch(M, ldx);
  ldw = lin_pitch(N, ldw);
  JENGA_CHECK_ARG((!dw || lin_operand_ok(x, ldx)) && (!dx || lin_operand_ok(w, ldw)),
                  "jenga_linear_bwd: x and w need 16-byte aligned rows (pitch a multiple of 8)");
  if (act == JENGA_ACT_NONE) pre = nullptr;
  if (!dw) x = nullptr;
  if (!dx) w = nullptr;
  const auto apart = [&](size_t ws_used) {
    return outputs_apart({mat_span(dx, M, K, ldd, 2), mat_span(dw, N, K, lddw, 4), vec_span(db, N, 4),
                          vec_span(ws, ws_used, 1)},
                         {mat_span(dy, M, N, ldy, 2), mat_span(x, M, K, ldx, 2), mat_span(w, N, K, ldw, 2),
                          mat_span(pre, M, N, ldp, 2), vec_span(n_kept, 1, 4)});
  };
  const char* met = "jenga_linear_bwd: an output or the workspace overlaps an input or another output";
  JENGA_CHECK_ARG(apart(0), "%s", met);
  // without dw one bf16 copy of dz is all that is kept
  const jenga_activation ws_act = dw || act == JENGA_ACT_NONE ? act : JENGA_ACT_RELU;
  const size_t need = jenga_linear_bwd_workspace_bytes(M, N, K, ws_act);
  if (!ws || ws_bytes < need)
    return fail(JENGA_EWORKSPACE, "jenga_linear_bwd: workspace %zu < %zu", ws ? ws_bytes : (size_t)0, need);
  JENGA_CHECK_ARG(apart(need), "%s", met);
  const LinBwdWs W = lin_bwd_carve(ws, M, N, K, ws_act);
  // dy itself is the operand when nothing has to be computed, aligned or cut off at a device count
  const bool direct = act == JENGA_ACT_NONE && !n_kept && lin_operand_ok(dy, ldy);
  const bf16* dz = direct ? (const bf16*)dy : W.dz;
  const int64_t ldz = direct ? ldy : W.ldz;
  const int parts = dw ? dz_parts(act) : 1;
  const int per = dz_rows_per(M, N), chunks = (M + per - 1) / per;
  if (!direct || db) {
    float* part = db ? W.part : nullptr;
    const bool vec = N % 8 == 0 && lin_operand_ok(dy, ldy) && (!pre || lin_operand_ok(pre, ldp));
    const dim3 grid((N + 255) / 256, chunks);
    auto go = [&](auto kernel) {
      kernel<<<grid, 256, 0, st>>>((const bf16*)dy, ldy, (const bf16*)pre, ldp, act, M, N, n_kept, blk, per, W.dz, W.ldz,
                                   W.stride, part);
    };
    const int ps = prof_begin("linear_dz", st);
    if (direct)
      vec ? go(linear_dz_kernel<true, false, 1>) : go(linear_dz_kernel<false, false, 1>);
    else if (vec)
      parts == 3 ? go(linear_dz_kernel<true, true, 3>) : go(linear_dz_kernel<true, true, 1>);
    else
      parts == 3 ? go(linear_dz_kernel<false, true, 3>) : go(linear_dz_kernel<false, true, 1>);
    prof_end(ps, st);
    JENGA_LAUNCH_CHECK();
    if (db && !dw) {  // with dw its kernel adds them
      const int p2 = prof_begin("linear_db_reduce", st);
      linear_db_reduce_kernel<<<(N + 127) / 128, 128, 0, st>>>(W.part, chunks, N, db, accumulate);
      prof_end(p2, st);
      JENGA_LAUNCH_CHECK();
    }
  }
  if (dx) {
    LinArgs p{};
    p.n_kept = n_kept;
    p.blk = blk;
    p.out = dx;
    p.ldo = ldd;
    JENGA_TRY(lin_out<true>(lin_shape(M, K, N), dz, ldz, w, ldw, M, K, N, p, W.dxpart, "linear_dx", st));
  }
  if (dw) {
    LinArgs p{};
    p.R = N;
    p.C = K;
    p.m = M;
    p.nkb = (M + 63) / 64;
    p.ksplit = dw_splits(M, N, K, act);
    p.part = W.dwpart;
    p.db_part = db ? W.part : nullptr;
    p.db_chunks = chunks;
    p.db = db;
    p.passes = parts;
    p.n_kept = n_kept;
    p.blk = blk;
    p.out = dw;
    p.ldo = lddw;
    p.accumulate = accumulate;
    p.tail = n_kept != nullptr;
    LinMats m;
    JENGA_TRY(make_tmap_bf16(&m.a, dz, M, N, ldz, 64));
    m.a2 = m.a3 = m.tail = m.out = m.pre = m.a;
    if (parts == 3) {
      JENGA_TRY(make_tmap_bf16(&m.a2, W.dz + W.stride, M, N, W.ldz, 64));
      JENGA_TRY(make_tmap_bf16(&m.a3, W.dz + 2 * W.stride, M, N, W.ldz, 64));
    }
    JENGA_TRY(make_tmap_bf16(&m.b, x, M, K, ldx, 64));
    if (p.tail) {
      const int ps = prof_begin("linear_tail", st);
      linear_tail_kernel<<<dim3((K + 1023) / 1024, 64), 256, 0, st>>>((const bf16*)x, ldx, M, K, n_kept, blk, W.tail,
                                                                      W.ldt);
      prof_end(ps, st);
      JENGA_LAUNCH_CHECK();
      JENGA_TRY(make_tmap_bf16(&m.tail, W.tail, 64, K, W.ldt, 64));
    }
    if (p.ksplit > 1)
      p.out_tma = K % 4 == 0 && make_tmap_f32(&m.out, p.part, (uint64_t)p.ksplit * N, K, K, 32) == JENGA_OK;
    else
      p.out_tma = is16(dw) && lddw % 4 == 0 && make_tmap_f32(&m.out, dw, N, K, lddw, 32) == JENGA_OK;
    const int64_t t256 = (int64_t)((N + 255) / 256) * ((K + 255) / 256);
    JENGA_TRY((t256 >= sm_count() / 2 ? linear_launch<256, true, true, LIN_GRAD, false>(m, p, "linear_dw", st)
                                      : linear_launch<128, true, true, LIN_GRAD, false>(m, p, "linear_dw", st)));
    if (p.ksplit > 1) {
      const int ps = prof_begin("linear_dw_sum", st);
      linear_dw_sum_kernel<<<dim3((K + 255) / 256, N), 256, 0, st>>>(W.dwpart, p.ksplit, N, K, dw, lddw, accumulate);
      prof_end(ps, st);
      JENGA_LAUNCH_CHECK();
    }
  }
  return JENGA_OK;
}
