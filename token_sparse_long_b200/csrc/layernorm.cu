// Layer norm over the rows of a matrix, forward and backward (the norm of OPT-style layers,
// one of the model families of the Jenga notes' evaluation; the Llama layer's RMSNorm has its
// own fused kernels).
//
//   mean = sum_c x / h,  var = sum_c (x - mean)^2 / h,  rstd = (var + eps)^(-1/2)
//   y    = (x - mean) rstd gamma + beta
// With n = (x - mean) rstd and g = dy gamma:
//   dx     = rstd (g - mean_c(g) - n mean_c(g n)) (+ dres)
//   dgamma = sum_r dy n,   dbeta = sum_r dy
// All arithmetic is fp32 on the rows as loaded (the row stays in registers, so the variance is
// the centred two-pass one: no cancellation for rows far off zero); y and dx are rounded once.
// Rows can be read through the kept-block list like the Llama layer's fused norm does, and
// the backward then writes dx to the same sequence rows.
#include "rows.cuh"

namespace jenga {

// ------------------------------------------------------------------ aligned rows
// Rows of whole 16-byte vectors stream through a shared-memory ring: the row group's first warp
// starts bulk copies ahead, a queue that does not depend on how many warps the registers leave
// room for.  (An elected lane of the converged warp issues them: from a divergent lane a copy
// takes about 100 clocks, on which the other warps wait at the next barrier; the backward of
// 26240 x 4096 took 126 instead of 115 us.)  A group of `gw` warps -- one, or the whole CTA --
// owns a row at a time and a thread the same NV vectors of every row; groups are persistent
// (group g of G takes rows g, g + G, ...), so what belongs to a column stays in registers.
// Arithmetic is on fp32 pairs.

// fp32 pairs as one 16-byte vector
template <typename T>
__device__ __forceinline__ uint4 pairs_vec(const uint64_t* f) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2unpack(f[i], a, b);
      w[i] = pack_bf2(a, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b;
      f2unpack(f[i], a, b);
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Rows in the ring.  More only queue up at the start, while the first warp, which issues them, should
// be at its first row: 4096 x 4096 bf16, forward 16.3 us with eight and 15.0 with two, backward
// 35.7 with six and 33.7 with four (two: 42, a stage of the backward is free a row later).
constexpr int LN_FWD_STAGES = 2, LN_BWD_STAGES = 4;
constexpr int LN_MAX_STAGES = 4;

// Row group state of the ring: per stage a barrier and the sequence row (-1: a bad list
// entry).
struct LnRing {
  uint64_t bar[LN_MAX_STAGES];
  int64_t row[LN_MAX_STAGES];
};

// Arm stage s for compact row r at sequence row `row` (one lane).  False for a bad list entry, which
// is recorded; the stage then completes at once.
__device__ __forceinline__ bool ln_claim(LnRing& st, int64_t row, int r, int s, uint32_t bytes) {
  st.row[s] = row;
  if (row < 0) {
    record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
    mbar_arrive(&st.bar[s]);
    return false;
  }
  mbar_arrive_expect_tx(&st.bar[s], bytes);
  return true;
}

// Barrier of a row group (a warp, or else the CTA) that also agrees on `ok`: a warp that timed out
// takes all with it.  (Barrier 0 only: a barrier number in a register would reserve all 16 for
// the CTA, and four such CTAs are all that an SM then holds.)
__device__ __forceinline__ bool group_agree(bool ok, int gw) {
  if (gw > 1) return __syncthreads_and(ok);
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();
  return ok;
}

// Forward: gamma and beta in registers; a row is unpacked once, centred in place, and takes one
// barrier.  FULL: every thread holds NV vectors (no bounds in the loop).
template <typename T, int NV, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 128 ? (sizeof(T) == 2 ? 4 : 6) : (MAXT <= 160 ? 3 : (MAXT <= 320 ? 2 : 1)))
    layernorm_fwd_ring_kernel(const T* x, int64_t ldx, RowMap map, int h, int gw, int stages, const void* gamma,
                              const void* beta, int wbf16, float eps, T* y, int64_t ldy, float* mean_out,
                              float* rstd_out) {
  constexpr int VEC = 16 / (int)sizeof(T), NP = VEC / 2;
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ LnRing s_ring[4];
  __shared__ float2 s_red[2][32];  // [parity][warp]: sum, squares about the warp's mean
  __shared__ float2 s_cnt[32];     // elements of a row that warp w of its group holds, and 1 / that
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int groups = (blockDim.x >> 5) / gw, grp = warp / gw, gwarp = warp - grp * gw;
  const int nvec = h / VEC, step = gw * 32, t0 = gwarp * 32 + lane;
  const int valid = valid_rows(map);
  const int G = gridDim.x * groups, r0 = blockIdx.x * groups + grp;
  const bool leader = t0 == 0;
  float cnt = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) cnt += (float)(max(0, min(32, nvec - (gwarp * 32 + i * step))) * VEC);
  const float inv_cnt = cnt > 0.f ? 1.f / cnt : 0.f, inv_h = 1.f / (float)h;
  if (lane == 0) s_cnt[warp] = make_float2(cnt, inv_cnt);
  const uint32_t row_bytes = (uint32_t)h * sizeof(T);
  uint8_t* ring = s_rows + (size_t)grp * stages * row_bytes;
  LnRing& st = s_ring[grp];
  if (leader) {
    for (int i = 0; i < stages; ++i) mbar_init(&st.bar[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  auto start = [&](int64_t r, int s) {  // first warp of the group: row r into stage s
    if (r >= valid) return;
    const int64_t row = sequence_row(map, (int)r);
    if (!elect_one()) return;
    if (!ln_claim(st, row, (int)r, s, row_bytes)) return;
    bulk_load_1d(ring + (size_t)s * row_bytes, x + row * ldx, row_bytes, &st.bar[s]);
  };
  if (gwarp == 0)
    for (int i = 0; i < stages; ++i) {
      start(r0 + (int64_t)i * G, i);
      __syncwarp();
    }
  int p2 = 1;
  while (p2 < gw) p2 *= 2;
  const int lw = lane & (p2 - 1);
  const float2 other = gw > 1 && lw < gw ? s_cnt[lw] : make_float2(0.f, 0.f);
  uint64_t ga[NV][NP], be[NV][NP];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[VEC], b[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) a[e] = b[e] = 0.f;
    if (FULL || t0 + i * step < nvec) {
      load_params<VEC>(gamma, wbf16, (int64_t)(t0 + i * step) * VEC, 1.f, a);
      load_params<VEC>(beta, wbf16, (int64_t)(t0 + i * step) * VEC, 0.f, b);
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      ga[i][e] = f2pack(a[2 * e], a[2 * e + 1]);
      be[i][e] = f2pack(b[2 * e], b[2 * e + 1]);
    }
  }
  int it = 0, s = 0;
  for (int64_t r = r0; r < valid; r += G, ++it) {
    bool ok = poll_wait(&st.bar[s], (it / stages) & 1, SITE_ROWS);
    const bool live = st.row[s] >= 0;  // the same for all threads of the group
    const uint4* src = reinterpret_cast<const uint4*>(ring + (size_t)s * row_bytes) + t0;
    uint64_t f[NV][NP];
    uint64_t acc = 0;  // (0.f, 0.f)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (FULL || t0 + i * step < nvec) raw = src[i * step];
      vec_pairs<T>(raw, f[i]);
#pragma unroll
      for (int e = 0; e < NP; ++e) acc = fadd2(acc, f[i][e]);
    }
    // the warp's sum and its squares about the warp's own mean: the warps then combine in one
    // step without cancellation, sum (M2_w + n_w (mean_w - mean)^2)
    const float sum = warp_sum(pair_sum(acc));
    const float wm = sum * inv_cnt;
    const uint64_t nwm = f2pack(-wm, -wm);
    uint64_t q = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (FULL || t0 + i * step < nvec) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          f[i][e] = fadd2(f[i][e], nwm);
          q = ffma2(f[i][e], f[i][e], q);
        }
      }
    }
    float m2 = warp_sum(pair_sum(q)), mean = sum * inv_h;
    if (gw > 1) {
      if (lane == 0) s_red[it & 1][warp] = make_float2(sum, m2);
      ok = group_agree(ok, gw);
      // lane l takes warp l mod p2 (the next power of two): log2(p2) shuffles a sum, where a loop
      // over the warps is a chain of shared-memory reads
      const float2 v = lw < gw ? s_red[it & 1][lw] : make_float2(0.f, 0.f);
      mean = v.x;
      for (int o = p2 >> 1; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
      mean *= inv_h;
      const float d = fmaf(v.x, other.y, -mean);
      m2 = fmaf(other.x * d, d, v.y);
      for (int o = p2 >> 1; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    } else {
      ok = group_agree(ok, gw);
    }
    if (!ok) return;
    if (gwarp == 0) {  // every warp has read the row: refill its stage
      start(r + (int64_t)stages * G, s);
      __syncwarp();
    }
    if (++s == stages) s = 0;
    if (!live) continue;
    const float rstd = 1.f / sqrtf(m2 * inv_h + eps);
    if (leader) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
    const float off = (wm - mean) * rstd;
    const uint64_t rs = f2pack(rstd, rstd), of = f2pack(off, off);
    uint4* yr = reinterpret_cast<uint4*>(y + r * ldy) + t0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (FULL || t0 + i * step < nvec) {
#pragma unroll
        for (int e = 0; e < NP; ++e) f[i][e] = ffma2(ffma2(f[i][e], rs, of), ga[i][e], be[i][e]);
        yr[i * step] = pairs_vec<T>(f[i]);
      }
    }
  }
}

// Backward: x, dy and dres rows stream through a shared-memory ring -- the group's leader starts
// bulk copies ahead, a queue that does not depend on how many warps the registers leave room for
// -- and a stage is refilled after the next row's barrier, when every warp has left it.  gamma
// and the sums of dgamma and dbeta stay in registers over all the group's rows, x - mean and
// dy gamma between the two halves of a row.  At the end the CTA's groups are added in order in
// shared memory and the CTA's partial sums stored in ws [CTAs][2][h], which
// layernorm_wgrad_reduce adds in order (no atomics: the same bits every run on a device).
template <typename T, int NV, bool RES, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 320 ? 2 : 1)
    layernorm_bwd_ring_kernel(const T* dy, int64_t ldy, const T* x, int64_t ldx, RowMap map, int h, int gw, int stages,
                              const float* mean, const float* rstd, const void* gamma, int wbf16, const T* dres,
                              int64_t ldr, T* dx, int64_t ldd, float* ws) {
  constexpr int VEC = 16 / (int)sizeof(T), NP = VEC / 2, MATS = RES ? 3 : 2;
  constexpr bool HOLD = MAXT != 320;  // 96 registers leave no room: x and dy are read a second time
  extern __shared__ __align__(128) uint8_t s_rows[];
  __shared__ LnRing s_ring[8];
  __shared__ float2 s_red[2][32];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int groups = (blockDim.x >> 5) / gw, grp = warp / gw, gwarp = warp - grp * gw;
  const int nvec = h / VEC, step = gw * 32, t0 = gwarp * 32 + lane;
  const int valid = valid_rows(map);
  const int G = gridDim.x * groups, r0 = blockIdx.x * groups + grp;
  const uint32_t row_bytes = (uint32_t)h * sizeof(T);
  uint8_t* ring = s_rows + (size_t)grp * stages * MATS * row_bytes;
  LnRing& st = s_ring[grp];
  const bool leader = t0 == 0;
  if (leader) {
    for (int i = 0; i < stages; ++i) mbar_init(&st.bar[i], 1);
    fence_barrier_init();
  }
  __syncthreads();
  auto start = [&](int64_t r, int s) {  // first warp of the group: row r into stage s
    if (r >= valid) return;
    const int64_t row = sequence_row(map, (int)r);
    if (!elect_one()) return;
    if (!ln_claim(st, row, (int)r, s, MATS * row_bytes)) return;
    uint8_t* d = ring + (size_t)s * MATS * row_bytes;
    bulk_load_1d(d, x + row * ldx, row_bytes, &st.bar[s]);
    bulk_load_1d(d + row_bytes, dy + r * ldy, row_bytes, &st.bar[s]);
    if (RES) bulk_load_1d(d + 2 * row_bytes, dres + row * ldr, row_bytes, &st.bar[s]);
  };
  if (gwarp == 0)
    for (int i = 0; i < stages; ++i) {
      start(r0 + (int64_t)i * G, i);
      __syncwarp();
    }
  uint64_t ga[NV][NP], ag[NV][NP], ab[NV][NP];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) a[e] = 0.f;
    if (FULL || t0 + i * step < nvec) load_params<VEC>(gamma, wbf16, (int64_t)(t0 + i * step) * VEC, 1.f, a);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      ga[i][e] = f2pack(a[2 * e], a[2 * e + 1]);
      ag[i][e] = 0;
      ab[i][e] = 0;
    }
  }
  int p2 = 1;  // lane l adds warp l mod p2's sums
  while (p2 < gw) p2 *= 2;
  const int lw = lane & (p2 - 1);
  const float inv_h = 1.f / (float)h;
  float mu = 0.f, rs = 0.f;  // of the row to come
  if (r0 < valid) {
    mu = mean[r0];
    rs = rstd[r0];
  }
  int it = 0, s = 0;
  bool ok = true;
  for (int64_t r = r0; r < valid; r += G, ++it) {
    const float cr = rs;
    const uint64_t nm = f2pack(-mu, -mu), r2 = f2pack(rs, rs);
    if (r + G < valid) {
      mu = mean[r + G];
      rs = rstd[r + G];
    }
    ok = poll_wait(&st.bar[s], (it / stages) & 1, SITE_ROWS);
    const int64_t row = st.row[s];
    const uint8_t* d = ring + (size_t)s * MATS * row_bytes + t0 * 16;
    float s1 = 0.f, s2 = 0.f;
    uint64_t xc[HOLD ? NV : 1][NP], gy[HOLD ? NV : 1][NP];  // x - mean, dy gamma
    if (row >= 0) {
      uint64_t p1 = 0, p2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (FULL || t0 + i * step < nvec) {
          uint64_t df[NP], *xi = xc[HOLD ? i : 0], *gi = gy[HOLD ? i : 0];
          vec_pairs<T>(*reinterpret_cast<const uint4*>(d + i * step * 16), xi);
          vec_pairs<T>(*reinterpret_cast<const uint4*>(d + row_bytes + i * step * 16), df);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            xi[e] = fadd2(xi[e], nm);
            gi[e] = fmul2(df[e], ga[i][e]);
            const uint64_t n = fmul2(xi[e], r2);
            p1 = fadd2(p1, gi[e]);
            p2 = ffma2(gi[e], n, p2);
            ag[i][e] = ffma2(df[e], n, ag[i][e]);
            ab[i][e] = fadd2(ab[i][e], df[e]);
          }
        }
      }
      s1 = pair_sum(p1);
      s2 = pair_sum(p2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (gw > 1) {
      if (lane == 0) s_red[it & 1][warp] = make_float2(s1, s2);
      ok = group_agree(ok, gw);
      const float2 v = lw < gw ? s_red[it & 1][lw] : make_float2(0.f, 0.f);
      s1 = v.x;
      s2 = v.y;
      for (int o = p2 >> 1; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
    } else {
      ok = group_agree(ok, gw);
    }
    if (!ok) break;
    if (gwarp == 0 && it > 0 && stages > 1) {
      start(r + (int64_t)(stages - 1) * G, s ? s - 1 : stages - 1);
      __syncwarp();
    }
    if (row >= 0) {
      // dx = rstd g - rstd mean(g) - (x - mean) rstd^2 mean(g n)
      const float c1 = -s1 * inv_h * cr, c2 = -s2 * inv_h * cr * cr;
      const uint64_t c1p = f2pack(c1, c1), c2p = f2pack(c2, c2);
      uint4* dst = reinterpret_cast<uint4*>(dx + row * ldd) + t0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (FULL || t0 + i * step < nvec) {
          uint64_t o[NP], ef[NP], *xi = xc[HOLD ? i : 0], *gi = gy[HOLD ? i : 0];
          if (!HOLD) {
            vec_pairs<T>(*reinterpret_cast<const uint4*>(d + i * step * 16), xi);
            vec_pairs<T>(*reinterpret_cast<const uint4*>(d + row_bytes + i * step * 16), gi);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
              xi[e] = fadd2(xi[e], nm);
              gi[e] = fmul2(gi[e], ga[i][e]);
            }
          }
          if (RES) vec_pairs<T>(*reinterpret_cast<const uint4*>(d + 2 * row_bytes + i * step * 16), ef);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            o[e] = ffma2(gi[e], r2, ffma2(xi[e], c2p, c1p));
            if (RES) o[e] = fadd2(o[e], ef[e]);
          }
          dst[i * step] = pairs_vec<T>(o);
        }
      }
    }
    if (stages == 1) {  // rows so wide that the next one waits until all warps have left this one
      ok = group_agree(ok, gw);
      if (!ok) break;
      if (gwarp == 0) {
        start(r + G, 0);
        __syncwarp();
      }
    }
    if (++s == stages) s = 0;
  }
  if (!ws) return;
  float* out = ws + (int64_t)blockIdx.x * 2 * h;
  float* mine = out;
  if (groups > 1) {  // the ring is idle once every group has left its loop
    __syncthreads();
    mine = reinterpret_cast<float*>(s_rows) + (int64_t)grp * 2 * h;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(t0 + i * step) * VEC;
    if (FULL || t0 + i * step < nvec) {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        *reinterpret_cast<uint64_t*>(mine + c + 2 * e) = ag[i][e];
        *reinterpret_cast<uint64_t*>(mine + h + c + 2 * e) = ab[i][e];
      }
    }
  }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * h; c += blockDim.x) {
    float a = 0.f;
    for (int g = 0; g < groups; ++g) a += reinterpret_cast<const float*>(s_rows)[(int64_t)g * 2 * h + c];
    out[c] = a;
  }
}

// ------------------------------------------------------------------ unaligned rows
// Element-wise loads, for rows that are not whole 16-byte vectors (odd widths, odd pitches,
// unaligned bases): a thread holds NV elements, 32 gw apart.  Forward and backward keep gamma
// (and beta, or the sums) in registers over the rows of a persistent group and load the next
// row's elements before this row is reduced.
template <typename T, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 128 ? 5 : (MAXT <= 256 ? 2 : 1))
    layernorm_fwd_kernel(const T* x, int64_t ldx, RowMap map, int h, int gw, const void* gamma, const void* beta,
                         int wbf16, float eps, T* y, int64_t ldy, float* mean_out, float* rstd_out) {
  __shared__ float2 s_red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (blockDim.x >> 5) / gw, grp = warp / gw, gwarp = warp - grp * gw;
  const int step = gw * 32, t0 = gwarp * 32 + lane;
  const int valid = valid_rows(map);
  const int G = gridDim.x * groups;
  const int64_t r0 = blockIdx.x * groups + grp;
  int p2 = 1;  // lane l combines warp l mod p2's sums
  while (p2 < gw) p2 *= 2;
  const int lw = lane & (p2 - 1);
  auto held = [&](int w) {  // elements of a row that warp w of the group holds
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) n += max(0, min(32, h - (w * 32 + i * step)));
    return (float)n;
  };
  const float inv_h = 1.f / (float)h, cnt = held(gwarp), inv_cnt = cnt > 0.f ? 1.f / cnt : 0.f;
  const float ocnt = lw < gw ? held(lw) : 0.f, inv_ocnt = ocnt > 0.f ? 1.f / ocnt : 0.f;
  float ga[NV], be[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ga[i] = be[i] = 0.f;
    if (t0 + i * step < h) {
      load_params<1>(gamma, wbf16, t0 + i * step, 1.f, &ga[i]);
      load_params<1>(beta, wbf16, t0 + i * step, 0.f, &be[i]);
    }
  }
  RowVec<T, 1> nxt[NV];
  auto fetch = [&](int64_t r) {
    if (r >= valid) return false;
    const int64_t row = sequence_row(map, (int)r);
    if (row < 0) {
      if (t0 == 0) record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
      return false;
    }
    const T* p = x + row * ldx + t0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t0 + i * step < h) nxt[i].load(p + i * step);
    return true;
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) nxt[i].zero();
  bool live = fetch(r0);
  int par = 0;
  for (int64_t r = r0; r < valid; r += G) {
    float f[NV], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nxt[i].get(&f[i]);
      if (t0 + i * step < h) sum += f[i];
    }
    const bool now = live;  // the same for the whole group
    live = fetch(r + G);
    if (!now) continue;
    sum = warp_sum(sum);
    const float wm = sum * inv_cnt;
    float m2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f[i] -= wm;
      if (t0 + i * step < h) m2 = fmaf(f[i], f[i], m2);
    }
    m2 = warp_sum(m2);
    float mean = sum * inv_h;
    if (gw > 1) {
      if (lane == 0) s_red[par][warp] = make_float2(sum, m2);
      __syncthreads();  // the CTA is the row group
      const float2 v = lw < gw ? s_red[par][lw] : make_float2(0.f, 0.f);
      mean = v.x;
      for (int o = p2 >> 1; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
      mean *= inv_h;
      const float d = fmaf(v.x, inv_ocnt, -mean);
      m2 = fmaf(ocnt * d, d, v.y);
      for (int o = p2 >> 1; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
      par ^= 1;
    }
    const float rstd = 1.f / sqrtf(m2 * inv_h + eps);
    if (t0 == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
    const float off = (wm - mean) * rstd;
    T* yr = y + r * ldy + t0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t0 + i * step < h) {
        const float o = fmaf(fmaf(f[i], rstd, off), ga[i], be[i]);
        RowVec<T, 1>::store(yr + i * step, &o);
      }
  }
}

// Backward: as the ring kernel, the next row's elements loaded before this row's two sums.
template <typename T, int NV>
struct BwdRow {
  RowVec<T, 1> x[NV], dy[NV], res[NV];
  float mean, rstd;
  int64_t row;
};

template <typename T, int NV, bool RES, int MAXT>
__global__ void __launch_bounds__(MAXT)
    layernorm_bwd_kernel(const T* dy, int64_t ldy, const T* x, int64_t ldx, RowMap map, int h, int gw,
                         const float* mean, const float* rstd, const void* gamma, int wbf16, const T* dres,
                         int64_t ldr, T* dx, int64_t ldd, float* ws) {
  extern __shared__ float s_dyn[];
  __shared__ float s_red[2][2][32];  // [parity][sum][warp of the CTA]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (blockDim.x >> 5) / gw, grp = warp / gw, gwarp = warp - grp * gw;
  const int step = gw * 32, t0 = gwarp * 32 + lane;
  const int valid = valid_rows(map);
  const int G = gridDim.x * groups;
  float ga[NV], ag[NV], ab[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ga[i] = ag[i] = ab[i] = 0.f;
    if (t0 + i * step < h) load_params<1>(gamma, wbf16, t0 + i * step, 1.f, &ga[i]);
  }
  auto fetch = [&](BwdRow<T, NV>& b, int64_t r) {  // 64 bits: a row count near 2^31 plus a step
    b.row = -1;
    if (r >= valid) return;
    b.row = sequence_row(map, (int)r);
    if (b.row < 0) {
      if (t0 == 0) record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
      return;
    }
    b.mean = mean[r];
    b.rstd = rstd[r];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t0 + i * step;
      b.x[i].zero();
      b.dy[i].zero();
      if (c < h) {
        b.x[i].load(x + b.row * ldx + c);
        b.dy[i].load(dy + r * ldy + c);
        if (RES) b.res[i].load(dres + b.row * ldr + c);
      }
    }
  };
  int p2 = 1;  // lane l adds warp l mod p2's sums
  while (p2 < gw) p2 *= 2;
  const int lw = lane & (p2 - 1);
  const float inv_h = 1.f / (float)h;
  BwdRow<T, NV> cur, nxt;
  const int64_t r0 = blockIdx.x * groups + grp;
  fetch(cur, r0);
  int par = 0;
  for (int64_t r = r0; r < valid; r += G) {
    fetch(nxt, r + G);
    if (cur.row >= 0) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf, df;
        cur.x[i].get(&xf);
        cur.dy[i].get(&df);
        if (t0 + i * step < h) {
          const float n = (xf - cur.mean) * cur.rstd, g = df * ga[i];
          s1 += g;
          s2 = fmaf(g, n, s2);
          ag[i] = fmaf(df, n, ag[i]);
          ab[i] += df;
        }
      }
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      if (gw > 1) {
        if (lane == 0) {
          s_red[par][0][warp] = s1;
          s_red[par][1][warp] = s2;
        }
        __syncthreads();
        s1 = lw < gw ? s_red[par][0][lw] : 0.f;
        s2 = lw < gw ? s_red[par][1][lw] : 0.f;
        for (int o = p2 >> 1; o > 0; o >>= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        par ^= 1;
      }
      const float c1 = s1 * inv_h, c2 = s2 * inv_h;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (t0 + i * step < h) {
          float xf, df, rf, o;
          cur.x[i].get(&xf);
          cur.dy[i].get(&df);
          if (RES) cur.res[i].get(&rf);
          const float n = (xf - cur.mean) * cur.rstd;
          o = cur.rstd * (fmaf(df, ga[i], -c1) - n * c2);
          if (RES) o += rf;
          RowVec<T, 1>::store(dx + cur.row * ldd + t0 + i * step, &o);
        }
      }
    }
    cur = nxt;
  }
  if (!ws) return;
  // sums of the CTA: its one group's, or [group][2][h] in shared memory added in group order
  float* out = ws + (int64_t)blockIdx.x * 2 * h;
  float* mine = groups == 1 ? out : s_dyn + (int64_t)grp * 2 * h;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t0 + i * step;
    if (c < h) {
      mine[c] = ag[i];
      mine[h + c] = ab[i];
    }
  }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * h; c += blockDim.x) {
    float a = 0.f;
    for (int g = 0; g < groups; ++g) a += s_dyn[(int64_t)g * 2 * h + c];
    out[c] = a;
  }
}

// out[c] (+)= sum over the parts of part[p][c] for 2 h columns (dgamma, then dbeta): 32 columns
// per CTA, 16 interleaved runs of parts added in run order.
__global__ void __launch_bounds__(512) layernorm_wgrad_reduce_kernel(const float* __restrict__ part, int parts, int h,
                                                                     float* dgamma, float* dbeta, int accumulate) {
  __shared__ float s[16][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < 2 * h) {
#pragma unroll 8
    for (int p = run; p < parts; p += 16) a += part[(int64_t)p * 2 * h + c];
  }
  s[run][lane] = a;
  __syncthreads();
  if (run == 0 && c < 2 * h) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a += s[i][lane];
    float* o = c < h ? dgamma : dbeta;
    if (o) {
      o += c < h ? c : c - h;
      *o = accumulate ? *o + a : a;
    }
  }
}

constexpr int LN_MAX_H = 16384;

// Shape of a launch: row groups of gw warps, nv vectors (elements when vec == 1) a thread, and
// for the ring its stages and bytes.
struct LnShape {
  int vec, nv, gw, groups, ctas, stages;
  size_t smem;
};
// Ring bytes of a CTA with per_sm of them on an SM: the SM's shared memory less what a CTA takes
// besides.  (Without that allowance one CTA of eight did not fit and ran as a second wave: 768
// wide, 104960 rows of bf16 backward 200 us against 138.)
static int ln_room(int per_sm) {
  const int room = 228 * 1024 / per_sm - 3 * 1024;
  return room < 216 * 1024 ? room : 216 * 1024;
}
// Aligned forward.  bf16 is bound by instruction issue next to memory: 32 columns a thread spread
// the per-row steps (barrier, shuffles, copies) over more of them, at 16 warps an SM (with eight rows
// in the ring, 26240 x
// 4096: 78 us against 92 with 16 columns and 24 warps; 5120 wide: 94 against 122).  fp32 moves
// twice the bytes a column: 16 columns, two CTAs an SM for wide rows (16384 x 4096: 83 us
// against 93 with 32 columns, 101 with three CTAs).  Fewer columns when a warp holds the row.
static LnShape ln_fwd_shape(int rows, int h, int es) {
  LnShape s{};
  s.vec = 16 / es;
  const int nvec = h / s.vec, most = 4;  // 32 columns of bf16, 16 of fp32
  s.nv = 1;
  while (s.nv < most && nvec > 32 * s.nv) s.nv *= 2;
  s.gw = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.groups = s.gw > 1 ? 1 : 4;
  const int warps = s.gw * s.groups, per_stage = h * es * s.groups;
  int per_sm = warps <= 4 ? (es == 2 ? 16 : 24) / warps : (es == 2 && warps <= 5 ? 3 : (warps <= (es == 2 ? 8 : 10) ? 2 : 1));
  s.stages = ln_room(per_sm) / per_stage;  // 3 rows of 64 KB at the least
  s.stages = s.stages > LN_FWD_STAGES ? LN_FWD_STAGES : s.stages;
  s.smem = (size_t)s.stages * per_stage;
  const int want = (rows - 1) / s.groups + 1, cap = per_sm * sm_count();
  s.ctas = want < cap ? want : cap;
  return s;
}
// Aligned backward: 16 columns a thread (gamma and the two sums stay in registers), eight warps a
// CTA, fewer columns when a warp holds the row.  Rows too wide for two stages (fp32 above
// 13824 columns, 9216 with dres) take one, without overlap in the CTA.  Unaligned rows: one element a
// thread up to 512 threads.
static LnShape ln_bwd_shape(int rows, int h, int es, bool aligned, int mats) {
  LnShape s{};
  aligned = aligned && h * es * mats <= ln_room(1);
  s.vec = aligned ? 16 / es : 1;
  const int nvec = h / s.vec, most = aligned ? 16 / s.vec : 16;
  s.nv = 1;
  while (s.nv < most && nvec > (aligned ? 32 : 512) * s.nv) s.nv *= 2;
  s.gw = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.groups = s.gw > 1 ? 1 : 8;
  const int warps = s.gw * s.groups, per_stage = h * es * mats * s.groups;
  int per_sm = !aligned ? 2 : (warps > 10 ? 1 : (warps < 8 ? 16 / warps : 2));
  if (aligned) {
    while (per_sm > 1 && ln_room(per_sm) / per_stage < 3) --per_sm;  // one stage ahead while one drains
    s.stages = ln_room(per_sm) / per_stage;
    s.stages = s.stages > LN_BWD_STAGES ? LN_BWD_STAGES : s.stages;
    s.smem = (size_t)s.stages * per_stage;
  }
  const size_t sums = s.groups > 1 ? (size_t)s.groups * 2 * h * sizeof(float) : 0;
  if (s.smem < sums) s.smem = sums;
  const int want = (rows - 1) / s.groups + 1, cap = per_sm * sm_count();
  s.ctas = want < cap ? want : cap;
  return s;
}

struct LnFwdCall {
  const void* x;
  int64_t ldx;
  RowMap map;
  int h;
  const void *gamma, *beta;
  int wbf16;
  float eps;
  void* y;
  int64_t ldy;
  float *mean, *rstd;
};
template <typename T, int NV, int MAXT>
static cudaError_t ln_fwd_ring(const LnShape& s, const LnFwdCall& c, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    if ((e = allow_smem((const void*)kernel)) != cudaSuccess) return;
    kernel<<<s.ctas, s.gw * s.groups * 32, s.smem, st>>>((const T*)c.x, c.ldx, c.map, c.h, s.gw, s.stages, c.gamma,
                                                         c.beta, c.wbf16, c.eps, (T*)c.y, c.ldy, c.mean, c.rstd);
  };
  c.h == s.gw * 32 * s.nv * s.vec ? go(layernorm_fwd_ring_kernel<T, NV, true, MAXT>)
                                  : go(layernorm_fwd_ring_kernel<T, NV, false, MAXT>);
  return e;
}
template <typename T, int NV, int MAXT>
static cudaError_t ln_fwd_one(const LnFwdCall& c, int gw, cudaStream_t st) {
  const int groups = gw == 1 ? 4 : 1, warps = gw * groups;
  const int per_sm = warps <= 4 ? 20 / warps : (warps <= 8 ? 2 : 1);
  const int want = (c.map.rows - 1) / groups + 1, cap = per_sm * sm_count();
  layernorm_fwd_kernel<T, NV, MAXT><<<want < cap ? want : cap, warps * 32, 0, st>>>(
      (const T*)c.x, c.ldx, c.map, c.h, gw, c.gamma, c.beta, c.wbf16, c.eps, (T*)c.y, c.ldy, c.mean, c.rstd);
  return cudaSuccess;
}
template <typename T>
static cudaError_t ln_fwd(bool aligned, const LnFwdCall& c, cudaStream_t st) {
  if (!aligned) {
    const int gw = c.h <= 512 ? 1 : (c.h + 511) / 512;  // 16 elements a thread
    if (c.h <= 128) return ln_fwd_one<T, 4, 128>(c, 1, st);
    if (gw <= 4) return ln_fwd_one<T, 16, 128>(c, gw, st);
    if (gw <= 8) return ln_fwd_one<T, 16, 256>(c, gw, st);
    if (gw <= 16) return ln_fwd_one<T, 16, 512>(c, gw, st);
    return ln_fwd_one<T, 16, 1024>(c, gw, st);
  }
  const LnShape s = ln_fwd_shape(c.map.rows, c.h, sizeof(T));
  if (s.nv == 1) return ln_fwd_ring<T, 1, 128>(s, c, st);  // a warp holds the row: four rows a CTA
  if (s.nv == 2) return ln_fwd_ring<T, 2, 128>(s, c, st);
  const int threads = s.gw * s.groups * 32;
  if (threads <= 128) return ln_fwd_ring<T, 4, 128>(s, c, st);
  if constexpr (sizeof(T) == 2) {
    if (threads <= 160) return ln_fwd_ring<T, 4, 160>(s, c, st);
    if (threads <= 256) return ln_fwd_ring<T, 4, 256>(s, c, st);
    return ln_fwd_ring<T, 4, 512>(s, c, st);  // 16384 columns: 16 warps
  } else {
    if (threads <= 320) return ln_fwd_ring<T, 4, 320>(s, c, st);
    if (threads <= 512) return ln_fwd_ring<T, 4, 512>(s, c, st);
    return ln_fwd_ring<T, 4, 1024>(s, c, st);
  }
}

struct LnBwdCall {
  const void* dy;
  int64_t ldy;
  const void* x;
  int64_t ldx;
  RowMap map;
  int h;
  const float *mean, *rstd;
  const void* gamma;
  int wbf16;
  const void* dres;
  int64_t ldr;
  void* dx;
  int64_t ldd;
  float* part;
};
template <typename T, int NV, int MAXT>
static cudaError_t ln_bwd_ring(const LnShape& s, const LnBwdCall& c, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) {
    if ((e = allow_smem((const void*)kernel)) != cudaSuccess) return;
    kernel<<<s.ctas, s.gw * s.groups * 32, s.smem, st>>>((const T*)c.dy, c.ldy, (const T*)c.x, c.ldx, c.map, c.h, s.gw,
                                                         s.stages, c.mean, c.rstd, c.gamma, c.wbf16, (const T*)c.dres,
                                                         c.ldr, (T*)c.dx, c.ldd, c.part);
  };
  if (c.h == s.gw * 32 * s.nv * s.vec)
    c.dres ? go(layernorm_bwd_ring_kernel<T, NV, true, true, MAXT>) : go(layernorm_bwd_ring_kernel<T, NV, false, true, MAXT>);
  else
    c.dres ? go(layernorm_bwd_ring_kernel<T, NV, true, false, MAXT>)
           : go(layernorm_bwd_ring_kernel<T, NV, false, false, MAXT>);
  return e;
}
template <typename T, int NV>
static cudaError_t ln_bwd_one(const LnShape& s, const LnBwdCall& c, cudaStream_t st) {
  const int threads = s.gw * s.groups * 32;
  auto go = [&](auto kernel) {
    kernel<<<s.ctas, threads, s.smem, st>>>((const T*)c.dy, c.ldy, (const T*)c.x, c.ldx, c.map, c.h, s.gw, c.mean,
                                            c.rstd, c.gamma, c.wbf16, (const T*)c.dres, c.ldr, (T*)c.dx, c.ldd, c.part);
  };
  if constexpr (NV == 16) {  // fewer elements a thread stay within 512 threads
    if (threads > 512) {
      c.dres ? go(layernorm_bwd_kernel<T, NV, true, 1024>) : go(layernorm_bwd_kernel<T, NV, false, 1024>);
      return cudaSuccess;
    }
  }
  c.dres ? go(layernorm_bwd_kernel<T, NV, true, 512>) : go(layernorm_bwd_kernel<T, NV, false, 512>);
  return cudaSuccess;
}
template <typename T>
static cudaError_t ln_bwd(const LnShape& s, const LnBwdCall& c, cudaStream_t st) {
  if (s.vec == 1) {
    if (s.nv == 1) return ln_bwd_one<T, 1>(s, c, st);
    if (s.nv == 2) return ln_bwd_one<T, 2>(s, c, st);
    if (s.nv == 4) return ln_bwd_one<T, 4>(s, c, st);
    if (s.nv == 8) return ln_bwd_one<T, 8>(s, c, st);
    return ln_bwd_one<T, 16>(s, c, st);
  }
  constexpr int MOST = sizeof(T) == 2 ? 2 : 4;
  if (s.nv < MOST) {  // a warp holds the row: eight rows a CTA
    if (s.nv == 1) return ln_bwd_ring<T, 1, 256>(s, c, st);
    if constexpr (MOST == 4) return ln_bwd_ring<T, 2, 256>(s, c, st);
  }
  const int threads = s.gw * s.groups * 32;
  if (threads <= 256) return ln_bwd_ring<T, MOST, 256>(s, c, st);
  if (threads <= 320) return ln_bwd_ring<T, MOST, 320>(s, c, st);
  if (threads <= 512) return ln_bwd_ring<T, MOST, 512>(s, c, st);
  return ln_bwd_ring<T, MOST, 1024>(s, c, st);
}

// shared argument checks of the row operators
static jenga_status check_rows(const char* who, int S, int h, const int32_t* idx, const int32_t* n_kept, int blk,
                               int rows, jenga_dtype dt) {
  JENGA_CHECK_ARG(rows >= 0 && h >= 1 && S >= 0 && blk >= 1, "%s: bad sizes rows=%d S=%d h=%d blk=%d", who, rows, S, h,
                  blk);
  JENGA_CHECK_ARG(dt == JENGA_F32 || dt == JENGA_BF16, "%s: dtype", who);
  JENGA_CHECK_ARG(!(idx || n_kept) || rows % blk == 0, "%s: rows (%d) must be whole blocks of %d", who, rows, blk);
  if (idx)
    JENGA_CHECK_ARG(S % blk == 0 && rows <= S, "%s: S=%d must be whole blocks and hold the rows (%d)", who, S, rows);
  else
    JENGA_CHECK_ARG(rows <= S, "%s: rows=%d of S=%d", who, rows, S);
  return JENGA_OK;
}

}  // namespace jenga

using namespace jenga;

extern "C" jenga_status jenga_layernorm_fwd(const void* x, int64_t ldx, int S, int h, const int32_t* idx,
                                            const int32_t* n_kept, int blk, int rows, const void* gamma,
                                            const void* beta, jenga_dtype wdt, float eps, jenga_dtype dt, void* y,
                                            int64_t ldy, float* mean, float* rstd, jenga_stream_t stream) {
  JENGA_TRY(check_rows("jenga_layernorm_fwd", S, h, idx, n_kept, blk, rows, dt));
  JENGA_CHECK_ARG(wdt == JENGA_F32 || wdt == JENGA_BF16, "jenga_layernorm_fwd: parameter dtype");
  JENGA_CHECK_ARG(ldx >= h && ldy >= h, "jenga_layernorm_fwd: row pitch smaller than h");
  JENGA_CHECK_ARG(eps > 0.f && eps < INFINITY, "jenga_layernorm_fwd: eps must be positive and finite");
  if (h > LN_MAX_H) return fail(JENGA_EUNSUPPORTED, "jenga_layernorm_fwd: h=%d above %d", h, LN_MAX_H);
  if (rows == 0) return JENGA_OK;
  JENGA_CHECK_ARG(x && y, "jenga_layernorm_fwd: null pointer");
  const int es = dt == JENGA_F32 ? 4 : 2;
  const int wes = wdt == JENGA_F32 ? 4 : 2;
  JENGA_CHECK_ARG(outputs_apart({mat_span(y, rows, h, ldy, es), vec_span(mean, rows, 4), vec_span(rstd, rows, 4)},
                                {mat_span(x, idx ? S : rows, h, ldx, es, !idx), vec_span(gamma, h, wes),
                                 vec_span(beta, h, wes), vec_span(idx, rows / blk, 4), vec_span(n_kept, 1, 4)}),
                  "jenga_layernorm_fwd: an output overlaps an input or another output (allowed only for y = x, the same "
                  "matrix, without a block list)");
  const int v = 16 / es;
  const bool aligned =
      h % v == 0 && ldx % v == 0 && ldy % v == 0 && is16(x) && is16(y) && is16(gamma) && is16(beta);
  const LnFwdCall c{x, ldx, RowMap{idx, n_kept, blk, S / blk, rows}, h, gamma, beta, wdt == JENGA_BF16, eps, y, ldy, mean,
                    rstd};
  cudaStream_t st = (cudaStream_t)stream;
  const int _ps = prof_begin("layernorm_fwd", st);
  JENGA_CUDA_TRY(dt == JENGA_BF16 ? ln_fwd<bf16>(aligned, c, st) : ln_fwd<float>(aligned, c, st));
  prof_end(_ps, st);
  JENGA_LAUNCH_CHECK();
  return JENGA_OK;
}

extern "C" size_t jenga_layernorm_bwd_workspace_bytes(int rows, int h) {
  if (rows < 1 || h < 1 || h > LN_MAX_H) return 0;
  int ctas = 0;  // the most of the types, alignments and residual forms
  for (int es = 2; es <= 4; es += 2)
    for (int mats = 2; mats <= 3; ++mats)
      for (int aligned = 0; aligned <= (h % (16 / es) == 0); ++aligned) {
        const int n = ln_bwd_shape(rows, h, es, aligned, mats).ctas;
        ctas = n > ctas ? n : ctas;
      }
  return (size_t)ctas * 2 * h * sizeof(float) + 256;
}

extern "C" jenga_status jenga_layernorm_bwd(const void* dy, int64_t ldy, const void* x, int64_t ldx, int S, int h,
                                            const int32_t* idx, const int32_t* n_kept, int blk, int rows,
                                            const float* mean, const float* rstd, const void* gamma, jenga_dtype wdt,
                                            const void* dres, int64_t ldr, jenga_dtype dt, void* dx, int64_t ldd,
                                            float* dgamma, float* dbeta, int accumulate, void* ws, size_t ws_bytes,
                                            jenga_stream_t stream) {
  JENGA_TRY(check_rows("jenga_layernorm_bwd", S, h, idx, n_kept, blk, rows, dt));
  JENGA_CHECK_ARG(wdt == JENGA_F32 || wdt == JENGA_BF16, "jenga_layernorm_bwd: parameter dtype");
  JENGA_CHECK_ARG(ldx >= h && ldy >= h && ldd >= h && (!dres || ldr >= h),
                  "jenga_layernorm_bwd: row pitch smaller than h");
  if (h > LN_MAX_H) return fail(JENGA_EUNSUPPORTED, "jenga_layernorm_bwd: h=%d above %d", h, LN_MAX_H);
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // empty sums
    if (!accumulate && dgamma) JENGA_CUDA_TRY(cudaMemsetAsync(dgamma, 0, (size_t)h * sizeof(float), st));
    if (!accumulate && dbeta) JENGA_CUDA_TRY(cudaMemsetAsync(dbeta, 0, (size_t)h * sizeof(float), st));
    return JENGA_OK;
  }
  JENGA_CHECK_ARG(dy && x && mean && rstd && dx, "jenga_layernorm_bwd: null pointer");
  const int es = dt == JENGA_F32 ? 4 : 2;
  const int64_t xrows = idx ? S : rows;
  const auto apart = [&](size_t ws_used) {  // dx as a row operand is compact or, through a list, the sequence
    return outputs_apart(
        {mat_span(dx, xrows, h, ldd, es), vec_span(dgamma, h, 4), vec_span(dbeta, h, 4), vec_span(ws, ws_used, 1)},
        {mat_span(x, xrows, h, ldx, es, true), mat_span(dy, rows, h, ldy, es, !idx),
         mat_span(dres, xrows, h, ldr, es, true), vec_span(mean, rows, 4), vec_span(rstd, rows, 4),
         vec_span(gamma, h, wdt == JENGA_F32 ? 4 : 2), vec_span(idx, rows / blk, 4), vec_span(n_kept, 1, 4)});
  };
  const char* met = "jenga_layernorm_bwd: an output or the workspace overlaps an input or another output (allowed only "
                    "for dx as the same matrix as dres, x or, without a block list, dy)";
  JENGA_CHECK_ARG(apart(0), "%s", met);
  const bool wgrad = dgamma || dbeta;
  const size_t need = jenga_layernorm_bwd_workspace_bytes(rows, h);
  if (wgrad && (!ws || ws_bytes < need))
    return fail(JENGA_EWORKSPACE, "jenga_layernorm_bwd: workspace %zu < %zu", ws ? ws_bytes : (size_t)0, need);
  JENGA_CHECK_ARG(!wgrad || apart(need), "%s", met);
  float* part = wgrad ? (float*)(((uintptr_t)ws + 255) & ~uintptr_t(255)) : nullptr;
  const int v = 16 / es;
  const bool aligned = h % v == 0 && ldx % v == 0 && ldy % v == 0 && ldd % v == 0 && (!dres || ldr % v == 0) &&
                       is16(x) && is16(dy) && is16(dx) && is16(dres) && is16(gamma);
  const LnShape s = ln_bwd_shape(rows, h, es, aligned, dres ? 3 : 2);
  const LnBwdCall c{dy,  ldy,  x,   ldx, RowMap{idx, n_kept, blk, S / blk, rows}, h, mean, rstd, gamma, wdt == JENGA_BF16,
                    dres, ldr, dx, ldd, part};
  int _ps = prof_begin("layernorm_bwd", st);
  JENGA_CUDA_TRY(dt == JENGA_BF16 ? ln_bwd<bf16>(s, c, st) : ln_bwd<float>(s, c, st));
  prof_end(_ps, st);
  JENGA_LAUNCH_CHECK();
  if (wgrad) {
    _ps = prof_begin("layernorm_wgrad_reduce", st);
    layernorm_wgrad_reduce_kernel<<<(2 * h + 31) / 32, 512, 0, st>>>(part, s.ctas, h, dgamma, dbeta, accumulate);
    prof_end(_ps, st);
    JENGA_LAUNCH_CHECK();
  }
  return JENGA_OK;
}
