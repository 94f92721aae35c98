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

// ------------------------------------------------------------------ forward
// One row group of `gw` warps per row, NV vectors of VEC elements per thread.  gw == 1: four
// rows per CTA, one per warp, no block-wide step.  Wider rows: the CTA is the row group.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__((VEC > 1 ? NV <= 4 : NV <= 16) ? 1024 : 128) layernorm_fwd_kernel(const T* x, int64_t ldx, RowMap map, int h, int gw,
                                                             const void* gamma, const void* beta, int wbf16,
                                                             float eps, T* y, int64_t ldy, float* mean_out,
                                                             float* rstd_out) {
  __shared__ float s_red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gwarp = gw == 1 ? 0 : warp;
  const int r = gw == 1 ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  if (r >= valid_rows(map)) return;  // uniform over the row group
  const int64_t row = sequence_row(map, r);
  if (row < 0) {
    if (lane == 0 && gwarp == 0) record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
    return;
  }
  const T* xr = x + row * ldx;
  const int nvec = h / VEC, step = gw * 32, t0 = gwarp * 32 + lane;
  RowVec<T, VEC> v[NV];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i].zero();
    if (t0 + i * step < nvec) v[i].load(xr + (int64_t)(t0 + i * step) * VEC);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[VEC];
    v[i].get(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += f[e];
  }
  const float inv_h = 1.f / (float)h;
  const float mean = group_sum(s, s_red[0], gwarp, gw, 1) * inv_h;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (t0 + i * step < nvec) {
      float f[VEC];
      v[i].get(f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = f[e] - mean;
        q = fmaf(d, d, q);
      }
    }
  }
  const float var = group_sum(q, s_red[1], gwarp, gw, 1) * inv_h;
  const float rstd = 1.f / sqrtf(var + eps);
  if (t0 == 0) {
    if (mean_out) mean_out[r] = mean;
    if (rstd_out) rstd_out[r] = rstd;
  }
  T* yr = y + (int64_t)r * ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(t0 + i * step) * VEC;
    if (t0 + i * step < nvec) {
      float f[VEC], ga[VEC], be[VEC];
      v[i].get(f);
      load_params<VEC>(gamma, wbf16, c, 1.f, ga);
      load_params<VEC>(beta, wbf16, c, 0.f, be);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mean) * rstd, ga[e], be[e]);
      RowVec<T, VEC>::store(yr + c, f);
    }
  }
}

// ------------------------------------------------------------------ backward
// Persistent row groups of `gw` warps (blockDim / (32 gw) groups per CTA): group g of G takes
// rows g, g + G, ...; a thread owns the same NV * VEC columns of every row, so the sums of
// dgamma and dbeta stay in its registers until the group's rows are done.  The CTA's groups
// are then added in order in shared memory and the CTA's partial sums stored in ws
// [CTAs][2][h]; layernorm_wgrad_reduce adds the CTAs in order (no atomics: the same bits every
// run on the same device).  The next row's dy, x (and dres) are loaded before this row's two
// sums, so the loads cover the reduction.
template <typename T, int VEC, int NV>
struct BwdRow {
  RowVec<T, VEC> x[NV], dy[NV], res[NV];
  float mean, rstd;
  int64_t row;
};

template <typename T, int VEC, int NV, bool RES, int MAXT>
__global__ void __launch_bounds__(MAXT)
    layernorm_bwd_kernel(const T* dy, int64_t ldy, const T* x, int64_t ldx, RowMap map, int h, int gw,
                         const float* mean, const float* rstd, const void* gamma, int wbf16, const T* dres,
                         int64_t ldr, T* dx, int64_t ldd, float* ws) {
  extern __shared__ float s_dyn[];
  __shared__ float s_red[2][2][32];  // [parity][sum][warp of the CTA]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (blockDim.x >> 5) / gw, grp = warp / gw, gwarp = warp - grp * gw;
  const int nvec = h / VEC, step = gw * 32, t0 = gwarp * 32 + lane;
  const int valid = valid_rows(map);
  const int G = gridDim.x * groups;
  float ga[NV][VEC], ag[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      ga[i][e] = 0.f;
      ag[i][e] = 0.f;
      ab[i][e] = 0.f;
    }
    if (t0 + i * step < nvec) load_params<VEC>(gamma, wbf16, (int64_t)(t0 + i * step) * VEC, 1.f, ga[i]);
  }
  auto fetch = [&](BwdRow<T, VEC, NV>& b, int r) {
    b.row = -1;
    if (r >= valid) return;
    b.row = sequence_row(map, r);
    if (b.row < 0) {
      if (t0 == 0) record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
      return;
    }
    b.mean = mean[r];
    b.rstd = rstd[r];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(t0 + i * step) * VEC;
      b.x[i].zero();
      b.dy[i].zero();
      if (t0 + i * step < nvec) {
        b.x[i].load(x + b.row * ldx + c);
        b.dy[i].load(dy + (int64_t)r * ldy + c);
        if (RES) b.res[i].load(dres + b.row * ldr + c);
      }
    }
  };
  const float inv_h = 1.f / (float)h;
  BwdRow<T, VEC, NV> cur, nxt;
  const int r0 = blockIdx.x * groups + grp;
  fetch(cur, r0);
  int par = 0;
  for (int r = r0; r < valid; r += G) {
    fetch(nxt, r + G);
    if (cur.row >= 0) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[VEC], df[VEC];
        cur.x[i].get(xf);
        cur.dy[i].get(df);
        if (t0 + i * step < nvec) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float n = (xf[e] - cur.mean) * cur.rstd, g = df[e] * ga[i][e];
            s1 += g;
            s2 = fmaf(g, n, s2);
            ag[i][e] = fmaf(df[e], n, ag[i][e]);
            ab[i][e] += df[e];
          }
        }
      }
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      if (gw > 1) {
        if (lane == 0) {
          s_red[par][0][warp] = s1;
          s_red[par][1][warp] = s2;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(gw * 32) : "memory");
        s1 = 0.f;
        s2 = 0.f;
        for (int i = 0; i < gw; ++i) {
          s1 += s_red[par][0][grp * gw + i];
          s2 += s_red[par][1][grp * gw + i];
        }
        par ^= 1;
      }
      const float c1 = s1 * inv_h, c2 = s2 * inv_h;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(t0 + i * step) * VEC;
        if (t0 + i * step < nvec) {
          float xf[VEC], df[VEC], rf[VEC], o[VEC];
          cur.x[i].get(xf);
          cur.dy[i].get(df);
          if (RES) cur.res[i].get(rf);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float n = (xf[e] - cur.mean) * cur.rstd;
            o[e] = cur.rstd * (fmaf(df[e], ga[i][e], -c1) - n * c2);
            if (RES) o[e] += rf[e];
          }
          RowVec<T, VEC>::store(dx + cur.row * ldd + c, o);
        }
      }
    }
    cur = nxt;
  }
  if (!ws) return;
  float* out = ws + (int64_t)blockIdx.x * 2 * h;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(t0 + i * step) * VEC;
      if (t0 + i * step < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          out[c + e] = ag[i][e];
          out[h + c + e] = ab[i][e];
        }
      }
    }
    return;
  }
  // several groups: [group][2][h] in shared memory, added in group order
  float* mine = s_dyn + (int64_t)grp * 2 * h;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(t0 + i * step) * VEC;
    if (t0 + i * step < nvec) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        mine[c + e] = ag[i][e];
        mine[h + c + e] = ab[i][e];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * h; c += blockDim.x) {
    float a = 0.f;
    for (int g = 0; g < groups; ++g) a += s_dyn[(int64_t)g * 2 * h + c];
    out[c] = a;
  }
}

// out[c] (+)= sum over the parts of part[p][c] for 2 h columns (dgamma, then dbeta): 32 columns
// per CTA, eight interleaved runs of parts added in run order.
__global__ void __launch_bounds__(256) layernorm_wgrad_reduce_kernel(const float* __restrict__ part, int parts, int h,
                                                                     float* dgamma, float* dbeta, int accumulate) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < 2 * h)
    for (int p = run; p < parts; p += 8) a += part[(int64_t)p * 2 * h + c];
  s[run][lane] = a;
  __syncthreads();
  if (run == 0 && c < 2 * h) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a += s[i][lane];
    float* o = c < h ? dgamma : dbeta;
    if (o) {
      o += c < h ? c : c - h;
      *o = accumulate ? *o + a : a;
    }
  }
}

constexpr int LN_MAX_H = 16384;

// CTAs of the backward: enough row groups for two CTAs an SM, at most one group per row.
struct LnBwdShape {
  int vec, nv, gw, groups, ctas;
};
static LnBwdShape ln_bwd_shape(int rows, int h, int vec) {
  LnBwdShape s;
  s.vec = vec;
  const int nvec = h / vec;
  // columns a thread owns: as few as one vector while the row group stays within 512 threads
  s.nv = 1;
  const int most = vec == 8 ? 2 : (vec == 4 ? 4 : 16);
  while (s.nv < most && nvec > s.nv * 512) s.nv *= 2;
  s.gw = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  s.groups = s.gw >= 8 ? 1 : 8 / s.gw;
  const int want = (rows + s.groups - 1) / s.groups;
  const int cap = 2 * sm_count();
  s.ctas = want < 1 ? 1 : (want < cap ? want : cap);
  return s;
}

template <typename T, int VEC, int NV>
static void ln_fwd_launch(const void* x, int64_t ldx, const RowMap& map, int h, const void* gamma, const void* beta,
                          int wbf16, float eps, void* y, int64_t ldy, float* mean, float* rstd, cudaStream_t st) {
  const int nvec = h / VEC, gw = (nvec + 32 * NV - 1) / (32 * NV);
  const int threads = gw == 1 ? 128 : gw * 32;
  const int grid = gw == 1 ? (map.rows + 3) / 4 : map.rows;
  layernorm_fwd_kernel<T, VEC, NV><<<grid, threads, 0, st>>>((const T*)x, ldx, map, h, gw, gamma, beta, wbf16, eps,
                                                             (T*)y, ldy, mean, rstd);
}

template <typename T, int VEC, int NV>
static void ln_bwd_launch(const LnBwdShape& s, const void* dy, int64_t ldy, const void* x, int64_t ldx,
                          const RowMap& map, int h, const float* mean, const float* rstd, const void* gamma,
                          int wbf16, const void* dres, int64_t ldr, void* dx, int64_t ldd, float* ws,
                          cudaStream_t st) {
  const int threads = s.gw * s.groups * 32;
  const size_t smem = s.groups > 1 && ws ? (size_t)s.groups * 2 * h * sizeof(float) : 0;
  auto go = [&](auto kernel) {
    kernel<<<s.ctas, threads, smem, st>>>((const T*)dy, ldy, (const T*)x, ldx, map, h, s.gw, mean, rstd, gamma, wbf16,
                                          (const T*)dres, ldr, (T*)dx, ldd, ws);
  };
  if (threads <= 512)
    dres ? go(layernorm_bwd_kernel<T, VEC, NV, true, 512>) : go(layernorm_bwd_kernel<T, VEC, NV, false, 512>);
  else
    dres ? go(layernorm_bwd_kernel<T, VEC, NV, true, 1024>) : go(layernorm_bwd_kernel<T, VEC, NV, false, 1024>);
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

#define JENGA_LN_DISPATCH(FN, NVV, ...)                                   \
  do {                                                                    \
    if (dt == JENGA_BF16 && vec == 8) {                                   \
      FN##_VEC(bf16, 8, NVV, __VA_ARGS__);                                \
    } else if (dt == JENGA_F32 && vec == 4) {                             \
      FN##_VEC(float, 4, NVV, __VA_ARGS__);                               \
    } else if (dt == JENGA_BF16) {                                        \
      FN##_ONE(bf16, NVV, __VA_ARGS__);                                   \
    } else {                                                              \
      FN##_ONE(float, NVV, __VA_ARGS__);                                  \
    }                                                                     \
  } while (0)

#define LN_FWD_VEC(T, V, n, ...)                                    \
  (n) == 1   ? ln_fwd_launch<T, V, 1>(__VA_ARGS__)                  \
  : (n) == 2 ? ln_fwd_launch<T, V, 2>(__VA_ARGS__)                  \
  : (n) == 4 ? ln_fwd_launch<T, V, 4>(__VA_ARGS__)                  \
  : (n) == 8 ? ln_fwd_launch<T, V, 8>(__VA_ARGS__)                  \
             : ln_fwd_launch<T, V, 16>(__VA_ARGS__)
#define LN_FWD_ONE(T, n, ...)                                       \
  (n) == 2    ? ln_fwd_launch<T, 1, 2>(__VA_ARGS__)                 \
  : (n) == 8  ? ln_fwd_launch<T, 1, 8>(__VA_ARGS__)                 \
  : (n) == 16 ? ln_fwd_launch<T, 1, 16>(__VA_ARGS__)                \
              : ln_fwd_launch<T, 1, 32>(__VA_ARGS__)
#define LN_BWD_VEC(T, V, n, ...)                                    \
  (n) == 1   ? ln_bwd_launch<T, V, 1>(__VA_ARGS__)                  \
  : (n) == 2 ? ln_bwd_launch<T, V, 2>(__VA_ARGS__)                  \
             : ln_bwd_launch<T, V, 4>(__VA_ARGS__)
#define LN_BWD_ONE(T, n, ...)                                       \
  (n) == 1   ? ln_bwd_launch<T, 1, 1>(__VA_ARGS__)                  \
  : (n) == 2 ? ln_bwd_launch<T, 1, 2>(__VA_ARGS__)                  \
  : (n) == 4 ? ln_bwd_launch<T, 1, 4>(__VA_ARGS__)                  \
  : (n) == 8 ? ln_bwd_launch<T, 1, 8>(__VA_ARGS__)                  \
             : ln_bwd_launch<T, 1, 16>(__VA_ARGS__)

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
  JENGA_CHECK_ARG(alias_ok(y, ldy, span_bytes(rows, h, ldy, es), x, ldx, span_bytes(S, h, ldx, es), !idx),
                  "jenga_layernorm_fwd: y overlaps x (allowed only as the same matrix, without a block list)");
  const int v = 16 / es;
  const int vec = h % v == 0 && ldx % v == 0 && ldy % v == 0 && is16(x) && is16(y) && is16(gamma) && is16(beta) ? v : 1;
  const RowMap map{idx, n_kept, blk, S / blk, rows};
  cudaStream_t st = (cudaStream_t)stream;
  const int wb = wdt == JENGA_BF16;
  // a warp per row while the row fits its registers, else a CTA of as few warps as hold it
  const int nvec = h / vec;
  int nv;
  if (vec > 1) {
    nv = 1;
    while (nv < 16 && nvec > 32 * nv) nv *= 2;
    if (nvec > 32 * 16) nv = 4;
  } else {
    nv = nvec <= 64 ? 2 : (nvec <= 256 ? 8 : (nvec <= 1024 ? 32 : 16));
  }
  const int _ps = prof_begin("layernorm_fwd", st);
  JENGA_LN_DISPATCH(LN_FWD, nv, x, ldx, map, h, gamma, beta, wb, eps, y, ldy, mean, rstd, st);
  prof_end(_ps, st);
  JENGA_LAUNCH_CHECK();
  return JENGA_OK;
}

extern "C" size_t jenga_layernorm_bwd_workspace_bytes(int rows, int h) {
  if (rows < 1 || h < 1 || h > LN_MAX_H) return 0;
  const int cap = 2 * sm_count();
  return (size_t)(rows < cap ? rows : cap) * 2 * h * sizeof(float) + 256;
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
  const uint64_t nd = span_bytes(idx ? S : rows, h, ldd, es);
  JENGA_CHECK_ARG(alias_ok(dx, ldd, nd, x, ldx, span_bytes(idx ? S : rows, h, ldx, es), true) &&
                      alias_ok(dx, ldd, nd, dy, ldy, span_bytes(rows, h, ldy, es), !idx) &&
                      alias_ok(dx, ldd, nd, dres, ldr, span_bytes(idx ? S : rows, h, ldr, es), true),
                  "jenga_layernorm_bwd: dx overlaps an input other than as the same matrix");
  const bool wgrad = dgamma || dbeta;
  const size_t need = jenga_layernorm_bwd_workspace_bytes(rows, h);
  if (wgrad && (!ws || ws_bytes < need))
    return fail(JENGA_EWORKSPACE, "jenga_layernorm_bwd: workspace %zu < %zu", ws ? ws_bytes : (size_t)0, need);
  float* part = wgrad ? (float*)(((uintptr_t)ws + 255) & ~uintptr_t(255)) : nullptr;
  const int v = 16 / es;
  const int vec = h % v == 0 && ldx % v == 0 && ldy % v == 0 && ldd % v == 0 && (!dres || ldr % v == 0) && is16(x) &&
                          is16(dy) && is16(dx) && is16(dres) && is16(gamma)
                      ? v
                      : 1;
  const RowMap map{idx, n_kept, blk, S / blk, rows};
  const int wb = wdt == JENGA_BF16;
  const LnBwdShape s = ln_bwd_shape(rows, h, vec);
  int _ps = prof_begin("layernorm_bwd", st);
  JENGA_LN_DISPATCH(LN_BWD, s.nv, s, dy, ldy, x, ldx, map, h, mean, rstd, gamma, wb, dres, ldr, dx, ldd, part, st);
  prof_end(_ps, st);
  JENGA_LAUNCH_CHECK();
  if (wgrad) {
    _ps = prof_begin("layernorm_wgrad_reduce", st);
    layernorm_wgrad_reduce_kernel<<<(2 * h + 31) / 32, 256, 0, st>>>(part, s.ctas, h, dgamma, dbeta, accumulate);
    prof_end(_ps, st);
    JENGA_LAUNCH_CHECK();
  }
  return JENGA_OK;
}
