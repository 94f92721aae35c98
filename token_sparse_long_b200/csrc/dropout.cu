// Dropout whose mask is a function of (seed, offset, sequence position, column): nothing is
// stored, and the backward pass is the same call on the gradient.
//
// Generator: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC'11).  Counter words (column / 8, sequence position, offset low, offset high),
// key words (seed low, seed high); the four output words are eight 16-bit numbers u for the
// eight columns of the group, low half first.  An element is kept when u >= T,
// T = floor(p 2^16 + 1/2), and multiplied by 2^16 / (2^16 - T): the drop rate is p to within
// 2^-17 and the scale matches the rate used, so the expectation is exact.  16 bits an element
// instead of 32 halve the generator's work.
//
// The position is the token's row in the full sequence (through the block list), so a token's
// mask depends neither on which other blocks are kept nor on how the rows are cut into segments.
//
//   y = keep ? x * scale : 0, + residual      (a dropped infinity or NaN leaves 0)
// One fp32 multiply and add per element, rounded once.
#include "rows.cuh"

namespace jenga {

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
    c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

struct DropoutArgs {
  RowMap map;
  int cols;
  int64_t row0;         // position of compact row 0 (no block list)
  uint32_t threshold;   // keep when the 16-bit number is >= threshold
  float scale;
  uint32_t seed[2], offset[2];
  FastDiv per_row;      // column groups per row
  uint32_t items;       // rows of this launch * column groups
  int r0;               // first compact row of this launch
};

constexpr int DROP_UNROLL = 4;

// One item = eight columns of a row; DROP_UNROLL items a thread, 256 apart (coalesced).
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y,
                                                      int64_t ldy, DropoutArgs p) {
  constexpr int PER = VEC ? 16 / (int)sizeof(T) : 1, NV = 8 / PER;
  const int valid = valid_rows(p.map);
  const uint64_t first = (uint64_t)blockIdx.x * (256 * DROP_UNROLL) + threadIdx.x;
  RowVec<T, PER> xv[DROP_UNROLL][NV], rv[DROP_UNROLL][NV];
  int rr[DROP_UNROLL];
  uint32_t gg[DROP_UNROLL];
#pragma unroll
  for (int u = 0; u < DROP_UNROLL; ++u) {
    const uint64_t w = first + u * 256;
    rr[u] = -1;
    if (w >= p.items) continue;
    const uint32_t r = fast_div((uint32_t)w, p.per_row);
    gg[u] = (uint32_t)w - r * p.per_row.d;
    if (p.r0 + (int)r >= valid) continue;
    rr[u] = p.r0 + (int)r;
    const int c = (int)gg[u] * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (c + i * PER < p.cols) {
        xv[u][i].load(x + (int64_t)rr[u] * ldx + c + i * PER);
        if (RES) rv[u][i].load(res + (int64_t)rr[u] * ldr + c + i * PER);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < DROP_UNROLL; ++u) {
    if (rr[u] < 0) continue;
    int64_t pos = p.map.idx ? sequence_row(p.map, rr[u]) : p.row0 + rr[u];
    if (pos < 0 || pos > 0x7fffffff) {
      record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)rr[u]);
      continue;
    }
    const uint4 bits = philox4x32_10(make_uint4(gg[u], (uint32_t)pos, p.offset[0], p.offset[1]), p.seed[0], p.seed[1]);
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
    const int c = (int)gg[u] * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (c + i * PER < p.cols) {
        float f[PER], g[PER];
        xv[u][i].get(f);
        if (RES) rv[u][i].get(g);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int k = i * PER + e;
          const uint32_t n = (k & 1) ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu;
          f[e] = n >= p.threshold ? f[e] * p.scale : 0.f;
          if (RES) f[e] += g[e];
        }
        RowVec<T, PER>::store(y + (int64_t)rr[u] * ldy + c + i * PER, f);
      }
    }
  }
}

template <typename T>
static void dropout_launch(bool vec, const void* x, int64_t ldx, const void* res, int64_t ldr, void* y, int64_t ldy,
                           const DropoutArgs& p, cudaStream_t st) {
  const unsigned grid = (unsigned)(((uint64_t)p.items + 256 * DROP_UNROLL - 1) / (256 * DROP_UNROLL));
  auto go = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>((const T*)x, ldx, (const T*)res, ldr, (T*)y, ldy, p);
  };
  if (vec)
    res ? go(dropout_kernel<T, true, true>) : go(dropout_kernel<T, true, false>);
  else
    res ? go(dropout_kernel<T, false, true>) : go(dropout_kernel<T, false, false>);
}

}  // namespace jenga

using namespace jenga;

extern "C" jenga_status jenga_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, int rows, int cols,
                                      const int32_t* idx, const int32_t* n_kept, int blk, int64_t row0, double p,
                                      uint64_t seed, uint64_t offset, jenga_dtype dt, void* y, int64_t ldy,
                                      jenga_stream_t stream) {
  JENGA_CHECK_ARG(rows >= 0 && cols >= 1 && blk >= 1, "jenga_dropout: bad sizes rows=%d cols=%d blk=%d", rows, cols,
                  blk);
  JENGA_CHECK_ARG(dt == JENGA_F32 || dt == JENGA_BF16, "jenga_dropout: dtype");
  JENGA_CHECK_ARG(p >= 0.0 && p <= 1.0, "jenga_dropout: p=%g outside [0, 1]", p);
  JENGA_CHECK_ARG(ldx >= cols && ldy >= cols && (!residual || ldr >= cols),
                  "jenga_dropout: row pitch smaller than the row");
  JENGA_CHECK_ARG(!(idx || n_kept) || rows % blk == 0, "jenga_dropout: rows (%d) must be whole blocks of %d", rows, blk);
  JENGA_CHECK_ARG(row0 >= 0 && row0 + rows <= (1ll << 31), "jenga_dropout: positions must stay below 2^31");
  JENGA_CHECK_ARG(!idx || row0 == 0, "jenga_dropout: row0 has no meaning with a block list");
  if (rows == 0) return JENGA_OK;
  JENGA_CHECK_ARG(x && y, "jenga_dropout: null pointer");
  const int es = dt == JENGA_F32 ? 4 : 2;
  const uint64_t ny = span_bytes(rows, cols, ldy, es);
  JENGA_CHECK_ARG(alias_ok(y, ldy, ny, x, ldx, span_bytes(rows, cols, ldx, es), true) &&
                      alias_ok(y, ldy, ny, residual, ldr, span_bytes(rows, cols, ldr, es), true),
                  "jenga_dropout: y overlaps an input other than as the same matrix");
  const int v = 16 / es;
  const bool vec = cols % v == 0 && ldx % v == 0 && ldy % v == 0 && (!residual || ldr % v == 0) && is16(x) && is16(y) &&
                   is16(residual);
  DropoutArgs a;
  a.map = RowMap{idx, n_kept, blk, 0x7fffffff / blk, rows};
  a.cols = cols;
  a.row0 = row0;
  a.threshold = (uint32_t)floor(p * 65536.0 + 0.5);
  a.scale = a.threshold >= 65536u ? 0.f : (float)(65536.0 / (65536.0 - (double)a.threshold));
  a.seed[0] = (uint32_t)seed;
  a.seed[1] = (uint32_t)(seed >> 32);
  a.offset[0] = (uint32_t)offset;
  a.offset[1] = (uint32_t)(offset >> 32);
  const int groups = (cols + 7) / 8;
  a.per_row = make_fastdiv((uint32_t)groups);
  cudaStream_t st = (cudaStream_t)stream;
  // 32-bit item numbers: very large matrices go out in several launches of whole rows
  const int most = (int)((1ll << 30) / groups) > 0 ? (int)((1ll << 30) / groups) : 1;
  for (int r0 = 0; r0 < rows; r0 += most) {
    const int n = rows - r0 < most ? rows - r0 : most;
    a.r0 = r0;
    a.items = (uint32_t)n * (uint32_t)groups;
    const int _ps = prof_begin("dropout", st);
    if (dt == JENGA_BF16)
      dropout_launch<bf16>(vec, x, ldx, residual, ldr, y, ldy, a, st);
    else
      dropout_launch<float>(vec, x, ldx, residual, ldr, y, ldy, a, st);
    prof_end(_ps, st);
    JENGA_LAUNCH_CHECK();
    if (rows - r0 <= most) break;  // r0 + most may pass 2^31
  }
  return JENGA_OK;
}
