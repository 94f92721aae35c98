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
  int cols, groups;     // columns, and their groups of eight
  int64_t row0;         // position of compact row 0 (no block list)
  uint32_t threshold;   // T << 16 (0 < T < 2^16)
  float scale;
  uint32_t seed[2], offset[2];
  FastDiv blk;          // rows per block
  int tx;               // threads along a row (a power of two), 256 / tx rows at a time
};

enum DropMode : int { DROP_RANDOM = 0, DROP_NONE = 1, DROP_ALL = 2 };  // T = 0 and T = 2^16 need no bits

constexpr int DROP_ROWS = 4;

// A thread takes one group of eight columns of DROP_ROWS rows (loads first); row and position are
// worked out once per row and thread, so that what is left per group is the generator's ten
// rounds (40 instructions), a comparison, a multiply-add and a select per element -- a flat index
// with its divisions per group made the kernel compute-bound (26240 x 4096 bf16 with the
// residual through a block list: 138 us; now 104 us, 6.2 TB/s; without the residual 88 us, where
// the generator bounds it).  Unaligned rows (VEC false) are read and written lane by lane, the
// bits of a warp's 256 columns passing through shared memory: the words of a group lie there
// in column order.
template <typename T, bool VEC, bool RES, int MODE>
__global__ void __launch_bounds__(256, !VEC ? 1 : (sizeof(T) == 2 ? (RES ? 4 : 5) : (RES ? 2 : 3))) dropout_kernel(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y,
                                                      int64_t ldy, DropoutArgs p) {
  constexpr int PER = VEC ? 16 / (int)sizeof(T) : 1, NV = 8 / PER;
  __shared__ uint4 s_bits[VEC ? 1 : 256];
  const int valid = valid_rows(p.map);
  const int ty = 256 / p.tx, g = blockIdx.x * p.tx + (threadIdx.x & (p.tx - 1));
  const int lane = threadIdx.x & 31;
  // column of the thread's vector i: eight neighbours, or (VEC false, tx >= 32) every 32nd
  const int c = VEC ? g * 8 : (g - lane) * 8 + lane;
  constexpr int CSTEP = VEC ? PER : 32;
  if ((VEC ? g : g - lane) >= p.groups) return;  // VEC false: the whole warp
  for (int64_t r0 = (int64_t)blockIdx.y * ty * DROP_ROWS + threadIdx.x / p.tx; r0 < valid;
       r0 += (int64_t)gridDim.y * ty * DROP_ROWS) {
    RowVec<T, PER> xv[DROP_ROWS][NV], rv[DROP_ROWS][NV];
    // position = base + row up to the block's last row; the next block is looked up when reached
    int base = (int)p.row0, next = 0x7fffffff;
    bool good = true;
    auto locate = [&](int r) {
      const int i = (int)fast_div((uint32_t)r, p.blk), b = __ldg(p.map.idx + i);
      good = b >= 0 && b < p.map.nb && (i == 0 || __ldg(p.map.idx + i - 1) < b);
      base = good ? (b - i) * p.map.blk : 0;
      next = (int)min((int64_t)(i + 1) * p.map.blk, (int64_t)0x7fffffff);
    };
    if (p.map.idx) locate((int)r0);
#pragma unroll
    for (int u = 0; u < DROP_ROWS; ++u) {
      const int64_t r = r0 + u * ty;
      if (r >= valid) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c + i * CSTEP < p.cols) {
          if (MODE != DROP_ALL) xv[u][i].load(x + r * ldx + c + i * CSTEP);
          if (RES) rv[u][i].load(res + r * ldr + c + i * CSTEP);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < DROP_ROWS; ++u) {
      const int64_t r = r0 + u * ty;  // one row per warp where VEC is false
      if (r >= valid) continue;
      if (r >= next) locate((int)r);
      if (!good) {
        record_device_error(JENGA_EINTERNAL, SITE_INDEX_RANGE, (unsigned)r);
        continue;
      }
      uint32_t w[4] = {0, 0, 0, 0};
      if (MODE == DROP_RANDOM) {
        const uint4 bits =
            philox4x32_10(make_uint4((uint32_t)g, (uint32_t)(base + (int)r), p.offset[0], p.offset[1]), p.seed[0], p.seed[1]);
        w[0] = bits.x;
        w[1] = bits.y;
        w[2] = bits.z;
        w[3] = bits.w;
        if (!VEC) {
          __syncwarp();  // the row before is done
          s_bits[threadIdx.x] = bits;
          __syncwarp();
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c + i * CSTEP < p.cols) {
          float f[PER], q[PER];
          if (MODE != DROP_ALL) xv[u][i].get(f);
          if (RES) rv[u][i].get(q);
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const int k = i * PER + e;
            // the 16-bit number against T: in the high half the low half does not matter
            uint32_t n = (k & 1) ? w[k >> 1] : w[k >> 1] << 16;
            if (!VEC && MODE == DROP_RANDOM)
              n = (uint32_t)reinterpret_cast<const uint16_t*>(s_bits + (threadIdx.x - lane))[i * 32 + lane] << 16;
            const bool keep = MODE == DROP_NONE || (MODE == DROP_RANDOM && n >= p.threshold);
            if (MODE == DROP_ALL)
              f[e] = RES ? q[e] : 0.f;
            else
              f[e] = RES ? (keep ? fmaf(f[e], p.scale, q[e]) : q[e]) : (keep ? f[e] * p.scale : 0.f);
          }
          RowVec<T, PER>::store(y + r * ldy + c + i * CSTEP, f);
        }
      }
    }
  }
}

template <typename T, int MODE>
static void dropout_launch(bool vec, dim3 grid, const void* x, int64_t ldx, const void* res, int64_t ldr, void* y,
                           int64_t ldy, const DropoutArgs& p, cudaStream_t st) {
  auto go = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>((const T*)x, ldx, (const T*)res, ldr, (T*)y, ldy, p);
  };
  if (vec)
    res ? go(dropout_kernel<T, true, true, MODE>) : go(dropout_kernel<T, true, false, MODE>);
  else
    res ? go(dropout_kernel<T, false, true, MODE>) : go(dropout_kernel<T, false, false, MODE>);
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
  JENGA_CHECK_ARG(outputs_apart({mat_span(y, rows, cols, ldy, es)},
                                {mat_span(x, rows, cols, ldx, es, true), mat_span(residual, rows, cols, ldr, es, true),
                                 vec_span(idx, rows / blk, 4), vec_span(n_kept, 1, 4)}),
                  "jenga_dropout: y overlaps an input other than as the same matrix");
  const int v = 16 / es;
  const bool vec = cols % v == 0 && ldx % v == 0 && ldy % v == 0 && (!residual || ldr % v == 0) && is16(x) && is16(y) &&
                   is16(residual);
  const uint32_t T = (uint32_t)floor(p * 65536.0 + 0.5);
  DropoutArgs a;
  a.map = RowMap{idx, n_kept, blk, 0x7fffffff / blk, rows};
  a.cols = cols;
  a.groups = (cols + 7) / 8;
  a.row0 = row0;
  a.threshold = T << 16;
  a.scale = T >= 65536u ? 0.f : (float)(65536.0 / (65536.0 - (double)T));
  a.seed[0] = (uint32_t)seed;
  a.seed[1] = (uint32_t)(seed >> 32);
  a.offset[0] = (uint32_t)offset;
  a.offset[1] = (uint32_t)(offset >> 32);
  a.blk = make_fastdiv((uint32_t)blk);
  a.tx = 256;
  while (a.tx > (vec ? 1 : 32) && a.tx / 2 >= a.groups) a.tx /= 2;
  const int strips = (a.groups + a.tx - 1) / a.tx, ty = 256 / a.tx;
  // one step of DROP_ROWS rows a thread, or a loop beyond the grid's limit
  const int64_t want = ((int64_t)rows + (int64_t)ty * DROP_ROWS - 1) / ((int64_t)ty * DROP_ROWS);
  const dim3 grid(strips, (unsigned)(want < 65535 ? want : 65535));
  cudaStream_t st = (cudaStream_t)stream;
  const int _ps = prof_begin("dropout", st);
  const bool f32 = dt == JENGA_F32;
  if (T == 0)
    f32 ? dropout_launch<float, DROP_NONE>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st)
        : dropout_launch<bf16, DROP_NONE>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st);
  else if (T >= 65536u)
    f32 ? dropout_launch<float, DROP_ALL>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st)
        : dropout_launch<bf16, DROP_ALL>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st);
  else
    f32 ? dropout_launch<float, DROP_RANDOM>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st)
        : dropout_launch<bf16, DROP_RANDOM>(vec, grid, x, ldx, residual, ldr, y, ldy, a, st);
  prof_end(_ps, st);
  JENGA_LAUNCH_CHECK();
  return JENGA_OK;
}
