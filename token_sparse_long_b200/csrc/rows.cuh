// Shared pieces of the row-wise operators (layer norm, dropout, the linear layer's
// element-wise passes): the retained-row map and 16-byte row vectors.
#pragma once

#include <atomic>
#include <initializer_list>

#include "common.cuh"

namespace jenga {

// Rows of an operator call.  Compact row r (0 <= r < rows) is sequence row r without a block
// list and idx[r / blk] * blk + r % blk with one.  n_kept (device, nullable) counts the valid
// blocks: rows at and past *n_kept * blk are neither read nor written.
struct RowMap {
  const int32_t* idx;
  const int32_t* n_kept;
  int blk, nb, rows;
};

// Valid rows of the call; an n_kept outside [0, rows / blk] is recorded and nothing is done.
__device__ __forceinline__ int valid_rows(const RowMap& m) {
  if (!m.n_kept) return m.rows;
  const int nk = __ldg(m.n_kept);
  if (nk < 0 || (int64_t)nk * m.blk > m.rows) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_device_error(JENGA_EINTERNAL, SITE_NKEPT_RANGE, (unsigned)nk);
    return 0;
  }
  return nk * m.blk;
}

// Sequence row of compact row r, or -1 for a list entry that is out of range or does not
// ascend (a block listed twice would make two rows write one place).
__device__ __forceinline__ int64_t sequence_row(const RowMap& m, int r) {
  if (!m.idx) return r;
  const int i = r / m.blk;
  const int b = __ldg(m.idx + i);
  if (b < 0 || b >= m.nb || (i > 0 && __ldg(m.idx + i - 1) >= b)) return -1;
  return (int64_t)b * m.blk + (r - i * m.blk);
}

// VEC consecutive elements of a row as loaded: one 16-byte vector (VEC = 16 / sizeof(T)), or
// one element (VEC = 1) for rows that are not 16-byte aligned.
template <typename T, int VEC>
struct RowVec;
template <>
struct RowVec<bf16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(bf16* p, const float* f) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
  }
};
template <>
struct RowVec<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = r.x;
    f[1] = r.y;
    f[2] = r.z;
    f[3] = r.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct RowVec<bf16, 1> {
  bf16 r;
  __device__ __forceinline__ void load(const bf16* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = __float2bfloat16_rn(0.f); }
  __device__ __forceinline__ void get(float* f) const { f[0] = __bfloat162float(r); }
  static __device__ __forceinline__ void store(bf16* p, const float* f) { *p = __float2bfloat16_rn(f[0]); }
};
template <>
struct RowVec<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = 0.f; }
  __device__ __forceinline__ void get(float* f) const { f[0] = r; }
  static __device__ __forceinline__ void store(float* p, const float* f) { *p = f[0]; }
};

// fp32 pairs of one 16-byte vector
template <typename T>
__device__ __forceinline__ void vec_pairs(const uint4& r, uint64_t* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    f[0] = f2pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
    f[1] = f2pack(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}
__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  f2unpack(v, a, b);
  return a + b;
}

// N consecutive parameters (N = 1, 4 or 8) of type F32 or BF16; `fill` without a tensor.
// N > 1 needs a 16-byte aligned tensor and a column that is a multiple of N.
template <int N>
__device__ __forceinline__ void load_params(const void* p, int wbf16, int64_t col, float fill, float* f) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fill;
  } else if (wbf16) {
    const bf16* q = reinterpret_cast<const bf16*>(p) + col;
    if constexpr (N == 1) {
      f[0] = __bfloat162float(*q);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + i));
        f[i] = __uint_as_float(w.x << 16);
        f[i + 1] = __uint_as_float(w.x & 0xffff0000u);
        f[i + 2] = __uint_as_float(w.y << 16);
        f[i + 3] = __uint_as_float(w.y & 0xffff0000u);
      }
    }
  } else {
    const float* q = reinterpret_cast<const float*>(p) + col;
    if constexpr (N == 1) {
      f[0] = *q;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(q + i));
        f[i] = w.x;
        f[i + 1] = w.y;
        f[i + 2] = w.z;
        f[i + 3] = w.w;
      }
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ bool aligned16_dev(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Bounded wait like mbar_wait, reading the timer and the budget only every 256 polls (each poll
// itself suspends for a hardware-defined time): those reads would sit on the critical path.
__device__ __forceinline__ bool poll_wait(uint64_t* bar, uint32_t phase, unsigned site) {
  if (mbar_try_wait(bar, phase)) return true;
  unsigned long long t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (mbar_try_wait(bar, phase)) return true;
    const unsigned long long t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > g_wait_budget_ns) {
      record_device_error(JENGA_ETIMEOUT, site, phase);
      return false;
    }
  }
}

// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// ------------------------------------------------------------------ host checks
// Memory that a call reads or writes: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Span {
  const void* p;
  int64_t rows, width, pitch;
  bool may_be_out0 = false;  // an input that the call's first output may be (same matrix): each element
                             // is read before it is written, by one thread
};
inline Span mat_span(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, bool may_be_out0 = false) {
  return Span{p, rows, cols * es, ld * es, may_be_out0};
}
inline Span vec_span(const void* p, int64_t n, int es) { return Span{p, 1, n * es, n * es}; }
// Do two spans share no byte?  Either one ends before the other begins, or they are columns side by
// side of rows of the same pitch.
inline bool spans_apart(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return true;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  const uint64_t na = (uint64_t)(a.rows - 1) * a.pitch + a.width, nb = (uint64_t)(b.rows - 1) * b.pitch + b.width;
  if (x + na <= y || y + nb <= x) return true;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  if (b.rows > 1 && b.pitch != pitch) return false;
  const int64_t off = y >= x ? (int64_t)((y - x) % pitch) : (int64_t)((pitch - (x - y) % pitch) % pitch);
  return off >= a.width && off + b.width <= pitch;  // b's columns within a's gaps
}
// No output meets an input or another output, but that the first one may be an input that says so.
inline bool outputs_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  const Span* o0 = outs.begin();
  for (const Span* o = o0; o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (!(o == o0 && i.may_be_out0 && o->p == i.p && o->pitch == i.pitch) && !spans_apart(*o, i)) return false;
    for (const Span* q = o0; q != o; ++q)
      if (!spans_apart(*o, *q)) return false;
  }
  return true;
}
// Allow a kernel `most` bytes of dynamic shared memory on the current device (set once per kernel,
// always with the same value, and device: the call costs as much as a tenth of a short launch).
inline cudaError_t allow_smem(const void* kernel, int most = 222 * 1024) {
  static std::atomic<const void*> seen[16][256];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 16)
    for (auto& slot : seen[dev]) {
      const void* k = slot.load(std::memory_order_acquire);
      if (k == kernel) return cudaSuccess;
      if (!k) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        const void* none = nullptr;
        if (e == cudaSuccess) slot.compare_exchange_strong(none, kernel);  // losing a race only sets it again later
        return e;
      }
    }
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

inline bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace jenga
