// What the row calls share (gfx950): element types, pieces of rows in registers, reductions of a wave and of
// a workgroup, int8 rows, 64-bit functions, and the host's checks of rows in memory.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/moe_route.h"
#include "moe_device.hpp"

namespace moe {

int hip_fail(hipError_t e, const char* what);   // moe_route.hip: keeps the text for moe_last_error

// ------------------------------------------------------------------ element types -----------

struct bf16_t {
  uint16_t v;
};
struct f16_t {
  uint16_t v;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16_t x) { return __builtin_bit_cast(float, (uint32_t)x.v << 16); }
__device__ __forceinline__ float to_f(f16_t x) { return h2f(x.v); }

template <typename T>
__device__ __forceinline__ T from_f(float f);
template <>
__device__ __forceinline__ float from_f<float>(float f) { return f; }
template <>
__device__ __forceinline__ bf16_t from_f<bf16_t>(float f) {   // round to nearest even, NaN kept
  return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <>
__device__ __forceinline__ f16_t from_f<f16_t>(float f) { return f16_t{(uint16_t)f2h(f)}; }

template <typename F>
auto with_type(int dtype, F f) {
  switch (dtype) {
    case MOE_BF16: return f(bf16_t{});
    case MOE_F16: return f(f16_t{});
    default: return f(float{});
  }
}

__host__ __device__ constexpr int type_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
inline bool type_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

__device__ __forceinline__ float load_f(const void* p, int dtype, int64_t i) {
  return dtype == MOE_F32 ? ((const float*)p)[i]
         : dtype == MOE_BF16 ? to_f(((const bf16_t*)p)[i]) : to_f(((const f16_t*)p)[i]);
}

// ------------------------------------------------------------------ rows --------------------
//
// moe_add_rmsnorm and moe_swiglu_i8 give a row to one workgroup, which reads it once and keeps it in
// registers, eight neighbouring values a thread (16-byte accesses for 16-bit types) and C such pieces.

constexpr int kPiece = 8;

template <typename T>
__device__ __forceinline__ void load_raw(const T* p, int i, int n, T (&v)[kPiece]) {
  if (i + kPiece <= n) {
    __builtin_memcpy(v, p + i, sizeof v);   // any alignment T allows
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = T{};
    if (i < n) {
#pragma unroll
      for (int e = 0; e < kPiece - 1; ++e)
        if (i + e < n) v[e] = p[i + e];
    }
  }
}
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, int i, int n, float (&f)[kPiece]) {
  T v[kPiece];
  load_raw(p, i, n, v);
#pragma unroll
  for (int e = 0; e < kPiece; ++e) f[e] = to_f(v[e]);
}
__device__ __forceinline__ void load_piece(const void* p, int dtype, int i, int n, float (&f)[kPiece]) {
  if (dtype == MOE_F32) load_piece((const float*)p, i, n, f);
  else if (dtype == MOE_BF16) load_piece((const bf16_t*)p, i, n, f);
  else load_piece((const f16_t*)p, i, n, f);
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int i, int n, const float (&f)[kPiece]) {
  if (i + kPiece <= n) {
    T v[kPiece];
#pragma unroll
    for (int e = 0; e < kPiece; ++e) v[e] = from_f<T>(f[e]);
    __builtin_memcpy(p + i, v, sizeof v);
  } else if (i < n) {
#pragma unroll
    for (int e = 0; e < kPiece - 1; ++e)
      if (i + e < n) p[i + e] = from_f<T>(f[e]);
  }
}
__device__ __forceinline__ void store_piece(void* p, int dtype, int64_t at, int i, int n, const float (&f)[kPiece]) {
  if (dtype == MOE_F32) store_piece((float*)p + at, i, n, f);
  else if (dtype == MOE_BF16) store_piece((bf16_t*)p + at, i, n, f);
  else store_piece((f16_t*)p + at, i, n, f);
}

// Sum and maximum over the wave, the same in every lane: four steps inside rows of 16 lanes, then
// lane 15 of a row into the next row and lane 31 into the upper half, and lane 63 has all.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {   // 0 where no lane is read
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp0(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp0<CTRL, ROWS>((uint32_t)b) |
                                        (uint64_t)dpp0<CTRL, ROWS>((uint32_t)(b >> 32)) << 32);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp0<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v += dpp0<0x112, 0xF>(v);
  v += dpp0<0x114, 0xF>(v);
  v += dpp0<0x118, 0xF>(v);
  v += dpp0<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
  v += dpp0<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63) |
                                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63) << 32);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp0<0x111, 0xF>(v));
  v = max(v, dpp0<0x112, 0xF>(v));
  v = max(v, dpp0<0x114, 0xF>(v));
  v = max(v, dpp0<0x118, 0xF>(v));
  v = max(v, dpp0<0x142, 0xA>(v));
  v = max(v, dpp0<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Over the workgroup; `red` is used for one call only.
template <int THREADS>
__device__ __forceinline__ double row_sum(double v, double* red) {
  v = wave_sum(v);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v += red[w];
  }
  return v;
}
template <int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = wave_max(v);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = max(v, red[w]);
  }
  return v;
}

// The largest |y| as its bits, which order like the values, infinities and NaNs above all; in two running
// maxima: of the bits as signed numbers (the positive values) and as unsigned (the negative).
struct AbsMax {
  int pos = 0;
  uint32_t neg = 0x80000000u;
  __device__ __forceinline__ void add(const float (&y)[kPiece]) {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      pos = max(pos, __builtin_bit_cast(int, y[e]));
      neg = max(neg, __builtin_bit_cast(uint32_t, y[e]));
    }
  }
  __device__ __forceinline__ uint32_t bits() const { return max((uint32_t)pos, neg & 0x7FFFFFFFu); }
};

// A float32 whose last mantissa bits are the integer nearest to x rd, and how far x rd is from it.
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
__device__ __forceinline__ float to_code(float x, float rd, float& off) {
  const float y = __builtin_fmaf(x, rd, kMagic);
  off = __builtin_fabsf(__builtin_fmaf(x, rd, kMagic - y));
  return y;
}
__device__ __forceinline__ uint32_t low_bytes(const float (&y)[4]) {
  const uint32_t a = __builtin_bit_cast(uint32_t, y[0]), b = __builtin_bit_cast(uint32_t, y[1]);
  const uint32_t c = __builtin_bit_cast(uint32_t, y[2]), d = __builtin_bit_cast(uint32_t, y[3]);
  return __builtin_amdgcn_perm(b, a, 0x0C0C0400u) | __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
}

// The codes of eight values in a block of scale s (|y| <= amax), as the division gives them, mostly without it:
// x rd is within 2^-16 of x / d (rcp is good to 1 ulp) and the rounded quotient within 2^-18, so that
// where x rd is more than 2^-15 from every half-integer all three round alike; the sum and distance above are
// exact to far less. Elsewhere (2^-13 is asked), and where the scale is out of range, the division.
__device__ __forceinline__ void codes8(const float (&x)[kPiece], const QScale& s, uint32_t (&q)[2]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float y[4], most = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float off;
      y[e] = to_code(x[4 * w + e], s.rd, off);
      most = __builtin_fmaxf(most, off);
    }
    q[w] = low_bytes(y);
    if (!s.ok || !(most < 0.5f - 0x1p-13f)) {
      q[w] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[w] |= ((uint32_t)code_of(x[4 * w + e] / s.d) & 0xFFu) << (8 * e);
    }
  }
}

__device__ __forceinline__ void store_codes(int8_t* q, int i, int n, const uint32_t (&v)[2]) {
  if (i + kPiece <= n) {
    __builtin_memcpy(q + i, v, 8);
  } else {
#pragma unroll
    for (int e = 0; e < kPiece - 1; ++e)
      if (i + e < n) q[i + e] = (int8_t)(v[e / 4] >> (8 * (e & 3)));
  }
}

// The int8 row of y.
template <int THREADS, int C>
__device__ __forceinline__ void write_i8_row(const float (&y)[C][kPiece], int n, int8_t* q, float* scale, uint32_t* red) {
  AbsMax most;
#pragma unroll
  for (int c = 0; c < C; ++c) most.add(y[c]);
  const uint32_t m = row_max<THREADS>(most.bits(), red);
  const bool finite = m < 0x7F800000u;
  const QScale s = q_scale(__builtin_bit_cast(float, m));
  const bool codes = finite && s.d != 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * THREADS + (int)threadIdx.x) * kPiece;
    if (i >= n) break;
    uint32_t v[2] = {0, 0};
    if (codes) codes8(y[c], s, v);
    store_codes(q, i, n, v);
  }
  if (threadIdx.x == 0) *scale = finite ? s.d : __builtin_nanf("");
}

// ------------------------------------------------------------------ 64 bits -----------------

// exp(x) to an ulp or two for x <= 709 (below -745: 0): x = n ln 2 + r, |r| <= ln(2) / 2, and e^r by its
// power series to r^13 (the next term is below 2^-57).
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(__builtin_fmax(x, -1100.0) * 1.4426950408889634);
  const double y = __builtin_fmax(x, -1100.0);
  const double r = __builtin_fma(-n, 2.3190468138462996e-17, __builtin_fma(-n, 0.6931471805599453, y));
  double e = 1.0 / 6227020800.0;
  e = __builtin_fma(e, r, 1.0 / 479001600.0);
  e = __builtin_fma(e, r, 1.0 / 39916800.0);
  e = __builtin_fma(e, r, 1.0 / 3628800.0);
  e = __builtin_fma(e, r, 1.0 / 362880.0);
  e = __builtin_fma(e, r, 1.0 / 40320.0);
  e = __builtin_fma(e, r, 1.0 / 5040.0);
  e = __builtin_fma(e, r, 1.0 / 720.0);
  e = __builtin_fma(e, r, 1.0 / 120.0);
  e = __builtin_fma(e, r, 1.0 / 24.0);
  e = __builtin_fma(e, r, 1.0 / 6.0);
  e = __builtin_fma(e, r, 0.5);
  e = __builtin_fma(e, r, 1.0);
  e = __builtin_fma(e, r, 1.0);
  return __builtin_ldexp(e, (int)n);
}

// 1 / x to an ulp for normal x (infinity gives 0): the seed and two Newton steps.
__device__ __forceinline__ double inverse64(double x) {
  const double s = __builtin_amdgcn_rcp(x);
  const double r = __builtin_fma(__builtin_fma(-x, s, 1.0), s, s);
  const double y = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
  return x < __builtin_inf() ? y : 0.0;
}

// 1 / (1 + exp(-x)) within 4.3 * 2^-53 relative (exp 2.2 of them: r, the last two steps of the series and its end;
// the sum 1, the inverse 1); 0 where exp(-x) passes the largest double.
__device__ __forceinline__ double sigmoid64(double x) { return inverse64(1.0 + exp64(-__builtin_fmax(x, -1000.0))); }

// ------------------------------------------------------------------ host checks -------------

inline bool aligned(const void* p, int size) { return ((uintptr_t)p & (uintptr_t)(size - 1)) == 0; }

// Rows in memory, in bytes: `rows` of `len`, `step` apart (one row: its length).
struct Rows {
  const void* p;
  int64_t rows, len, step;
};
inline Rows rows_of(const void* p, int64_t rows, int64_t n, int64_t ld, int size) { return Rows{p, rows, n * size, (rows > 1 ? ld : n) * size}; }

// Whether a row stride is none: below the row length, or rows that no memory holds (offsets and spans in bytes,
// also those of a tile's rows past the last, then stay far below 2^63).
inline bool bad_stride(int64_t ld, int64_t n, int64_t rows) { return ld < n || ld > MOE_MAX_SPAN / rows; }

// Whether two sets of rows share a byte (for different steps: whether their spans do).
inline bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !a.rows || !b.rows) return false;
  const Rows &x = (uintptr_t)a.p <= (uintptr_t)b.p ? a : b, &y = &x == &a ? b : a;   // x starts first
  const uint64_t gap = (uintptr_t)y.p - (uintptr_t)x.p;
  if (gap >= (uint64_t)((x.rows - 1) * x.step + x.len)) return false;
  if (x.rows > 1 && y.rows > 1 && x.step != y.step) return true;
  const int64_t step = x.rows > 1 ? x.step : y.step;      // one row has the other's
  const int64_t shift = (int64_t)(gap % (uint64_t)step);   // of y's columns
  return shift < x.len || shift + y.len > step;
}

inline int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

constexpr int64_t kLaunchThreads = 0xFFFFFFFFll;   // of one launch, at most

}  // namespace moe
