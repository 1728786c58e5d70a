// Operators around the routed layer for MI355X (gfx950): RMS norm with the residual's addition and
// outputs in 8 bits, the general router, SwiGLU into int8 rows, and the int8 matrix product with
// scales per token and channel. Formulas and edge rules: include/moe_route.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/moe_route.h"
#include "moe_device.hpp"

namespace moe {

int hip_fail(hipError_t e, const char* what);   // moe_route.hip: keeps the text for moe_last_error

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));

// s_waitcnt vmcnt(n), the other counters left alone (n < 64; vmcnt in bits 3:0 and 15:14)
#define MOE_OPS_VM(n) (((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))
// Every LDS access of the wave has finished, then the workgroup meets.
__device__ __forceinline__ void ops_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

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
bool type_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

__device__ __forceinline__ float load_f(const void* p, int dtype, int64_t i) {
  return dtype == MOE_F32 ? ((const float*)p)[i]
         : dtype == MOE_BF16 ? to_f(((const bf16_t*)p)[i]) : to_f(((const f16_t*)p)[i]);
}
__device__ __forceinline__ void store_f(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_F32) ((float*)p)[i] = v;
  else if (dtype == MOE_BF16) ((bf16_t*)p)[i] = from_f<bf16_t>(v);
  else ((f16_t*)p)[i] = from_f<f16_t>(v);
}

// ------------------------------------------------------------------ rows --------------------
//
// moe_add_rmsnorm and moe_swiglu_i8 give a row to one workgroup, which reads it once and keeps it in
// registers, eight neighbouring values a thread (16-byte accesses for 16-bit types) and C such pieces.

constexpr int kPiece = 8;

template <typename T>
__device__ __forceinline__ void load_piece(const T* p, int i, int n, float (&f)[kPiece]) {
  if (i + kPiece <= n) {
    T v[kPiece];
    __builtin_memcpy(v, p + i, sizeof v);   // any alignment T allows
#pragma unroll
    for (int e = 0; e < kPiece; ++e) f[e] = to_f(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) f[e] = i + e < n ? to_f(p[i + e]) : 0.0f;
  }
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
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e)
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
// |y| as its bits: they order like the values, infinities and NaNs above all.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __builtin_bit_cast(uint32_t, y) & 0x7FFFFFFFu; }

__device__ __forceinline__ void codes8(const float (&y)[kPiece], const QScale& s, uint32_t (&q)[2]) {
  const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
  q[0] = quant_pack4(lo, s);
  q[1] = quant_pack4(hi, s);
}

// The int8 row of y.
template <int THREADS, int C>
__device__ __forceinline__ void write_i8_row(const float (&y)[C][kPiece], int n, int8_t* q, float* scale, uint32_t* red) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < kPiece; ++e) m = max(m, abs_bits(y[c][e]));
  m = row_max<THREADS>(m, red);
  const bool finite = m < 0x7F800000u;
  const QScale s = q_scale(__builtin_bit_cast(float, m));
  const bool codes = finite && s.d != 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * THREADS + (int)threadIdx.x) * kPiece;
    if (i >= n) break;
    uint32_t v[2] = {0, 0};
    if (codes) codes8(y[c], s, v);
    if (i + kPiece <= n) {
      __builtin_memcpy(q + i, v, 8);
    } else {
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        if (i + e < n) q[i + e] = (int8_t)(v[e / 4] >> (8 * (e & 3)));
    }
  }
  if (threadIdx.x == 0) *scale = finite ? s.d : __builtin_nanf("");
}

// ------------------------------------------------------------------ norm --------------------

struct NormArgs {
  const void *x, *res, *weight;
  void *res_out, *y, *q8_1;
  int8_t* q;
  float* scale;
  int64_t ldx, ldres, ldro, ldy, ldq;
  int w_dtype, y_dtype, n;
  float eps;
};

// The sum of squares and y are in 64 bits (y's one rounding to float32 then decides every code, whatever
// the order of the sum): on this chip a 64-bit product costs what a 32-bit one does, and the row's bytes
// take longer.
template <typename T, int THREADS, int C>
__global__ __launch_bounds__(THREADS) void k_add_rmsnorm(NormArgs a) {
  __shared__ double s_sum[THREADS / 64];
  __shared__ uint32_t s_max[THREADS / 64];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* res = (const T*)a.res + row * a.ldres;
  float r[C][kPiece], w[C][kPiece];
#pragma unroll
  for (int c = 0; c < C; ++c) load_piece(x, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, r[c]);
  if (a.res) {
    float s[C][kPiece];
#pragma unroll
    for (int c = 0; c < C; ++c) load_piece(res, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, s[c]);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < kPiece; ++e) r[c][e] = to_f(from_f<T>(r[c][e] + s[c][e]));
  }
#pragma unroll
  for (int c = 0; c < C; ++c) load_piece(a.weight, a.w_dtype, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, w[c]);
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < kPiece; ++e) sum = __builtin_fma((double)r[c][e], (double)r[c][e], sum);
  if (a.res_out) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      store_piece((T*)a.res_out + row * a.ldro, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, r[c]);
  }
  sum = row_sum<THREADS>(sum, s_sum);
  const double rinv = 1.0 / __builtin_sqrt(sum / a.n + (double)a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      const int i = (c * THREADS + (int)threadIdx.x) * kPiece + e;
      const float y = (float)((double)r[c][e] * rinv * (double)w[c][e]);
      r[c][e] = i < a.n ? y : 0.0f;   // past the row 0 * rinv * 0, where rinv may not be finite
    }
  if (a.y) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      store_piece(a.y, a.y_dtype, row * a.ldy, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, r[c]);
  }
  if (a.q8_1) {   // four threads a block of 32
    const int nb = a.n / 32;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * THREADS + (int)threadIdx.x) * kPiece, part = threadIdx.x & 3;
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        const float v = __builtin_fabsf(r[c][e]);
        amax = v > amax ? v : amax;
      }
      float o = dpp<0xB1>(amax);   // quad_perm: the neighbour, then the other pair
      amax = o > amax ? o : amax;
      o = dpp<0x4E>(amax);
      amax = o > amax ? o : amax;
      const QScale qs = q_scale(amax);
      uint32_t v[2] = {0, 0};
      if (amax != 0.0f) codes8(r[c], qs, v);
      int isum = 0;
#pragma unroll
      for (int e = 0; e < kPiece; ++e) isum += (int)(int8_t)(v[e / 4] >> (8 * (e & 3)));
      isum += __builtin_amdgcn_update_dpp(0, isum, 0xB1, 0xF, 0xF, false);
      isum += __builtin_amdgcn_update_dpp(0, isum, 0x4E, 0xF, 0xF, false);
      if (i < a.n) {
        uint32_t* blk = (uint32_t*)((uint8_t*)a.q8_1 + 36 * (row * nb + i / 32));
        const uint32_t d16 = f2h(qs.d);
        if (part == 0) blk[0] = d16 | (sum_field(d16, isum) << 16);
        blk[1 + 2 * part] = v[0];
        blk[2 + 2 * part] = v[1];
      }
    }
  }
  if (a.q) write_i8_row<THREADS, C>(r, a.n, a.q + row * a.ldq, a.scale + row, s_max);
}

// ------------------------------------------------------------------ SwiGLU ------------------

// 1 / (1 + exp(-g)) within some 2^-45 relative: exp(-g) = 2^n 2^f with n = rint(t), t = -g log2(e), and
// 2^f, |f| <= 1/2, by its power series to f^11 (the next term is below 2^-47); the reciprocal's seed takes
// one Newton step. t is held to +-1000: beyond, the result times any two float32 values rounds as it
// does there.
__device__ __forceinline__ double sigmoid64(double g) {
  const double t = __builtin_fmin(__builtin_fmax(g * -1.4426950408889634, -1000.0), 1000.0);
  const double n = __builtin_rint(t), f = t - n;
  double e = 4.44553827187081e-10;
  e = __builtin_fma(e, f, 7.054911620801121e-09);
  e = __builtin_fma(e, f, 1.0178086009239696e-07);
  e = __builtin_fma(e, f, 1.3215486790144305e-06);
  e = __builtin_fma(e, f, 1.5252733804059838e-05);
  e = __builtin_fma(e, f, 0.00015403530393381606);
  e = __builtin_fma(e, f, 0.0013333558146428441);
  e = __builtin_fma(e, f, 0.009618129107628477);
  e = __builtin_fma(e, f, 0.055504108664821576);
  e = __builtin_fma(e, f, 0.2402265069591007);
  e = __builtin_fma(e, f, 0.6931471805599453);
  e = __builtin_fma(e, f, 1.0);
  const double den = 1.0 + __builtin_ldexp(e, (int)n);
  const double x = __builtin_amdgcn_rcp(den);
  return __builtin_fma(__builtin_fma(-den, x, 1.0), x, x);
}

struct SwigluArgs {
  const void *g, *u;
  int8_t* q;
  float* scale;
  int64_t ldg, ldu, ldq;
  int n;
};

template <typename T, int THREADS, int C>
__global__ __launch_bounds__(THREADS) void k_swiglu_i8(SwigluArgs a) {
  __shared__ uint32_t s_max[THREADS / 64];
  const int64_t row = blockIdx.x;
  const T* gp = (const T*)a.g + row * a.ldg;
  const T* up = (const T*)a.u + row * a.ldu;
  float g[C][kPiece], u[C][kPiece];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_piece(gp, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, g[c]);
    load_piece(up, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, u[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      const double gd = (double)g[c][e];
      g[c][e] = (float)(gd * sigmoid64(gd) * (double)u[c][e]);
    }
  write_i8_row<THREADS, C>(g, a.n, a.q + row * a.ldq, a.scale + row, s_max);
}

// ------------------------------------------------------------------ router ------------------

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int64_t ld;
  int dtype, E, k, score, n_groups, keep, top, renorm;
  float factor;
};

constexpr int kRouteE = 1024;

// One wave a token; expert e sits in lane e % 64.
__global__ __launch_bounds__(64) void k_route_scores(RouteArgs a) {
  __shared__ double s_c[kRouteE];        // scores to order by; -inf: masked
  __shared__ float s_l[kRouteE];         // logits as float32
  __shared__ double s_group[64];
  __shared__ unsigned char s_alive[kRouteE];
  __shared__ int s_ids[32];
  __shared__ double s_w[32];
  const int lane = threadIdx.x, E = a.E, per = E / a.n_groups;
  const int64_t t = blockIdx.x;
  float peak = -__builtin_inff();
  for (int e = lane; e < E; e += 64) {
    float l = load_f(a.logits, a.dtype, t * a.ld + e);
    l = l != l ? -__builtin_inff() : __builtin_fminf(l, 3.40282347e38f);
    s_l[e] = l;
    peak = __builtin_fmaxf(peak, l);
  }
  for (int o = 32; o; o >>= 1) peak = __builtin_fmaxf(peak, __shfl_xor(peak, o));
  double total = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    for (int e = lane; e < E; e += 64)
      if (s_l[e] > -__builtin_inff()) total += exp((double)s_l[e] - (double)peak);
    for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
  }
  auto score = [&](float l) -> double {
    if (!(l > -__builtin_inff())) return 0.0;
    return a.score == MOE_SCORE_SOFTMAX ? exp((double)l - (double)peak) / total : 1.0 / (1.0 + exp(-(double)l));
  };
  for (int e = lane; e < E; e += 64) {
    const bool masked = !(s_l[e] > -__builtin_inff());
    double c = score(s_l[e]);
    if (a.bias) c = fmin(fmax(c + (double)a.bias[e], -1e300), 1e300);
    s_c[e] = masked ? -__builtin_inf() : c;
    s_alive[e] = 1;
  }
  __syncthreads();
  if (a.n_groups > 1) {
    double gs = -__builtin_inf();
    if (lane < a.n_groups) {
      double b0 = -__builtin_inf(), b1 = b0;
      for (int i = 0; i < per; ++i) {
        const double c = s_c[lane * per + i];
        if (c > b0) {
          b1 = b0;
          b0 = c;
        } else if (c > b1) {
          b1 = c;
        }
      }
      gs = a.top == 2 && b1 > -__builtin_inf() ? b0 + b1 : b0;
      s_group[lane] = gs;
    }
    __syncthreads();
    if (lane < a.n_groups) {
      int ahead = 0;
      for (int g = 0; g < a.n_groups; ++g) ahead += s_group[g] > gs || (s_group[g] == gs && g < lane);
      if (ahead >= a.keep)
        for (int i = 0; i < per; ++i) s_alive[lane * per + i] = 0;
    }
    __syncthreads();
  }
  for (int j = 0; j < a.k; ++j) {
    double best = -__builtin_inf();
    int at = kRouteE;
    for (int e = lane; e < E; e += 64) {
      const double c = a.bias ? s_c[e] : (double)s_l[e];
      if (s_alive[e] && (c > best || (c == best && e < at))) {
        best = c;
        at = e;
      }
    }
    for (int o = 32; o; o >>= 1) {
      const double c = __shfl_xor(best, o);
      const int e = __shfl_xor(at, o);
      if (c > best || (c == best && e < at)) {
        best = c;
        at = e;
      }
    }
    if (lane == 0) {
      s_ids[j] = at;
      s_w[j] = score(s_l[at]);
      s_alive[at] = 0;
    }
    __syncthreads();
  }
  if (lane < a.k) {
    double sum = 1.0;
    if (a.renorm) {
      sum = 0.0;
      for (int j = 0; j < a.k; ++j) sum += s_w[j];
      if (sum == 0.0) sum = 1.0;
    }
    a.ids[t * a.k + lane] = s_ids[lane];
    a.w[t * a.k + lane] = (float)(s_w[lane] / sum * (double)a.factor);
  }
}

// ------------------------------------------------------------------ int8 product ------------

struct MatmulArgs {
  const int8_t *a, *b;
  const float *sa, *sb;
  void* c;
  int64_t lda, ldb, ldc;
  int M, N, K, accumulate;
  int tiles_n, tiles;   // tile grid: channels, all
  int vec;              // rows of C and sb take four-value accesses
  int c_dtype;
};

// 16 bytes of a row from column k, zero from column K on (rows at any alignment): the last 16 bytes of
// the row shifted down where the piece passes K. Rows shorter than that are read byte by byte.
__device__ __forceinline__ i32x4 row16(const int8_t* p, int k, int K) {
  uint64_t lo = 0, hi = 0;
  if (K < 16) {
#pragma unroll 1
    for (int i = K - 1; i >= k; --i) {
      hi = hi << 8 | lo >> 56;
      lo = lo << 8 | (uint64_t)(uint8_t)p[i];
    }
  } else {
    const int at = min(k, K - 16), cut = min(k - at, 16), sh = 8 * (cut & 7);
    __builtin_memcpy(&lo, p + at, 8);
    __builtin_memcpy(&hi, p + at + 8, 8);
    if (cut >= 8) lo = hi, hi = 0;
    if (sh) lo = lo >> sh | hi << (64 - sh), hi >>= sh;
    if (cut == 16) lo = 0;
  }
  return __builtin_bit_cast(i32x4, u64x2{lo, hi});
}
__device__ __forceinline__ i32x4 any16(const int8_t* p) {   // 16 bytes at any alignment
  i32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// One value of C: scales, the previous value, the type's rounding.
template <typename T>
__device__ __forceinline__ void store_one(const MatmulArgs& p, int m, int n, int sum) {
  T* c = (T*)p.c + m * p.ldc + n;
  float v = (float)sum * p.sa[m] * p.sb[n];
  if (p.accumulate) v += to_f(*c);
  *c = from_f<T>(v);
}
// Four neighbouring channels of one token.
template <typename T>
__device__ __forceinline__ void store_four(const MatmulArgs& p, int m, int n, float sa, const f32x4& sb, i32x4 s) {
  struct alignas(4 * sizeof(T)) T4 {
    T v[4];
  };
  T4* c = (T4*)((T*)p.c + m * p.ldc + n);
  T4 o;
  if (p.accumulate) {
    const T4 old = *c;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = from_f<T>((float)s[i] * sa * sb[i] + to_f(old.v[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = from_f<T>((float)s[i] * sa * sb[i]);
  }
  *c = o;
}

constexpr int kMmK = 128;   // bytes of K per step

// One workgroup a tile of BT tokens x BC channels, WT x WC waves. v_mfma_i32_16x16x64_i8 with the
// channels as rows and the tokens as columns, so that a lane ends with four neighbouring channels of
// one token. A ring of S stages in LDS holds BT + BC rows of 128 bytes, a row's 16-byte chunk c at
// place c ^ (row & 7): the eight rows that eight lanes read at one chunk then sit in different banks.
// DIRECT: rows and their stride are 16-byte aligned and go straight to LDS; else through registers. A
// last piece of K below 128 bytes is taken first, through registers, zero past K.
template <int BT, int BC, int WT, int WC, bool DIRECT>
__global__ __launch_bounds__(64 * WT * WC) void k_matmul_tile(MatmulArgs p) {
  extern __shared__ __align__(16) uint8_t s_ring[];
  constexpr int W = WT * WC, R = BT + BC, L = R / 8 / W;   // L: 8-row pieces a wave loads per step
  constexpr int NT = BT / WT / 16, NC = BC / WC / 16, STAGE = R * kMmK;
  static_assert(R % (8 * W) == 0 && BT % (16 * WT) == 0 && BC % (16 * WC) == 0 && NC >= 2, "tile split");
  static_assert(2 * STAGE >= W * NC * 1024, "the epilogue's piece of each wave fits");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // Workgroups go to the eight dies in turn: each die takes one run of tiles, in 4-token-tile strips, so
  // that what its workgroups read together is a near-square patch that its L2 holds.
  int id = blockIdx.x;
  {
    const int per = p.tiles / 8, extra = p.tiles % 8, die = id & 7, i = id >> 3;
    id = die * per + min(die, extra) + i;
  }
  const int tiles_m = p.tiles / p.tiles_n, strip = id / (4 * p.tiles_n), in = id - strip * 4 * p.tiles_n;
  const int hs = min(4, tiles_m - 4 * strip);
  const int m0 = (4 * strip + in % hs) * BT, n0 = (in / hs) * BC;

  // this lane's rows: piece i of the wave is rows 8 (wave + W i) .. + 7 of the stage, tokens first
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  const int8_t* src[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int r = 8 * (wave + W * i) + (lane >> 3);
    src[i] = (r < BT ? p.a + min(m0 + r, p.M - 1) * p.lda : p.b + min(n0 + r - BT, p.N - 1) * p.ldb) + chunk;
  }
  const int rem = p.K % kMmK, steps = (p.K + kMmK - 1) / kMmK;
  i32x4 hold[L];
  auto fetch = [&](int t) {   // step t on its way to LDS, or to registers
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if constexpr (DIRECT)
        __builtin_amdgcn_global_load_lds((const void*)src[i],
                                         (MOE_LDS void*)(s_ring + (t & 1) * STAGE + 1024 * (wave + W * i)), 16, 0, 0);
      else
        hold[i] = any16(src[i]);
      src[i] += kMmK;
    }
  };
  auto put = [&](int t) {     // registers to LDS
#pragma unroll
    for (int i = 0; i < L; ++i) *(i32x4*)(s_ring + (t & 1) * STAGE + 1024 * (wave + W * i) + 16 * lane) = hold[i];
  };
  const int wt = wave % WT, wc = wave / WT, row = lane & 15, quad = lane >> 4;
  i32x4 acc[NC][NT];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto compute = [&](int t) {
    const uint8_t* st = s_ring + (t & 1) * STAGE;
    i32x4 av[2][NC], bv[2][NT];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int at = ((4 * kk + quad) ^ (row & 7)) * 16 + row * kMmK;
#pragma unroll
      for (int j = 0; j < NT; ++j) bv[kk][j] = *(const i32x4*)(st + (wt * NT + j) * 16 * kMmK + at);
#pragma unroll
      for (int i = 0; i < NC; ++i) av[kk][i] = *(const i32x4*)(st + (BT + (wc * NC + i) * 16) * kMmK + at);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[kk][i], bv[kk][j], acc[i][j], 0, 0, 0);
    // reads two channel tiles ahead of the products that use them
    __builtin_amdgcn_sched_group_barrier(0x100, NT + 2, 0);
#pragma unroll
    for (int s = 0; s < 2 * NC; ++s) {
      __builtin_amdgcn_sched_group_barrier(0x008, NT, 0);
      if (s < NC - 2 || (s >= NC && s < 2 * NC - 2)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (s == NC - 2) __builtin_amdgcn_sched_group_barrier(0x100, NT / 2 + 1, 0);
      if (s == NC - 1) __builtin_amdgcn_sched_group_barrier(0x100, NT - NT / 2 + 1, 0);
    }
  };
  if (rem) {
#pragma unroll
    for (int i = 0; i < L; ++i) hold[i] = row16(src[i] - chunk, p.K - rem + chunk, p.K);
    put(0);
  } else {
    fetch(0);
    if (!DIRECT) put(0);
  }
  for (int t = 0; t < steps; ++t) {
    __builtin_amdgcn_s_waitcnt(MOE_OPS_VM(0));
    ops_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (t + 1 < steps) fetch(t + 1);
    compute(t);
    __builtin_amdgcn_sched_barrier(0);
    if (!DIRECT && t + 1 < steps) put(t + 1);
  }
  auto finish = [&](auto type) {
    using T = decltype(type);
    if (p.vec && m0 + BT <= p.M && n0 + BC <= p.N) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = m0 + (wt * NT + j) * 16 + row;
        const float sa = p.sa[m];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int n = n0 + (wc * NC + i) * 16 + 4 * quad;
          store_four<T>(p, m, n, sa, *(const f32x4*)(p.sb + n), acc[i][j]);
        }
      }
    } else {   // ragged or unaligned: through the wave's piece of LDS, so that lanes write along a row
      ops_barrier();
      int* mine = (int*)(s_ring + wave * NC * 1024);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < NC; ++i) *(i32x4*)(mine + row * 16 * NC + 16 * i + 4 * quad) = acc[i][j];
        __builtin_amdgcn_wave_barrier();
        const int m1 = m0 + (wt * NT + j) * 16, n1 = n0 + wc * NC * 16;
#pragma unroll 1
        for (int e = lane; e < 256 * NC; e += 64) {
          const int m = m1 + e / (16 * NC), n = n1 + e % (16 * NC);
          if (m < p.M && n < p.N) store_one<T>(p, m, n, mine[e]);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  };
  if (p.c_dtype == MOE_F32) finish(float{});
  else if (p.c_dtype == MOE_BF16) finish(bf16_t{});
  else finish(f16_t{});
}

// Few tokens (M <= 16 MT): the weights are read once, straight into the lanes of the matrix
// instruction, and a workgroup's W waves share out K, so that each has few dependent loads. C = 16 / P
// channels a workgroup: with P > 1 (M <= C) the instruction's 16 rows are C channels at P neighbouring
// pieces of K and its 16 columns the tokens at the same pieces; the blocks of its result where the
// two pieces agree are partial sums of the product. Few channels then still fill the chip.
template <int MT, int P, int W>
__global__ __launch_bounds__(64 * W) void k_matmul_thin(MatmulArgs p) {
  constexpr int C = 16 / P, PIECE = 128 * P, STRIDE = PIECE * W, UN = MT == 4 ? 2 : 4;
  __shared__ i32x4 s_sum[W][MT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int row = lane & 15, quad = lane >> 4, n0 = blockIdx.x * C;
  const int8_t* b = p.b + (int64_t)min(n0 + row % C, p.N - 1) * p.ldb;
  const int8_t* a[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) a[j] = p.a + (int64_t)min(16 * j + row % C, p.M - 1) * p.lda;
  // what this thread stores at the end: channels on .. on + 3 of token om
  const int outs = MT * C * C / 4, om = (int)threadIdx.x / (C / 4), on = n0 + 4 * ((int)threadIdx.x % (C / 4));
  const bool mine = (int)threadIdx.x < outs && om < p.M && on < p.N;
  float sa = 0.0f;
  f32x4 sb = {0.0f, 0.0f, 0.0f, 0.0f};
  if (mine) {
    sa = p.sa[om];
#pragma unroll
    for (int i = 0; i < 4; ++i) sb[i] = p.sb[min(on + i, p.N - 1)];
  }
  i32x4 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = i32x4{0, 0, 0, 0};
  int k = wave * PIECE + (row / C) * 64 + quad * 16;   // this lane's 16 bytes; the next are 64 P on
  int left = p.K - wave * PIECE;                       // bytes of K from the wave's piece on
  for (; left >= PIECE + (UN - 1) * STRIDE; left -= UN * STRIDE) {
    i32x4 bv[UN][2], av[UN][2][MT];
#pragma unroll
    for (int v = 0; v < UN; ++v)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = k + v * STRIDE + u * 64 * P;
        bv[v][u] = any16(b + at);
#pragma unroll
        for (int j = 0; j < MT; ++j) av[v][u][j] = any16(a[j] + at);
      }
#pragma unroll
    for (int v = 0; v < UN; ++v)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[v][u], av[v][u][j], acc[j], 0, 0, 0);
    k += UN * STRIDE;
  }
  for (; left >= PIECE; left -= STRIDE) {
    i32x4 bv[2], av[2][MT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bv[u] = any16(b + k + u * 64 * P);
#pragma unroll
      for (int j = 0; j < MT; ++j) av[u][j] = any16(a[j] + k + u * 64 * P);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[u], av[u][j], acc[j], 0, 0, 0);
    k += STRIDE;
  }
  if (left > 0) {   // the wave that K ends in: zeros past it
    i32x4 bv[2], av[2][MT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bv[u] = row16(b, k + u * 64 * P, p.K);
#pragma unroll
      for (int j = 0; j < MT; ++j) av[u][j] = row16(a[j], k + u * 64 * P, p.K);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[u], av[u][j], acc[j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) s_sum[wave][j][lane] = acc[j];
  __syncthreads();
  if (!mine) return;
  // rows 4 q .. 4 q + 3 of the result are with quad q: channel group g of piece s is rows s C + 4 g
  const int j = om / 16, t = om % 16, g = (on - n0) / 4;
  i32x4 sum = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int s = 0; s < P; ++s) sum += s_sum[w][j][(s * C / 4 + g) * 16 + s * C + t];
  auto finish = [&](auto type) {
    using T = decltype(type);
    if (p.vec && on + 4 <= p.N) {
      store_four<T>(p, om, on, sa, sb, sum);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (on + i < p.N) store_one<T>(p, om, on + i, sum[i]);
    }
  };
  if (p.c_dtype == MOE_F32) finish(float{});
  else if (p.c_dtype == MOE_BF16) finish(bf16_t{});
  else finish(f16_t{});
}

// ------------------------------------------------------------------ host checks -------------

bool aligned(const void* p, int size) { return ((uintptr_t)p & (uintptr_t)(size - 1)) == 0; }

// Whether two sets of rows share a byte (their whole spans, padding included).
bool overlap(const void* p, int64_t ldp, int sp, const void* q, int64_t ldq, int sq, int rows, int n) {
  if (!p || !q) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const uintptr_t na = (uintptr_t)(((rows - 1) * ldp + n) * sp), nb = (uintptr_t)(((rows - 1) * ldq + n) * sq);
  return a < b + nb && b < a + na;
}

// A row call's type and workgroup: by the row length alone, so that a row's sums have one order.
template <typename F>
void with_row(int dtype, int n, F f) {
  auto size = [&](auto t) {
    using std::integral_constant;
    if (n <= 64 * kPiece) f(t, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (n <= 256 * kPiece) f(t, integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (n <= 512 * kPiece) f(t, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (n <= 1024 * kPiece) f(t, integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else f(t, integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  };
  with_type(dtype, size);
}
static_assert(1024 * 2 * kPiece == MOE_MAX_ROW, "the longest row fits one workgroup");

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

template <int BT, int BC, int WT, int WC>
int launch_tile(hipStream_t st, MatmulArgs p, bool direct) {
  const int64_t tn = (p.N + BC - 1) / BC, tiles = tn * ((p.M + BT - 1) / BT);
  if (tiles > 0x7FFFFFFF) return MOE_E_SHAPE;
  p.tiles_n = (int)tn;
  p.tiles = (int)tiles;
  constexpr int lds = 2 * (BT + BC) * kMmK;
  auto go = [&](auto kern) {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return hip_fail(e, "moe_matmul_i8");
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(64 * WT * WC), lds, st, p);
    return launched("moe_matmul_i8");
  };
  return direct ? go(k_matmul_tile<BT, BC, WT, WC, true>) : go(k_matmul_tile<BT, BC, WT, WC, false>);
}

int run_matmul(hipStream_t st, MatmulArgs p) {
  const bool direct = aligned(p.a, 16) && aligned(p.b, 16) && p.lda % 16 == 0 && p.ldb % 16 == 0;
  p.vec = aligned(p.sb, 16) && aligned(p.c, 4 * type_size(p.c_dtype)) && p.ldc % 4 == 0;
  if (p.M <= 64) {
    auto go = [&](auto kern, int channels, int threads) {
      hipLaunchKernelGGL(kern, dim3((unsigned)(((int64_t)p.N + channels - 1) / channels)), dim3(threads), 0, st, p);
      return launched("moe_matmul_i8");
    };
    // as few pieces of K side by side as leave two workgroups a CU
    if (p.M <= 4 && p.N < 8 * 512) return go(k_matmul_thin<1, 4, 8>, 4, 512);
    if (p.M <= 8 && p.N < 16 * 512) return go(k_matmul_thin<1, 2, 8>, 8, 512);
    if (p.M <= 16) return go(k_matmul_thin<1, 1, 8>, 16, 512);
    if (p.M <= 32) return go(k_matmul_thin<2, 1, 8>, 16, 512);
    return go(k_matmul_thin<4, 1, 8>, 16, 512);
  }
  const int64_t big = (int64_t)((p.M + 255) / 256) * ((p.N + 255) / 256);
  const int64_t mid = (int64_t)((p.M + 127) / 128) * ((p.N + 127) / 128);
  if (big >= 200) return launch_tile<256, 256, 4, 2>(st, p, direct);
  if (mid >= 200) return launch_tile<128, 128, 2, 2>(st, p, direct);
  return launch_tile<64, 64, 2, 2>(st, p, direct);
}

}  // namespace moe

using namespace moe;

// ------------------------------------------------------------------ C ABI -------------------

extern "C" {

int moe_add_rmsnorm(void* stream, int dtype, const void* x, int64_t ldx, const void* res, int64_t ldres,
                    int w_dtype, const void* weight, float eps, int rows, int n, void* res_out, int64_t ldro,
                    int y_dtype, void* yout, int64_t ldy, int8_t* q, int64_t ldq, float* scale, void* q8_1) {
  if (!type_ok(dtype) || !type_ok(w_dtype) || (yout && !type_ok(y_dtype)) || rows < 0) return MOE_E_ARG;
  if (!(eps > 0.0f) || !(eps < __builtin_inff())) return MOE_E_ARG;
  if (n < 1 || n > MOE_MAX_ROW || (q8_1 && n % 32)) return MOE_E_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !weight || !q != !scale || (!res_out && !yout && !q && !q8_1)) return MOE_E_ARG;
  if (ldx < n || (res && ldres < n) || (res_out && ldro < n) || (yout && ldy < n) || (q && ldq < n)) return MOE_E_ARG;
  const int sz = type_size(dtype), szy = type_size(y_dtype);
  if (!aligned(x, sz) || !aligned(res, sz) || !aligned(res_out, sz) || !aligned(weight, type_size(w_dtype)) ||
      (yout && !aligned(yout, szy)) || !aligned(scale, 4) || !aligned(q8_1, 4))
    return MOE_E_ARG;
  const int64_t nb8 = (int64_t)n / 32 * 36;
  for (int i = 0; i < 2; ++i) {   // outputs over inputs: r over x or res, the very same rows, and nothing else
    const void* in = i ? res : x;
    const int64_t ldi = i ? ldres : ldx;
    if (!(in == res_out && ldi == ldro) && overlap(in, ldi, sz, res_out, ldro, sz, rows, n)) return MOE_E_ARG;
    if (overlap(in, ldi, sz, yout, ldy, szy, rows, n) || overlap(in, ldi, sz, q, ldq, 1, rows, n)) return MOE_E_ARG;
    if (overlap(in, ldi * sz, 1, q8_1, nb8, 1, rows, std::max<int>(n * sz, (int)nb8))) return MOE_E_ARG;
  }
  const NormArgs a{x, res, weight, res_out, yout, q8_1, q, scale, ldx, ldres, ldro, ldy, ldq, w_dtype, y_dtype, n, eps};
  with_row(dtype, n, [&](auto t, auto threads, auto pieces) {
    hipLaunchKernelGGL((k_add_rmsnorm<decltype(t), threads(), pieces()>), dim3(rows), dim3(threads()), 0, (hipStream_t)stream, a);
  });
  return launched("moe_add_rmsnorm");
}

int moe_route_scores(void* stream, int dtype, const void* logits, int64_t ld, int T, int E, int k, int score,
                     const float* bias, int n_groups, int keep_groups, int group_top, int renorm, float factor,
                     int32_t* ids, float* w) {
  if (!type_ok(dtype) || T < 0 || E < 1 || E > kRouteE || k < 1 || k > 32) return MOE_E_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_E_ARG;
  if (n_groups < 1 || n_groups > 64 || E % n_groups || keep_groups < 1 || keep_groups > n_groups) return MOE_E_ARG;
  const int per = E / n_groups;
  if (k > keep_groups * per || group_top < 1 || group_top > 2 || group_top > per) return MOE_E_ARG;
  if ((renorm != 0 && renorm != 1) || !(factor == factor) || ld < E) return MOE_E_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !w || !aligned(logits, type_size(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(w, 4))
    return MOE_E_ARG;
  const RouteArgs a{logits, bias, ids, w, ld, dtype, E, k, score, n_groups, keep_groups, group_top, renorm, factor};
  hipLaunchKernelGGL(k_route_scores, dim3(T), dim3(64), 0, (hipStream_t)stream, a);
  return launched("moe_route_scores");
}

int moe_swiglu_i8(void* stream, int dtype, const void* g, int64_t ldg, const void* u, int64_t ldu, int rows, int n,
                  int8_t* q, int64_t ldq, float* scale) {
  if (!type_ok(dtype) || rows < 0) return MOE_E_ARG;
  if (n < 1 || n > MOE_MAX_ROW) return MOE_E_SHAPE;
  if (rows == 0) return MOE_OK;
  const int sz = type_size(dtype);
  if (!g || !u || !q || !scale || ldg < n || ldu < n || ldq < n) return MOE_E_ARG;
  if (!aligned(g, sz) || !aligned(u, sz) || !aligned(scale, 4)) return MOE_E_ARG;
  if (overlap(g, ldg, sz, q, ldq, 1, rows, n) || overlap(u, ldu, sz, q, ldq, 1, rows, n)) return MOE_E_ARG;
  const SwigluArgs a{g, u, q, scale, ldg, ldu, ldq, n};
  with_row(dtype, n, [&](auto t, auto threads, auto pieces) {
    hipLaunchKernelGGL((k_swiglu_i8<decltype(t), threads(), pieces()>), dim3(rows), dim3(threads()), 0, (hipStream_t)stream, a);
  });
  return launched("moe_swiglu_i8");
}

int moe_matmul_i8(void* stream, const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb,
                  const float* sb, int M, int N, int K, int c_dtype, void* C, int64_t ldc, int accumulate) {
  if (!type_ok(c_dtype) || M < 0 || N < 0 || (accumulate != 0 && accumulate != 1)) return MOE_E_ARG;
  if (K < 1 || K > MOE_MAX_MATMUL_K) return MOE_E_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  if (!a || !sa || !b || !sb || !C || lda < K || ldb < K || ldc < N) return MOE_E_ARG;
  if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(C, type_size(c_dtype))) return MOE_E_ARG;
  return run_matmul((hipStream_t)stream, MatmulArgs{a, b, sa, sb, C, lda, ldb, ldc, M, N, K, accumulate, 0, 0, 0, c_dtype});
}

}  // extern "C"
