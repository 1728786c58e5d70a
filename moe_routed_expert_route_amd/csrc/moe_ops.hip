// Operators around the routed layer for MI355X (gfx950): RMS norm with the residual's addition and
// outputs in 8 bits, the general router, SwiGLU into int8 rows, and the int8 matrix product with
// scales per token and channel. Formulas and edge rules: include/moe_route.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_rows.hpp"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));

// s_waitcnt vmcnt(n), the other counters left alone (n < 64; vmcnt in bits 3:0 and 15:14)
#define MOE_OPS_VM(n) (((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))
// Every LDS access of the wave has finished, then the workgroup meets.
__device__ __forceinline__ void ops_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
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

// The sum of squares and y are in 64 bits: y's one rounding to float32 then decides every code, whatever the
// order of the sum. That is seven of some forty instructions a value, and the row's bytes take longer: 8192 x
// 4096 bf16 with a residual runs at 4.5 TB/s (52 us), float32 rows at 5.0.
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
  for (int c = 0; c < C; ++c) {
    if ((c * THREADS + (int)threadIdx.x) * kPiece >= a.n) break;   // whole waves, but for one
#pragma unroll
    for (int e = 0; e < kPiece; ++e) sum = __builtin_fma((double)r[c][e], (double)r[c][e], sum);
  }
  if (a.res_out) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      store_piece((T*)a.res_out + row * a.ldro, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, r[c]);
  }
  sum = row_sum<THREADS>(sum, s_sum);
  const double rinv = 1.0 / __builtin_sqrt(sum / a.n + (double)a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * THREADS + (int)threadIdx.x) * kPiece;
    if (i >= a.n) break;
#pragma unroll
    for (int e = 0; e < kPiece; ++e) r[c][e] = (float)((double)r[c][e] * rinv * (double)w[c][e]);
    if (i + kPiece > a.n) {   // past the row 0 * rinv * 0, where rinv may not be finite
#pragma unroll
      for (int e = 1; e < kPiece; ++e)
        if (i + e >= a.n) r[c][e] = 0.0f;
    }
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
      float amax = 0.0f, y[kPiece];
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        y[e] = r[c][e] == r[c][e] ? r[c][e] : 0.0f;   // the block quantizer gives a NaN code 0
        const float v = __builtin_fabsf(y[e]);
        amax = v > amax ? v : amax;
      }
      float o = dpp<0xB1>(amax);   // quad_perm: the neighbour, then the other pair
      amax = o > amax ? o : amax;
      o = dpp<0x4E>(amax);
      amax = o > amax ? o : amax;
      const QScale qs = q_scale(amax);
      uint32_t v[2] = {0, 0};
      if (amax != 0.0f) codes8(y, qs, v);
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

struct SwigluArgs {
  const void *g, *u;
  int8_t* q;
  float* scale;
  int64_t ldg, ldu, ldq;
  int n;
};

// h, the one that counts: 64 bits (within 2^-50: the sigmoid and two products), rounded once.
__device__ __forceinline__ float swiglu64(float g, float u) {
  return (float)((double)g * sigmoid64((double)g) * (double)u);
}

// The codes need h's last bits only next to a code's border, and the row's scale those of its largest value.
// So every h is first taken in float32, within 2^-20 relative: t = -g log2(e) in two parts, exp2 of the
// large one (2^-23) times 1 + ln(2) of the small, 1 / (1 + e) (rcp: 2^-23) and roundings of 2^-24 in the
// product of the parts, 1 + e, times g, times u and h in 64 bits: 4.5 * 2^-23 in all, and 8 * 2^-23 is allowed.
// The values within 2^-18 of the largest are taken again in 64 bits and give the scale; so is a value whose
// quotient lies within 2^-19 of its size, plus 2^-17, of a half-integer: the errors of the value, of rcp and of
// the float32 quotient come to 2^-20 + 2^-22 of it. Pieces with a value that the bound leaves out (exp2 past
// 2^100, a product below 2^-100 or not below 2^126) go in 64 bits altogether. Every result is that of 64 bits
// throughout, which took 38 us for 4096 x 5632 bf16; this takes 34.5 (3.4 TB/s). The pieces stay in their type
// in between: occupancy.
template <typename T, int THREADS, int C>
__global__ __launch_bounds__(THREADS) void k_swiglu_i8(SwigluArgs a) {
  __shared__ uint32_t s_near[THREADS / 64], s_max[THREADS / 64];
  const int64_t row = blockIdx.x;
  const T* gp = (const T*)a.g + row * a.ldg;
  const T* up = (const T*)a.u + row * a.ldu;
  T g[C][kPiece], u[C][kPiece];
  float h[C][kPiece];
  uint32_t most[C];   // |h| of each piece; like h, set for pieces of the row
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_raw(gp, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, g[c]);
    load_raw(up, (c * THREADS + (int)threadIdx.x) * kPiece, a.n, u[c]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if ((c * THREADS + (int)threadIdx.x) * kPiece >= a.n) break;   // whole waves, but for one
    float far = 0.0f, low = 1.0f;
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      const float x = to_f(g[c][e]), t = x * -1.44269502f;
      const float rest = __builtin_fmaf(x, -1.92596303e-8f, __builtin_fmaf(x, -1.44269502f, -t));
      const float p = __builtin_amdgcn_exp2f(t), q = __builtin_fmaf(p, rest * 0.693147182f, p);
      const float s = x * __builtin_amdgcn_rcpf(1.0f + q);
      h[c][e] = s * to_f(u[c][e]);
      far = __builtin_fmaxf(far, t);
      low = __builtin_fminf(low, __builtin_fminf(__builtin_fabsf(s), __builtin_fabsf(h[c][e])));
    }
    AbsMax piece;
    piece.add(h[c]);
    most[c] = piece.bits();
    if (!(far <= 100.0f) || !(low >= 0x1p-100f) || most[c] >= 0x7E800000u) {
      AbsMax again;
#pragma unroll
      for (int e = 0; e < kPiece; ++e) h[c][e] = swiglu64(to_f(g[c][e]), to_f(u[c][e]));
      again.add(h[c]);
      most[c] = again.bits();
    }
    m = max(m, most[c]);
  }
  m = row_max<THREADS>(m, s_near);
  const bool finite = m < 0x7F800000u;
  const float near = __builtin_bit_cast(float, m) * (1.0f - 0x1p-18f);
  m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if ((c * THREADS + (int)threadIdx.x) * kPiece >= a.n) break;   // h and most are set up to here
    if (__builtin_bit_cast(float, most[c]) >= near) {
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        if (__builtin_fabsf(h[c][e]) >= near)
          m = max(m, __builtin_bit_cast(uint32_t, __builtin_fabsf(swiglu64(to_f(g[c][e]), to_f(u[c][e])))));
    }
  }
  m = row_max<THREADS>(m, s_max);
  const QScale s = q_scale(__builtin_bit_cast(float, m));
  const bool codes = finite && s.d != 0.0f;
  int8_t* q = a.q + row * a.ldq;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * THREADS + (int)threadIdx.x) * kPiece;
    if (i >= a.n) break;
    uint32_t v[2] = {0, 0};
    if (codes) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float y[4], worst = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float off;
          y[e] = to_code(h[c][4 * w + e], s.rd, off);
          worst = __builtin_fmaxf(worst, __builtin_fmaf(__builtin_fabsf(y[e] - kMagic), 0x1p-19f, off));
        }
        v[w] = low_bytes(y);
        if (!s.ok || !(worst < 0.5f - 0x1p-17f)) {
          v[w] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[w] |= ((uint32_t)code_of(swiglu64(to_f(g[c][4 * w + e]), to_f(u[c][4 * w + e])) / s.d) & 0xFFu) << (8 * e);
        }
      }
    }
    store_codes(q, i, a.n, v);
  }
  if (threadIdx.x == 0) a.scale[row] = finite ? s.d : __builtin_nanf("");
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

// A logit as the definition takes it: NaN as -infinity, at most the largest float32, no negative zero.
__device__ __forceinline__ float route_logit(float l) {
  return l != l ? -__builtin_inff() : __builtin_fminf(l, 3.40282347e38f) + 0.0f;
}

// Sorting keys: a 64-bit value whose last ten bits say which expert (0..1023), so that one maximum decides
// value and tie: the lower expert is the larger key. A float32 logit leaves those bits empty; a 64-bit
// score loses them, which the caller has to look after.
__device__ __forceinline__ double key_of(double v, int e) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (b & ~(uint64_t)1023) | (uint64_t)((int64_t)b < 0 ? e : 1023 - e));
}
__device__ __forceinline__ int expert_of(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  return (int64_t)b < 0 ? (int)(b & 1023) : 1023 - (int)(b & 1023);
}
__device__ __forceinline__ uint64_t class_of(double key) { return __builtin_bit_cast(uint64_t, key) >> 10; }

constexpr double kMaskedKey = -0x1p960;   // a masked expert of a kept group; every score is above (|c| <= 2^700)
constexpr double kMostScore = 0x1p700;

// Larger to a, smaller to b. The instructions themselves: the keys are never NaN, and the compiler's own
// maximum would quiet its operands first.
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ void exchange(double& a, double& b) {
  const double m = max64(a, b);
  b = min64(a, b);
  a = m;
}
// A bitonic list of N into descending order.
template <int N>
__device__ __forceinline__ void bitonic(double* v) {
  if constexpr (N > 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) exchange(v[i], v[i + N / 2]);
    bitonic<N / 2>(v);
    bitonic<N / 2>(v + N / 2);
  }
}
// Any N values into descending order: the halves, then the second backwards after the first.
template <int N>
__device__ __forceinline__ void sort_down(double* v) {
  if constexpr (N > 1) {
    sort_down<N / 2>(v);
    sort_down<N / 2>(v + N / 2);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) exchange(v[i], v[N - 1 - i]);
    bitonic<N / 2>(v);
    bitonic<N / 2>(v + N / 2);
  }
}
// The N largest of two descending lists, descending.
template <int N>
__device__ __forceinline__ void merge_top(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = max64(a[i], b[N - 1 - i]);
  bitonic<N>(a);
}

// The value of the lane's partner in step STEP of a butterfly: the neighbour, the other pair, the other quad,
// the other half of 16 lanes, the other 16 of 32, the other half.
template <int STEP>
__device__ __forceinline__ int partner(int v) {
  if constexpr (STEP < 4) return __builtin_amdgcn_update_dpp(0, v, STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140, 0xF, 0xF, false);
  else return __shfl_xor(v, STEP == 4 ? 16 : 32);
}
template <int STEP>
__device__ __forceinline__ float partner(float v) { return __builtin_bit_cast(float, partner<STEP>(__builtin_bit_cast(int, v))); }
template <int STEP>
__device__ __forceinline__ double partner(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)partner<STEP>((int)(uint32_t)b) |
                                        (uint64_t)(uint32_t)partner<STEP>((int)(uint32_t)(b >> 32)) << 32);
}
// f(step) for the steps that meet LANES lanes.
template <int LANES, typename F>
__device__ __forceinline__ void butterfly(F f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
  if constexpr (LANES == 64) {
    f(std::integral_constant<int, 4>{});
    f(std::integral_constant<int, 5>{});
  }
}

// LANES (16, four tokens a wave, or 64) lanes a token; a lane keeps up to V neighbouring experts in registers, a group
// (of 1, 2, 4, 8 or 16) in whole lanes, KL >= k. The lanes sort their keys, and four (six) steps merge the
// lists of KL: no step waits on a round of choosing. Without a bias the keys are exact (the logits). With
// one they hold 42 of a score's 52 bits: where two of the chosen, or the last of them and one left out,
// agree in those, the token is chosen again by whole scores, one expert at a time.
// Measured: 16384 tokens of 256 bfloat16 logits 10 us, by sigmoid scores with a bias in 8 groups 22 us (sixteen
// 64-bit scores a lane, about half of it), 512 tokens of those, 64 lanes each, 6.7 us. float32 scores with 64 bits
// where two are near: 23 us for the 16384, and 37 instead of 20 for 4096 x 512 (registers).
template <int V, int KL, int LANES>
__global__ __launch_bounds__(64) void k_route_lists(RouteArgs a, int T) {
  const int lane = threadIdx.x % LANES, E = a.E, per = E / a.n_groups, lanes = LANES / a.n_groups, share = (per + lanes - 1) / lanes;
  const int64_t tok = (int64_t)blockIdx.x * (64 / LANES) + threadIdx.x / LANES, t = tok < T ? tok : T - 1;
  const int group = lane / lanes, sub = lane % lanes, e0 = group * per + sub * share;
  const int count = max(0, min(share, per - sub * share));
  const bool softmax = a.score == MOE_SCORE_SOFTMAX, scored = a.bias || a.n_groups > 1;
  float l[V];
  {
    auto load = [&](auto type) {
      using Ty = decltype(type);
      const Ty* p = (const Ty*)a.logits + t * a.ld;
      constexpr int PIECE = V < 8 ? V : 8;
#pragma unroll
      for (int j0 = 0; j0 < V; j0 += PIECE) {
        if (e0 + j0 + PIECE <= E) {
          Ty v[PIECE];
          __builtin_memcpy(v, p + e0 + j0, sizeof v);
#pragma unroll
          for (int j = 0; j < PIECE; ++j) l[j0 + j] = to_f(v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < PIECE; ++j) l[j0 + j] = e0 + j0 + j < E ? to_f(p[e0 + j0 + j]) : 0.0f;
        }
      }
    };
    if (a.dtype == MOE_F32) load(float{});
    else if (a.dtype == MOE_BF16) load(bf16_t{});
    else load(f16_t{});
  }
  float peak = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    l[j] = route_logit(l[j]);
    if (j < count) peak = __builtin_fmaxf(peak, l[j]);
  }
  butterfly<LANES>([&](auto c) { peak = __builtin_fmaxf(peak, partner<c()>(peak)); });
  double total = 1.0;   // softmax's sum, where it does not cancel
  if (softmax && (scored || !a.renorm)) {
    // Each term (at most 1) in multiples of 2^-26 and a rest in multiples of 2^-60: 1024 of either add up without
    // rounding, so that the sum is the same however the experts lie in the lanes.
    double coarse = 0.0, fine = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < count && l[j] > -__builtin_inff()) {
        const double e = exp64((double)l[j] - (double)peak), big = (e + 0x1.8p26) - 0x1.8p26;
        coarse += big;
        fine += ((e - big) + 0x1.8p-8) - 0x1.8p-8;
      }
    butterfly<LANES>([&](auto c) { coarse += partner<c()>(coarse); });
    butterfly<LANES>([&](auto c) { fine += partner<c()>(fine); });
    total = coarse + fine;
    if (total == 0.0) total = 1.0;
  }
  const double part = inverse64(total);
  auto score = [&](float v) -> double {
    if (!(v > -__builtin_inff())) return 0.0;
    const double e = exp64(softmax ? (double)v - (double)peak : -__builtin_fmax((double)v, -1000.0));
    return softmax ? e * part : inverse64(1.0 + e);
  };
  auto biased = [&](int j) {   // c of the lane's expert j
    return __builtin_fmin(__builtin_fmax(score(l[j]) + (double)a.bias[e0 + j], -kMostScore), kMostScore);
  };
  const double none = -__builtin_inf();   // not to be chosen
  double key[V];
  bool kept = true;
  if (!scored) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      key[j] = j >= count ? none : key_of(l[j] > -__builtin_inff() ? (double)l[j] : kMaskedKey, e0 + j);
  } else {
    double b0 = none, b1 = none;   // the lane's, then the group's two largest
#pragma unroll
    for (int j = 0; j < V; ++j) {
      double c = none;
      if (j < count && l[j] > -__builtin_inff()) c = a.bias ? biased(j) : score(l[j]);
      b1 = max64(b1, min64(b0, c));
      b0 = max64(b0, c);
      const double v = c == none ? kMaskedKey : a.bias ? c + 0.0 : (double)l[j];
      key[j] = j >= count ? none : key_of(v, e0 + j);
    }
    if (a.n_groups > 1) {
      auto with = [&](auto c) {
        const double o0 = partner<c()>(b0), o1 = partner<c()>(b1);
        b1 = max64(min64(b0, o0), max64(b1, o1));
        b0 = max64(b0, o0);
      };
      butterfly<LANES>([&](auto c) {
        if (lanes >= 2 << c()) with(c);
      });
      const double gs = a.top == 2 && b1 > none ? b0 + b1 : b0;
      int ahead = 0;
      for (int g = 1; g < a.n_groups; ++g) {
        const int other = (lane + g * lanes) % LANES;
        const double o = __shfl(gs, (int)threadIdx.x - lane + other);
        ahead += o > gs || (o == gs && other / lanes < group);
      }
      kept = ahead < a.keep;
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = kept ? key[j] : none;
    }
  }
  double top[KL];
  {
    constexpr int N = V < KL ? V : KL;   // a list of KL from pieces of N
#pragma unroll
    for (int j0 = 0; j0 < V; j0 += N) {
      double piece[KL];
#pragma unroll
      for (int j = 0; j < KL; ++j) piece[j] = j < N ? key[j0 + j] : none;
      sort_down<N>(piece);
      if (j0 == 0) {
#pragma unroll
        for (int j = 0; j < KL; ++j) top[j] = piece[j];
      } else {
        merge_top<KL>(top, piece);
      }
    }
    butterfly<LANES>([&](auto c) {
      double other[KL];
#pragma unroll
      for (int j = 0; j < KL; ++j) other[j] = partner<c()>(top[j]);
      merge_top<KL>(top, other);
    });
  }
  double mine = top[0], last = top[0];
  bool again = false;
#pragma unroll
  for (int j = 1; j < KL; ++j) {
    if (lane == j) mine = top[j];
    if (a.bias && j < a.k) {
      again = again || (class_of(top[j]) == class_of(top[j - 1]) && top[j] > kMaskedKey / 2);
      last = top[j];
    }
  }
  int choice = expert_of(mine);
  if (a.bias) {
    const uint64_t b = __builtin_bit_cast(uint64_t, last);
    const double low = __builtin_bit_cast(double, (int64_t)b < 0 ? b | 1023 : b & ~(uint64_t)1023);
    int n = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) n += key[j] >= low;
    butterfly<LANES>([&](auto c) { n += partner<c()>(n); });
    again = again || (n > a.k && last > kMaskedKey / 2);
    if (__any(again)) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        key[j] = !kept || j >= count ? none : l[j] > -__builtin_inff() ? biased(j) : kMaskedKey;
#pragma unroll 1
      for (int r = 0; r < a.k; ++r) {
        double best = none;
        int at = 1 << 20;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (key[j] > best) best = key[j], at = e0 + j;
        butterfly<LANES>([&](auto c) {
          const double ob = partner<c()>(best);
          const int oa = partner<c()>(at);
          if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        });
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (e0 + j == at) key[j] = none;
        if (lane == r) choice = at;
      }
    }
  }
  double s = 0.0;
  if (lane < a.k) s = score(route_logit(load_f(a.logits, a.dtype, t * a.ld + choice)));
  double sum = 1.0;
  if (a.renorm) {
    sum = s;
    butterfly<LANES>([&](auto c) { sum += partner<c()>(sum); });
    if (sum == 0.0) sum = 1.0;
  }
  if (lane < a.k && tok < T) {
    a.ids[tok * a.k + lane] = choice;
    a.w[tok * a.k + lane] = (float)(s / sum * (double)a.factor);
  }
}

// Any number of groups, up to 1024 experts and 32 choices: one wave a token, its scores in LDS; expert e
// belongs to lane e % 64.
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
    const float l = route_logit(load_f(a.logits, a.dtype, t * a.ld + e));
    s_l[e] = l;
    peak = __builtin_fmaxf(peak, l);
  }
  for (int o = 32; o; o >>= 1) peak = __builtin_fmaxf(peak, __shfl_xor(peak, o));
  double total = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    for (int e = lane; e < E; e += 64)
      if (s_l[e] > -__builtin_inff()) total += exp64((double)s_l[e] - (double)peak);
    for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
  }
  auto score = [&](float l) -> double {
    if (!(l > -__builtin_inff())) return 0.0;
    return a.score == MOE_SCORE_SOFTMAX ? exp64((double)l - (double)peak) / total
                                        : 1.0 / (1.0 + exp64(-__builtin_fmax((double)l, -1000.0)));
  };
  for (int e = lane; e < E; e += 64) {
    const bool masked = !(s_l[e] > -__builtin_inff());
    double c = score(s_l[e]);
    if (a.bias) c = __builtin_fmin(__builtin_fmax(c + (double)a.bias[e], -kMostScore), kMostScore);
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
  int wide;             // rows of C take 16-byte accesses, and 16-bit ones are only written
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

// f(0), .., f(N - 1) with the numbers as types.
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// s_waitcnt vmcnt(n * PER), n at most MAX, uniform.
template <int PER, int MAX>
__device__ __forceinline__ void wait_loads(int n) {
  static_assert(PER * MAX < 64, "vmcnt");
  if constexpr (MAX == 0) __builtin_amdgcn_s_waitcnt(MOE_OPS_VM(0));
  else if (n >= MAX) __builtin_amdgcn_s_waitcnt(MOE_OPS_VM(PER * MAX));
  else wait_loads<PER, MAX - 1>(n);
}

// One workgroup a tile of BT tokens x BC channels, WT x WC waves. v_mfma_i32_16x16x64_i8 with the
// channels as rows and the tokens as columns, so that a lane ends with four neighbouring channels of
// one token. A stage in LDS holds BT + BC rows of BK bytes in 16-byte chunks, placed so that the eight
// rows that eight lanes read at one chunk sit in different banks. KG groups of WT x WC waves take
// neighbouring BK bytes of K each step and their sums meet at the end (small tiles: fewer, larger
// steps). DIRECT: rows and their stride are 16-byte aligned; a ring of S stages takes them straight to
// LDS, S - 1 steps ahead. Else through registers, S steps ahead, and two stages. A last piece of K below
// a step is taken first, through registers, zero past K.
// A step runs in groups of NT matrix instructions (one channel tile); beside each group go the fragment
// read that the group after next needs and a share of the step's loads, so that neither the LDS nor the
// memory pipe sees them all at once; the next step's first reads follow the barrier ahead of the last
// two groups. The loads go beside the first two groups of a long step: spread over four or eight the large
// tile took 2-7% more.
// C leaves in whole lines through LDS: straight from the lanes, in 32- or 64-byte parts of them, the largest
// product took 245 us and 8192 x 2560 x 768 42 us instead of 34.
// Measured (GPU time of a launch, inputs not in a cache): 8192 x 8192 x 4096 231 us (2380 TOPS; the matrix
// instruction alone, from registers, 4240), x 8192 426 us (2580). A step takes 1.5 us where its matrix
// instructions take 1.0 to 1.2, its loads 0.5 and its LDS reads 0.4: the barrier and the first reads after it
// stand between; zeros instead of random codes run 10% faster, so power counts too. The rest is each tile's
// first loads and C. 512 x 1536 x 2560 8.4 us, 64 x 5120 x 2560 9.5: a launch, a latency and few steps.
// Slower for the largest: a tile 64 bytes of K deep in four stages (each line of memory twice; 270-280 us where
// this took 250), four waves of 128 x 128 (285), workgroups that go on to further tiles while C is
// stored (259), touching the lines of the step after next (262 where this took 244).
template <int BT, int BC, int WT, int WC, int KG, int BK, bool DIRECT, int S>
__global__ __launch_bounds__(64 * WT * WC * KG) void k_matmul_tile(MatmulArgs p) {
  extern __shared__ __align__(16) uint8_t s_ring[];
  constexpr int W = WT * WC * KG, R = BT + BC, RP = 1024 / BK;   // RP: rows of a 1 KB piece, one load of a wave
  constexpr int L = KG * R / RP / W;                             // pieces a wave loads per step
  constexpr int NT = BT / WT / 16, NC = BC / WC / 16, KK = BK / 64, G = NC * KK;
  constexpr int LG = G >= 16 ? 2 : G - 2;   // groups beside which a step's loads go
  constexpr int STEP = KG * BK, STAGE = R * STEP, RING = DIRECT ? S : 2;
  static_assert((BK == 64 || BK == 128) && KG * R % (RP * W) == 0 && R % RP == 0 && BT % (16 * WT) == 0 &&
                BC % (16 * WC) == 0 && NC >= 2 && G % 4 == 0, "tile split");
  static_assert(RING * STAGE >= W / KG * NC * 1024 && RING * STAGE >= (KG - 1) * (W / KG) * NC * NT * 1024,
                "the epilogue's pieces fit");
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

  // place of a row's chunk: 128-byte rows c ^ (row & 7); 64-byte rows, two to 128 bytes, c ^ (row / 2 & 3)
  auto place = [](int r, int c) { return BK == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3); };
  // this lane's rows: piece q = wave + W i is rows RP (q % (R / RP)) .., tokens first, of K group q / (R / RP)
  const int chunk = place(lane / (BK / 16), lane % (BK / 16)) * 16;
  auto of_tokens = [&](int i) { return (wave + W * i) % (R / RP) < BT / RP; };   // else channels; the same in all lanes
  auto column = [&](int i) { return (wave + W * i) / (R / RP) * BK + chunk; };
  const int8_t *a0 = p.a + m0 * p.lda, *b0 = p.b + n0 * p.ldb;
  using Offset = std::conditional_t<DIRECT, int, int64_t>;   // DIRECT: the tile's rows lie within 2^31 bytes
  Offset off[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int r = RP * ((wave + W * i) % (R / RP)) + lane / (BK / 16);
    off[i] = (r < BT ? min(r, p.M - 1 - m0) * (Offset)p.lda : min(r - BT, p.N - 1 - n0) * (Offset)p.ldb) + column(i);
  }
  const int8_t* src[DIRECT ? 1 : L];
#pragma unroll
  for (int i = 0; i < L && !DIRECT; ++i) src[i] = (of_tokens(i) ? a0 : b0) + off[i];
  const int rem = p.K % STEP, steps = (p.K + STEP - 1) / STEP;
  const int wt = wave % WT, wc = wave / WT % WC, kg = wave / (WT * WC), row = lane & 15, quad = lane >> 4;
  i32x4 acc[NC][NT], av[4], bv[2][NT], hold[DIRECT ? 1 : S][L];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto put = [&](int slot, int i, const i32x4& v) {   // a piece from registers to LDS
    *(i32x4*)(s_ring + slot * STAGE + 1024 * (wave + W * i) + 16 * lane) = v;
  };
  // A piece of column k's step on its way to LDS. A buffer load, since the compiler takes a global load to
  // LDS for one that the LDS counter counts too, and would then wait for every read in flight at each use.
  const auto a_rows = __builtin_amdgcn_make_buffer_rsrc((void*)a0, 0, 0x7FFFFFFF, 0x00027000);
  const auto b_rows = __builtin_amdgcn_make_buffer_rsrc((void*)b0, 0, 0x7FFFFFFF, 0x00027000);
  auto send = [&](int slot, int i, int k) {
    MOE_LDS void* to = (MOE_LDS void*)(s_ring + slot * STAGE + 1024 * (wave + W * i));
    if (of_tokens(i)) __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rows, to, 16, (int)off[i], k, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(b_rows, to, 16, (int)off[i], k, 0, 0);
  };
  auto take = [&](int i, i32x4& v) {                  // the same to registers
    v = any16(src[i]);
    src[i] += STEP;
  };
  auto first = [&](int i) {                           // a piece of step 0 where K leaves one
    return row16((of_tokens(i) ? a0 : b0) + (off[i] - column(i)), p.K - rem + column(i), p.K);
  };
  // the fragments that group g of the step in `slot` starts with; par: which of bv the step's first is
  auto read = [&](int slot, auto par, int g) {
    const int kk = g / NC, i = g % NC;
    const uint8_t* st = s_ring + slot * STAGE + kg * R * BK + row * BK + place(row, 4 * kk + quad) * 16;
    if (i == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j) bv[(par() + kk) & 1][j] = *(const i32x4*)(st + (wt * NT + j) * 16 * BK);
    }
    av[g & 3] = *(const i32x4*)(st + (BT + (wc * NC + i) * 16) * BK);
  };
  // One step. Its first two groups' fragments are read; `next` is the slot of step t + 1, `back` where the
  // loads of step t + S - 1 go, h the registers that hold step t + 1's pieces. steady: the steps that the
  // loads are for exist, so nothing is asked.
  auto step = [&](int t, auto steady, int slot, int next, int back, auto par, i32x4 (&h)[L]) __attribute__((always_inline)) {
    const bool more = steady() || t + 1 < steps, ahead = steady() || t + (DIRECT ? S - 1 : 1) < steps;
    const bool later = steady() || t + 1 + S < steps;
    const int k_ahead = (t + S - 1) * STEP - (rem ? STEP : 0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g < G - 2) read(slot, par, g + 2);
      if (g == G - 2) {
        if constexpr (DIRECT) wait_loads<L, S - 2>(steady() ? S - 2 : more ? steps - 2 - t : 0);   // step t + 1 has landed
        ops_barrier();
      }
      if (g >= G - 2 && more) read(next, std::integral_constant<int, (par() + KK) & 1>{}, g + 2 - G);
      if (g < LG && ahead) {
#pragma unroll
        for (int i = g * L / LG; i < (g + 1) * L / LG; ++i) {
          if constexpr (DIRECT) {
            send(back, i, k_ahead);
          } else {
            put(next, i, h[i]);
            if (later) take(i, h[i]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[g % NC][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[g & 3], bv[(par() + g / NC) & 1][j], acc[g % NC][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // U steps hold whole rounds of stages, registers and parities
  constexpr int U = S % 2 && (KK == 1 || !DIRECT) ? 2 * S : S;
  auto round = [&](int t, auto steady, auto d) __attribute__((always_inline)) {
    constexpr int D = d();
    using Par = std::integral_constant<int, (D * KK) & 1>;
    if constexpr (DIRECT) step(t, steady, D % S, (D + 1) % S, (D + S - 1) % S, Par{}, hold[0]);
    else step(t, steady, D & 1, (D & 1) ^ 1, 0, Par{}, hold[(D + 1) % S]);
  };
  if constexpr (DIRECT) {
    i32x4 v[L];
    if (rem) {
#pragma unroll
      for (int i = 0; i < L; ++i) v[i] = first(i);
    }
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
      if (t < steps && !(t == 0 && rem)) {
#pragma unroll
        for (int i = 0; i < L; ++i) send(t, i, t * STEP - (rem ? STEP : 0));
      }
    if (rem) {
#pragma unroll
      for (int i = 0; i < L; ++i) put(0, i, v[i]);
    }
    wait_loads<L, S - 2>(steps - 1);
  } else {   // hold[t % S] takes step t's pieces, from step 1 on; step 0 goes to LDS at once
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if (rem) hold[0][i] = first(i);
      else take(i, hold[0][i]);
    }
#pragma unroll
    for (int i = 0; i < L; ++i) put(0, i, hold[0][i]);
#pragma unroll
    for (int t = 1; t <= S; ++t)
      if (t < steps) {
#pragma unroll
        for (int i = 0; i < L; ++i) take(i, hold[t % S][i]);
      }
  }
  ops_barrier();
  read(0, std::integral_constant<int, 0>{}, 0);
  read(0, std::integral_constant<int, 0>{}, 1);
  int t = 0;
  for (; t + U + S < steps; t += U)
    each<U>([&](auto d) __attribute__((always_inline)) { round(t + d(), std::true_type{}, d); });
  for (; t < steps; t += U)
    each<U>([&](auto d) __attribute__((always_inline)) {
      if (t + d() < steps) round(t + d(), std::false_type{}, d);
    });
  if constexpr (KG > 1) {
    i32x4* sums = (i32x4*)s_ring + (wave % (WT * WC)) * NC * NT * 64 + lane;
    constexpr int GROUP = WT * WC * NC * NT * 64;
    ops_barrier();
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[(kg - 1) * GROUP + (i * NT + j) * 64] = acc[i][j];
    }
    ops_barrier();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] += sums[g * GROUP + (i * NT + j) * 64];
  }
  // Scales first, all of them (the compiler cannot move a load across a store), then the tile in its type.
  const int m1 = m0 + wt * NT * 16, n1 = n0 + wc * NC * 16;
  const bool whole = p.vec && (n0 + BC <= p.N || p.N % 4 == 0);   // four channels are stored or none
  float sa[NT];
  f32x4 sb[NC];
#pragma unroll
  for (int j = 0; j < NT; ++j) sa[j] = p.sa[min(m1 + 16 * j + row, p.M - 1)];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int n = n1 + 16 * i + 4 * quad;
    if (whole) {
      sb[i] = *(const f32x4*)(p.sb + min(n, p.N - 4));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) sb[i][e] = p.sb[min(n + e, p.N - 1)];
    }
  }
  auto finish = [&](auto type) __attribute__((always_inline)) {
    using T = decltype(type);
    struct alignas(4 * sizeof(T)) T4 {
      T v[4];
    };
    // Wide rows of C go through the wave's piece of LDS into whole lines: HALVES parts of the channels, one
    // after the other, of CHUNKS 16-byte chunks a row for 16 tokens.
    constexpr int HALVES = sizeof(T) / 2, NP = NC / HALVES, CHUNKS = 2 * NC, PITCH = 16 * CHUNKS + 16, X = CHUNKS / 4;
    static_assert(RING * STAGE >= W / KG * 16 * PITCH, "the rows fit");
    if (p.wide) {
      ops_barrier();
      uint8_t* mine = s_ring + (wave % (WT * WC)) * 16 * PITCH;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            T4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o.v[e] = from_f<T>((float)acc[h * NP + i][j][e] * sa[j] * sb[h * NP + i][e]);
            *(T4*)(mine + row * PITCH + (16 * i + 4 * quad) * sizeof(T)) = o;
          }
          __builtin_amdgcn_wave_barrier();
          const int n = n1 + 16 * h * NP + 16 / (int)sizeof(T) * (lane % CHUNKS);   // 64 is a multiple of CHUNKS
          i32x4 v[X];
          i32x4* c[X];
          bool in[X];
#pragma unroll
          for (int x = 0; x < X; ++x) {
            const int r = (x * 64 + lane) / CHUNKS, m = m1 + 16 * j + r;
            in[x] = m < p.M && n < p.N;
            c[x] = (i32x4*)((T*)p.c + m * p.ldc + n);
            v[x] = *(const i32x4*)(mine + r * PITCH + 16 * (lane % CHUNKS));
          }
          if (sizeof(T) == 4 && p.accumulate) {
#pragma unroll
            for (int x = 0; x < X; ++x)
              if (in[x]) v[x] = __builtin_bit_cast(i32x4, __builtin_bit_cast(f32x4, v[x]) + *(const f32x4*)c[x]);
          }
#pragma unroll
          for (int x = 0; x < X; ++x)
            if (in[x]) *c[x] = v[x];
          __builtin_amdgcn_wave_barrier();
        }
    } else if (whole) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = m1 + 16 * j + row;
        if (m >= p.M) break;
        T* c = (T*)p.c + m * p.ldc + n1 + 4 * quad;
        T4 old[NC];
        if (p.accumulate) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (n1 + 16 * i + 4 * quad < p.N) old[i] = *(const T4*)(c + 16 * i);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (n1 + 16 * i + 4 * quad >= p.N) break;
          T4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = (float)acc[i][j][e] * sa[j] * sb[i][e];
            if (p.accumulate) v += to_f(old[i].v[e]);
            o.v[e] = from_f<T>(v);
          }
          *(T4*)(c + 16 * i) = o;
        }
      }
    } else {   // ragged or unaligned: through the wave's piece of LDS, so that lanes write along a row
      ops_barrier();
      constexpr int U4 = 4 * NC, PER = 4 * NC;   // four-value units of a row; values a lane stores for 16 tokens
      float* mine = (float*)(s_ring + (wave % (WT * WC)) * NC * 1024);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * sa[j] * sb[i][e];
          *(f32x4*)(mine + 4 * (row * U4 + ((4 * i + quad) ^ (row & (U4 - 1))))) = v;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int x0 = 0; x0 < PER; x0 += 8) {
          float v[8];
          T* c[8];
          bool in[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int at = (x0 + x) * 64 + lane, r = at / (4 * U4), col = at % (4 * U4);
            const int m = m1 + 16 * j + r, n = n1 + col;
            in[x] = m < p.M && n < p.N;
            c[x] = (T*)p.c + m * p.ldc + n;
            v[x] = mine[4 * (r * U4 + ((col / 4) ^ (r & (U4 - 1)))) + col % 4];
          }
          if (p.accumulate) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (in[x]) v[x] += to_f(*c[x]);
          }
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (in[x]) *c[x] = from_f<T>(v[x]);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  };
  if (p.c_dtype == MOE_F32) finish(float{});
  else if (p.c_dtype == MOE_BF16) finish(bf16_t{});
  else finish(f16_t{});
}

// Few tokens (M <= 16 MT, MT 1 or 2): the weights are read once, straight into the lanes of the matrix
// instruction, and a workgroup's W waves share out K, so that each has few dependent loads. C = 16 / P
// channels a workgroup: with P > 1 (M <= C) the instruction's 16 rows are C channels at P neighbouring
// pieces of K and its 16 columns the tokens at the same pieces; the blocks of its result where the
// two pieces agree are partial sums of the product. Few channels then still fill the chip. Bound by the
// launch (1 x 1536 x 2560: 3.5 us) or the weights' bytes (1 x 8192 x 8192: 16.5 us, 4.1 TB/s); 16 tokens of
// 1536 x 2560 4.7 us.
template <int MT, int P, int W>
__global__ __launch_bounds__(64 * W) void k_matmul_thin(MatmulArgs p) {
  constexpr int C = 16 / P, PIECE = 128 * P, STRIDE = PIECE * W, UN = 4;
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

// A row call's type and workgroup: by the row length alone, so that a row's sums have one order. Two pieces a
// thread above 2048 values, one below. us for 8192 bf16 rows, norm / SwiGLU: 512 wide 64 x 1 11.7 / 9.5, 128 x 1
// 13.0 / 11.2; 1024 wide 128 x 1 18.0 / 14.6, 64 x 2 18.4 / 15.7; 2048 wide 256 x 1 28.9 / 22.5, 128 x 2 30.4 /
// 24.6; 2560 wide 256 x 2 40.3 / 32.9, 512 x 1 44.6 / 33.8; 4096 wide 52.1 / 41.1, 512 x 1 54.1 / 41.3; 5120
// wide, norm 512 x 2 69.6, 1024 x 1 78.6. One float32 row of 2560 has it the other way: 3.5, 512 x 1 3.2.
template <typename F>
void with_row(int dtype, int n, F f) {
  auto size = [&](auto t) {
    using std::integral_constant;
    if (n <= 64 * kPiece) f(t, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (n <= 128 * kPiece) f(t, integral_constant<int, 128>{}, integral_constant<int, 1>{});
    else if (n <= 256 * kPiece) f(t, integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (n <= 512 * kPiece) f(t, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (n <= 1024 * kPiece) f(t, integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else f(t, integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  };
  with_type(dtype, size);
}
static_assert(1024 * 2 * kPiece == MOE_MAX_ROW, "the longest row fits one workgroup");

// A tile's cost is its time over K (the one measured: K = 2560, one round of up to 256 tiles, us) times
// the rounds that 256 CUs need. Small tiles bring the chip's CUs to a small product (512 x 1536: 64 x 64
// 8.2 us, 128 x 128 14.2, 256 x 256 34), large ones read less for each product of a large one (8192 x
// 1536: 256 x 256 51 us, 64 x 64 72). Rounds count one workgroup a CU, though the three small tiles leave room for
// two. The largest tile takes the fewest threads for any product.
struct Tile {
  int bt, bc, threads;
  double us;
};
constexpr Tile kTiles[] = {{32, 32, 256, 5.6}, {64, 32, 512, 6.9}, {64, 64, 256, 8.2}, {128, 64, 512, 13.5},
                           {128, 128, 512, 18.8}, {256, 128, 512, 25.8}, {256, 256, 512, 41}};
int64_t tiles_of(const Tile& t, int M, int N) {
  return (((int64_t)M + t.bt - 1) / t.bt) * (((int64_t)N + t.bc - 1) / t.bc);
}
// The tile of least cost among those whose launch is possible; -1: none.
int choose_tile(int M, int N) {
  int best = -1;
  double least = 0;
  for (int i = 0; i < 7; ++i) {
    const int64_t n = tiles_of(kTiles[i], M, N);
    if (n * kTiles[i].threads > kLaunchThreads) continue;
    const double cost = kTiles[i].us * (double)((n + 255) / 256);
    if (best < 0 || cost < least) best = i, least = cost;
  }
  return best;
}

template <int I, int WT, int WC, int KG, int BK, int S, int BK_HELD, int S_HELD>
int launch_tile(hipStream_t st, MatmulArgs p, bool direct) {
  constexpr int BT = kTiles[I].bt, BC = kTiles[I].bc, THREADS = kTiles[I].threads;
  static_assert(THREADS == 64 * WT * WC * KG, "the table's threads are the kernel's");
  p.tiles_n = (int)(((int64_t)p.N + BC - 1) / BC);
  p.tiles = (int)tiles_of(kTiles[I], p.M, p.N);
  auto go = [&](auto kern, int lds) {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return hip_fail(e, "moe_matmul_i8");
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)p.tiles), dim3(THREADS), lds, st, p);
    return launched("moe_matmul_i8");
  };
  return direct ? go(k_matmul_tile<BT, BC, WT, WC, KG, BK, true, S>, S * (BT + BC) * KG * BK)
                : go(k_matmul_tile<BT, BC, WT, WC, KG, BK_HELD, false, S_HELD>, 2 * (BT + BC) * KG * BK_HELD);
}

int run_matmul(hipStream_t st, MatmulArgs p) {
  const bool direct = aligned(p.a, 16) && aligned(p.b, 16) && p.lda % 16 == 0 && p.ldb % 16 == 0 &&
                      std::max(p.lda, p.ldb) < (1 << 22);   // 256 rows and K within 2^31 bytes
  const int in16 = 16 / type_size(p.c_dtype);   // values of 16 bytes
  p.wide = (in16 == 4 || !p.accumulate) && aligned(p.sb, 16) && aligned(p.c, 16) && p.ldc % in16 == 0 && p.N % in16 == 0;
  p.vec = aligned(p.sb, 16) && aligned(p.c, 4 * type_size(p.c_dtype)) && p.ldc % 4 == 0;
  // Up to 16 tokens: 16 x 1536, K = 2560 4.7 us, and 5.7 in tiles; 16 x 2560, 768 3.3 and 4.4; 16 x 7936, 2560 8.2
  // and 7.8; 16 x 8448, 2560 10.1 and 10.4. Up to 32 where K is short: 32 x 2560, 768 3.6 and 4.4; 32 x 5120, 768 4.7
  // and 4.4; 32 x 4352, 2560 10.0 and 7.1.
  const bool launches = p.N <= kLaunchThreads / 512 * 16;   // 512 threads for 16 channels
  if (p.M <= 16 || (p.M <= 32 && p.K <= 1024 && launches)) {
    if (!launches) return MOE_E_SHAPE;
    auto go = [&](auto kern, int channels, int threads) {
      hipLaunchKernelGGL(kern, dim3((unsigned)(((int64_t)p.N + channels - 1) / channels)), dim3(threads), 0, st, p);
      return launched("moe_matmul_i8");
    };
    // Pieces of K side by side: more, and fewer channels a workgroup, where K is long and 256 CUs are not filled.
    // us by 1, 2 and 4 pieces (M x N, K): 1 x 1024, 8192 6.8 4.8 4.1; 1 x 1024, 1280 3.1 2.9 3.4; 1 x 1536, 2560 3.8
    // 3.5 3.7; 8 x 1536, 2560 4.3 3.8 -; 1 x 2560, 768 3.0 3.2 3.9; 4 x 2560, 2560 4.1 4.5 4.6; 1 x 2560, 8192 8.6
    // 8.2 7.4; 1 x 5120, 8192 14.2 11.1 10.9; 8 x 5120, 4096 9.6 8.6 -; 1 x 7936, 1024 3.9 4.1 6.2; 1 x 8448, 2560
    // 7.8 - 9.2.
    int pieces = 1;
    if (p.M <= 8 && p.K >= 1024) {
      if (p.N <= 2048) pieces = p.M <= 4 && p.N <= 1024 && p.K >= 2048 ? 4 : 2;
      else if (p.N < 4096) pieces = p.K < 4096 ? 1 : p.M <= 4 ? 4 : 2;
      else if (p.N < 8192) pieces = 2;
    }
    if (pieces == 4) return go(k_matmul_thin<1, 4, 8>, 4, 512);
    if (pieces == 2) return go(k_matmul_thin<1, 2, 8>, 8, 512);
    if (p.M <= 16) return go(k_matmul_thin<1, 1, 8>, 16, 512);
    return go(k_matmul_thin<2, 1, 8>, 16, 512);
  }
  switch (choose_tile(p.M, p.N)) {
    case 0: return launch_tile<0, 2, 1, 2, 128, 4, 128, 2>(st, p, direct);
    case 1: return launch_tile<1, 4, 1, 2, 128, 3, 128, 2>(st, p, direct);
    case 2: return launch_tile<2, 2, 2, 1, 128, 4, 128, 2>(st, p, direct);
    case 3: return launch_tile<3, 4, 2, 1, 128, 4, 128, 1>(st, p, direct);
    case 4: return launch_tile<4, 4, 2, 1, 128, 4, 128, 2>(st, p, direct);
    case 5: return launch_tile<5, 4, 2, 1, 128, 3, 128, 2>(st, p, direct);
    case 6: return launch_tile<6, 4, 2, 1, 128, 2, 64, 1>(st, p, direct);
    default: return MOE_E_SHAPE;
  }
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
  if (n < 1 || n > MOE_MAX_ROW || (q8_1 && n % 32) || rows > MOE_MAX_ROWS) return MOE_E_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !weight || !q != !scale || (!res_out && !yout && !q && !q8_1)) return MOE_E_ARG;
  if (bad_stride(ldx, n, rows) || (res && bad_stride(ldres, n, rows)) || (res_out && bad_stride(ldro, n, rows)) ||
      (yout && bad_stride(ldy, n, rows)) || (q && bad_stride(ldq, n, rows)))
    return MOE_E_ARG;
  const int sz = type_size(dtype), szy = type_size(y_dtype);
  if (!aligned(x, sz) || !aligned(res, sz) || !aligned(res_out, sz) || !aligned(weight, type_size(w_dtype)) ||
      (yout && !aligned(yout, szy)) || !aligned(scale, 4) || !aligned(q8_1, 4))
    return MOE_E_ARG;
  const int64_t nb8 = (int64_t)n / 32 * 36;
  const Rows in[] = {rows_of(x, rows, n, ldx, sz), rows_of(res, rows, n, ldres, sz),
                     rows_of(weight, 1, n, n, type_size(w_dtype))};
  const Rows out[] = {rows_of(res_out, rows, n, ldro, sz), rows_of(yout, rows, n, ldy, szy), rows_of(q, rows, n, ldq, 1),
                      rows_of(scale, 1, rows, rows, 4), rows_of(q8_1, rows, nb8, nb8, 1)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j)   // r over x or res: the very same rows
      if (!(i == 0 && j < 2 && in[j].p == out[0].p && in[j].step == out[0].step) && overlap(out[i], in[j])) return MOE_E_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MOE_E_ARG;
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
  if ((renorm != 0 && renorm != 1) || !(__builtin_fabsf(factor) < __builtin_inff()) || ld < E) return MOE_E_ARG;
  if (T > MOE_MAX_ROWS) return MOE_E_SHAPE;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !w || bad_stride(ld, E, T) || !aligned(logits, type_size(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(w, 4))
    return MOE_E_ARG;
  const Rows out[] = {rows_of(ids, T, k, k, 4), rows_of(w, T, k, k, 4)};
  const Rows in[] = {rows_of(logits, T, E, ld, type_size(dtype)), rows_of(bias, 1, E, E, 4)};
  if (overlap(out[0], out[1])) return MOE_E_ARG;
  for (const Rows& r : in)
    if (overlap(out[0], r) || overlap(out[1], r)) return MOE_E_ARG;
  const RouteArgs a{logits, bias, ids, w, ld, dtype, E, k, score, n_groups, keep_groups, group_top, renorm, factor};
  // Lists in registers where a group is whole lanes and a lane's share is up to 32 experts (16384 x 256: 10 us
  // by logits, 22 by scores in groups; 118 and 124 by one wave a token). The least V and KL that hold the share and
  // k: 16384 tokens of 64 / 128 / 256 experts 6.7 / 7.6 / 10.2 us, with the next V 7.6 / 9.1 / 14.1, with KL 16 for k = 8
  // 9.1 / 10.2 / 12.8.
  // Few tokens of scored experts take 64 lanes each, which spread the scores' 64-bit arithmetic (the bits are the
  // same: softmax's sum does not round): 512 x 256 10.4 -> 6.7 us, 2048 x 256 11.0 -> 8.1, 4096 x 256 11.6 -> 11.5;
  // 1024 x 128 6.6 -> 5.9, 4096 x 128 7.3 -> 9.5; 512 x 64 5.0 -> 5.3.
  const bool whole = n_groups <= 16 && 16 % n_groups == 0;
  auto shares = [&](int lanes) { return whole ? (per + lanes / n_groups - 1) / (lanes / n_groups) : kRouteE; };
  const bool wide = (bias || n_groups > 1) && shares(16) > 4 && T <= (shares(16) > 8 ? 2048 : 1024) && shares(64) <= 8;
  const int share = shares(wide ? 64 : 16);
  auto go = [&](auto kern, int tokens) {
    hipLaunchKernelGGL(kern, dim3((unsigned)(((int64_t)T + tokens - 1) / tokens)), dim3(64), 0, (hipStream_t)stream, a, T);
  };
  if (share > 32 || k > 16)
    hipLaunchKernelGGL(k_route_scores, dim3(T), dim3(64), 0, (hipStream_t)stream, a);
  else if (wide && k <= 8)
    share <= 4 ? go(k_route_lists<4, 8, 64>, 1) : go(k_route_lists<8, 8, 64>, 1);
  else if (wide)
    share <= 4 ? go(k_route_lists<4, 16, 64>, 1) : go(k_route_lists<8, 16, 64>, 1);
  else if (k <= 8)
    share <= 4 ? go(k_route_lists<4, 8, 16>, 4) : share <= 8 ? go(k_route_lists<8, 8, 16>, 4)
    : share <= 16 ? go(k_route_lists<16, 8, 16>, 4) : go(k_route_lists<32, 8, 16>, 4);
  else
    share <= 4 ? go(k_route_lists<4, 16, 16>, 4) : share <= 8 ? go(k_route_lists<8, 16, 16>, 4)
    : share <= 16 ? go(k_route_lists<16, 16, 16>, 4) : go(k_route_lists<32, 16, 16>, 4);
  return launched("moe_route_scores");
}

int moe_swiglu_i8(void* stream, int dtype, const void* g, int64_t ldg, const void* u, int64_t ldu, int rows, int n,
                  int8_t* q, int64_t ldq, float* scale) {
  if (!type_ok(dtype) || rows < 0) return MOE_E_ARG;
  if (n < 1 || n > MOE_MAX_ROW || rows > MOE_MAX_ROWS) return MOE_E_SHAPE;
  if (rows == 0) return MOE_OK;
  const int sz = type_size(dtype);
  if (!g || !u || !q || !scale || bad_stride(ldg, n, rows) || bad_stride(ldu, n, rows) || bad_stride(ldq, n, rows))
    return MOE_E_ARG;
  if (!aligned(g, sz) || !aligned(u, sz) || !aligned(scale, 4)) return MOE_E_ARG;
  const Rows out[] = {rows_of(q, rows, n, ldq, 1), rows_of(scale, 1, rows, rows, 4)};
  for (const Rows& o : out)
    if (overlap(o, rows_of(g, rows, n, ldg, sz)) || overlap(o, rows_of(u, rows, n, ldu, sz))) return MOE_E_ARG;
  if (overlap(out[0], out[1])) return MOE_E_ARG;
  const SwigluArgs a{g, u, q, scale, ldg, ldu, ldq, n};
  with_row(dtype, n, [&](auto t, auto threads, auto pieces) {
    hipLaunchKernelGGL((k_swiglu_i8<decltype(t), threads(), pieces()>), dim3(rows), dim3(threads()), 0, (hipStream_t)stream, a);
  });
  return launched("moe_swiglu_i8");
}

int moe_matmul_i8(void* stream, const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb,
                  const float* sb, int M, int N, int K, int c_dtype, void* C, int64_t ldc, int accumulate) {
  if (!type_ok(c_dtype) || M < 0 || N < 0 || (accumulate != 0 && accumulate != 1)) return MOE_E_ARG;
  if (K < 1 || K > MOE_MAX_MATMUL_K || std::max(M, N) > MOE_MAX_MATMUL_MN) return MOE_E_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  if (!a || !sa || !b || !sb || !C || bad_stride(lda, K, M) || bad_stride(ldb, K, N) || bad_stride(ldc, N, M))
    return MOE_E_ARG;
  if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(C, type_size(c_dtype))) return MOE_E_ARG;
  const Rows c = rows_of(C, M, N, ldc, type_size(c_dtype));
  if (overlap(c, rows_of(a, M, K, lda, 1)) || overlap(c, rows_of(b, N, K, ldb, 1)) || overlap(c, rows_of(sa, 1, M, M, 4)) ||
      overlap(c, rows_of(sb, 1, N, N, 4)))
    return MOE_E_ARG;
  return run_matmul((hipStream_t)stream, MatmulArgs{a, b, sa, sb, C, lda, ldb, ldc, M, N, K, accumulate, 0, 0, 0, 0, c_dtype});
}

}  // extern "C"
