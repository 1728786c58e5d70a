// Operators around the routed layer for MI355X (gfx950): RMS norm with the residual's addition and
// outputs in 8 bits, the general router, SwiGLU into int8 rows, and the int8 matrix product with
// scales per token and channel. Formulas and edge rules: include/moe_route.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// ------------------------------------------------------------------ workgroup sums ----------

constexpr int kRowThreads = 256;

__device__ __forceinline__ double block_sum(double v, double* red) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kRowThreads / 64; ++w) v += red[w];
  __syncthreads();
  return v;
}
// The largest |y| of the row as its bits: they order like the values, infinities and NaNs above all.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kRowThreads / 64; ++w) v = max(v, red[w]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ uint32_t abs_bits(float y) { return __builtin_bit_cast(uint32_t, y) & 0x7FFFFFFFu; }

// int8 row of the float32 values in LDS.
__device__ __forceinline__ void write_i8_row(const float* y, int n, int8_t* q, float* scale, uint32_t* red) {
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += kRowThreads) m = max(m, abs_bits(y[i]));
  m = block_max(m, red);
  const bool finite = m < 0x7F800000u;
  const QScale s = q_scale(__builtin_bit_cast(float, m));
  for (int i = threadIdx.x; i < n; i += kRowThreads)
    q[i] = finite && s.d != 0.0f ? (int8_t)quant_code(y[i], s) : (int8_t)0;
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

// One workgroup a row, the row in LDS.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void k_add_rmsnorm(NormArgs a) {
  extern __shared__ float s_row[];
  __shared__ double s_red[kRowThreads / 64];
  __shared__ uint32_t s_redu[kRowThreads / 64];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* res = a.res ? (const T*)a.res + row * a.ldres : nullptr;
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.n; i += kRowThreads) {
    T r = x[i];
    if (res) r = from_f<T>(to_f(r) + to_f(res[i]));
    if (a.res_out) ((T*)a.res_out)[row * a.ldro + i] = r;
    const double d = (double)to_f(r);
    s_row[i] = to_f(r);
    sum += d * d;
  }
  sum = block_sum(sum, s_red);
  const double rinv = 1.0 / __builtin_sqrt(sum / a.n + (double)a.eps);
  for (int i = threadIdx.x; i < a.n; i += kRowThreads) {
    const float y = (float)((double)s_row[i] * rinv * (double)load_f(a.weight, a.w_dtype, i));
    s_row[i] = y;
    if (a.y) store_f(a.y, a.y_dtype, row * a.ldy + i, y);
  }
  __syncthreads();
  if (a.q) write_i8_row(s_row, a.n, a.q + row * a.ldq, a.scale + row, s_redu);
  if (a.q8_1) {
    const int nb = a.n / 32;
    for (int b = threadIdx.x; b < nb; b += kRowThreads) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = s_row[32 * b + i];
      const QBlock qb = quant_block(v);
      uint32_t* o = (uint32_t*)((uint8_t*)a.q8_1 + 36 * (row * nb + b));
      o[0] = qb.d16 | (qb.s16 << 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[1 + i] = qb.q[i];
    }
  }
}

// ------------------------------------------------------------------ SwiGLU ------------------

struct SwigluArgs {
  const void *g, *u;
  int8_t* q;
  float* scale;
  int64_t ldg, ldu, ldq;
  int n;
};

template <typename T>
__global__ __launch_bounds__(kRowThreads) void k_swiglu_i8(SwigluArgs a) {
  extern __shared__ float s_row[];
  __shared__ uint32_t s_redu[kRowThreads / 64];
  const int64_t row = blockIdx.x;
  const T* g = (const T*)a.g + row * a.ldg;
  const T* u = (const T*)a.u + row * a.ldu;
  for (int i = threadIdx.x; i < a.n; i += kRowThreads) {
    const double gd = (double)to_f(g[i]);
    s_row[i] = (float)(gd / (1.0 + exp(-gd)) * (double)to_f(u[i]));
  }
  __syncthreads();
  write_i8_row(s_row, a.n, a.q + row * a.ldq, a.scale + row, s_redu);
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

// ------------------------------------------------------------------ host checks -------------

bool aligned(const void* p, int size) { return ((uintptr_t)p & (uintptr_t)(size - 1)) == 0; }

// Whether two sets of rows share a byte (their whole spans, padding included).
bool overlap(const void* p, int64_t ldp, int sp, const void* q, int64_t ldq, int sq, int rows, int n) {
  if (!p || !q) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const uintptr_t na = (uintptr_t)(((rows - 1) * ldp + n) * sp), nb = (uintptr_t)(((rows - 1) * ldq + n) * sq);
  return a < b + nb && b < a + na;
}

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
  with_type(dtype, [&](auto t) {
    hipLaunchKernelGGL(k_add_rmsnorm<decltype(t)>, dim3(rows), dim3(kRowThreads), n * 4, (hipStream_t)stream, a);
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
  with_type(dtype, [&](auto t) {
    hipLaunchKernelGGL(k_swiglu_i8<decltype(t)>, dim3(rows), dim3(kRowThreads), n * 4, (hipStream_t)stream, a);
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
