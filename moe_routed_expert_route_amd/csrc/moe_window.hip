// The attention half beside the routed layer for MI355X (gfx950), for windows of tokens of many sequences: norm and
// rotation of queries and keys with the append to a paged cache, attention of the window's tree over that cache, and log
// probabilities of the answers. Formulas and edge rules: include/moe_route.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_rows.hpp"

namespace moe {

// ------------------------------------------------------------------ cache and window --------

__device__ __forceinline__ float to_f(int8_t x) { return (float)x; }

struct CacheArgs {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t page, head, slot;   // strides in elements
  int n_pages, page_size, n_kv, d;
};
struct WindowArgs {
  const int32_t *row_start, *ctx_len, *pages, *pos;
  const uint64_t* seen;
  uint32_t* err;
  int64_t ld_pages;
  int n_seqs, n_tokens, max_window, max_keys;   // max_keys: slots that a sequence's pages have
};

struct Seq {
  int s, start, tokens, ctx;
};
// Whether a sequence's rows and keys are where they may be.
__device__ __forceinline__ bool seq_ok(const WindowArgs& w, int start, int end, int ctx, int most) {
  return start >= 0 && start <= end && end <= w.n_tokens && end - start <= most && ctx >= 0 && ctx <= w.max_keys - (end - start);
}
// The sequence that a row is of; tokens = 0: none, or one that is left out. Uniform over the wave: a lane looks at one sequence
// in 64, all it needs at once. The first entry past the row ends the only sequence that can have it: where the list
// ascends, that is its sequence; where it goes back, a sequence that starts below an earlier entry is left out.
__device__ __forceinline__ Seq seq_of(const WindowArgs& w, int row, int most) {
  const int lane = threadIdx.x & 63;
  int largest = (int)0x80000000;   // of the starts before, this lane's
  for (int i = 0; i < w.n_seqs; i += 64) {
    const int at = min(i + lane, w.n_seqs - 1);
    const int start = w.row_start[at], end = w.row_start[at + 1], ctx = w.ctx_len[at];
    const uint64_t past = __ballot(end > row);
    if (past != 0) {
      const int n = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(start, n), last = __builtin_amdgcn_readlane(end, n);
      const int before = __builtin_amdgcn_readlane(ctx, n);
      if (lane < n) largest = max(largest, start);
      if (first > row || __ballot(largest > first) || !seq_ok(w, first, last, before, most)) break;
      return Seq{i + n, first, last - first, before};
    }
    largest = max(largest, start);
  }
  return Seq{0, 0, 0, 0};
}
// One workgroup of a launch looks at every sequence (a list that goes back has a sequence whose end is below its start).
__device__ __forceinline__ void check_seqs(const WindowArgs& w, int most, int threads) {
  for (int i = threadIdx.x; i < w.n_seqs; i += threads)
    if (!seq_ok(w, w.row_start[i], w.row_start[i + 1], w.ctx_len[i], most)) atomicOr(w.err, MOE_ERR_WINDOW);
}

// ------------------------------------------------------------------ append ------------------

struct AppendArgs {
  CacheArgs c;
  WindowArgs w;
  const void *q, *k, *v, *q_weight, *k_weight;
  const float* freq;
  void* q_out;
  int64_t ldq, ldk, ldv, ldo;
  int n_heads, n_rot, layout, w_dtype, o_dtype, c_dtype, units;
  float eps;
  double amp;   // as given: rounded to float32 it would move one value in thousands to the next code
};

// cos and sin of a (|a| < 2^40; else NaN): a = n pi / 2 + r, |r| <= pi / 4, and the power series to r^17 and
// r^18 (the next terms are below 2^-60).
__device__ __forceinline__ void turn64(double a, double& c, double& s) {
  const double n = __builtin_rint(a * 0.6366197723675814);
  const double r = __builtin_fma(-n, 6.123233995736766e-17, __builtin_fma(-n, 1.5707963267948966, a)), r2 = r * r;
  double p = 1.0 / 355687428096000.0;
  p = __builtin_fma(-p, r2, 1.0 / 1307674368000.0);
  p = __builtin_fma(-p, r2, 1.0 / 6227020800.0);
  p = __builtin_fma(-p, r2, 1.0 / 39916800.0);
  p = __builtin_fma(-p, r2, 1.0 / 362880.0);
  p = __builtin_fma(-p, r2, 1.0 / 5040.0);
  p = __builtin_fma(-p, r2, 1.0 / 120.0);
  p = __builtin_fma(-p, r2, 1.0 / 6.0);
  const double sr = __builtin_fma(-p * r2, r, r);
  double q = 1.0 / 6402373705728000.0;
  q = __builtin_fma(-q, r2, 1.0 / 20922789888000.0);
  q = __builtin_fma(-q, r2, 1.0 / 87178291200.0);
  q = __builtin_fma(-q, r2, 1.0 / 479001600.0);
  q = __builtin_fma(-q, r2, 1.0 / 3628800.0);
  q = __builtin_fma(-q, r2, 1.0 / 40320.0);
  q = __builtin_fma(-q, r2, 1.0 / 720.0);
  q = __builtin_fma(-q, r2, 1.0 / 24.0);
  q = __builtin_fma(-q, r2, 0.5);
  const double cr = __builtin_fma(-q, r2, 1.0);
  const int turn = (int)(n - 4.0 * __builtin_floor(n * 0.25));
  c = turn & 1 ? sr : cr;
  s = turn & 1 ? cr : sr;
  if (turn == 1 || turn == 2) c = -c;
  if (turn >= 2) s = -s;
  if (!(__builtin_fabs(a) < 0x1p40)) c = s = __builtin_nan("");
}

template <typename F>
__device__ __forceinline__ void on_type(int dtype, F f) {
  dtype == MOE_F32 ? f(float{}) : dtype == MOE_BF16 ? f(bf16_t{}) : f(f16_t{});
}

// Four neighbouring values, `n` of them there (the others 0).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, T (&v)[4]) {
  if (n >= 4) {
    __builtin_memcpy(v, p, sizeof v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = T{};
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) v[e] = p[e];
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int n, const float* y) {
  T v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = from_f<T>(y[e]);
  if (n >= 4) {
    __builtin_memcpy(p, v, sizeof v);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void load4(const void* p, int dtype, int at, int n, float* f) {
  on_type(dtype, [&](auto t) {
    decltype(t) v[4];
    load4((const decltype(t)*)p + at, n, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = to_f(v[e]);
  });
}

// Sum and maximum over LG neighbouring lanes, in all of them: halves of 8 mirrored, rows of 16 turned round, then the
// neighbouring rows.
template <int LG>
__device__ __forceinline__ double lanes_sum(double v) {
  if constexpr (LG == 8) {
    v += dpp0<0x141, 0xF>(v);
    v += dpp0<0x4E, 0xF>(v);
    v += dpp0<0xB1, 0xF>(v);
  } else {
    v += dpp0<0x128, 0xF>(v);
    v += dpp0<0x124, 0xF>(v);
    v += dpp0<0x122, 0xF>(v);
    v += dpp0<0x121, 0xF>(v);
  }
  if constexpr (LG >= 32) v += __shfl_xor(v, 16);
  if constexpr (LG >= 64) v += __shfl_xor(v, 32);
  return v;
}
template <int LG>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LG == 8) {
    v = max(v, dpp0<0x141, 0xF>(v));
    v = max(v, dpp0<0x4E, 0xF>(v));
    v = max(v, dpp0<0xB1, 0xF>(v));
  } else {
    v = max(v, dpp0<0x128, 0xF>(v));
    v = max(v, dpp0<0x124, 0xF>(v));
    v = max(v, dpp0<0x122, 0xF>(v));
    v = max(v, dpp0<0x121, 0xF>(v));
  }
  if constexpr (LG >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  if constexpr (LG >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
  return v;
}
// 1 / sqrt(x) to two ulps for normal x > 0: the seed and two Newton steps; 0 for infinity, NaN for NaN.
__device__ __forceinline__ double inverse_sqrt64(double x) {
  const double s = __builtin_amdgcn_rsq(x);
  const double h = 0.5 * x;
  const double r = __builtin_fma(s, __builtin_fma(-h * s, s, 0.5), s);
  const double y = __builtin_fma(r, __builtin_fma(-h * r, r, 0.5), r);
  return x < __builtin_inf() ? y : s;
}

// A head's row is with LG neighbouring lanes, eight values each: four pairs (of MOE_ROPE_HALF: four values and their
// four partners), or eight values that do not turn. A workgroup takes `units` heads of a token, or all of TK tokens, which
// it looks up side by side, a wave each; the next head's values are on their way while it works on one, the first before
// the sequences are known. Everything is in 64 bits: sums and products at full rate, conversions at a quarter, which bound
// 8192 tokens of 48 heads of 128 (77 us, 2.6 TB/s; without the norm 69). One token takes 5.3 us: loads that wait for each other.
// Slower for the 8192: one token a workgroup (99 us), two to four heads on their way (82 to 98), weights kept in 64 bits (101).
template <typename T, int LG, int TK>
__global__ __launch_bounds__(256) void k_window_append(AppendArgs a) {
  constexpr int GROUPS = 256 / LG;
  __shared__ double s_turn[TK][128][2];
  __shared__ int s_place[TK][4];   // key (-1: no token), page (-1: none), slot
  const int first_row = blockIdx.x * TK, l = threadIdx.x % LG, d = a.c.d, half = a.n_rot / 2, all = a.n_heads + 2 * a.c.n_kv;
  const int last = min((int)(blockIdx.y + 1) * a.units, all);   // of the heads (TK = 1)
  struct Part {   // this lane's values of a head: n0 from at0 on, n1 from at1 on
    int at0, at1, n0, n1;
    bool turns, halves;
  };
  auto part_of = [&](bool is_v) {
    const int rot = is_v ? 0 : a.n_rot, turning = (rot + 7) / 8;
    Part p;
    p.turns = l < turning, p.halves = p.turns && a.layout == MOE_ROPE_HALF;
    p.at0 = p.halves ? 4 * l : p.turns ? 8 * l : rot + 8 * (l - turning);
    p.at1 = p.halves ? half + 4 * l : p.at0 + 4;
    const int end = p.turns ? rot : d;
    p.n0 = (p.halves ? half : end) - p.at0, p.n1 = end - p.at1;
    return p;
  };
  const Part turning = part_of(false), plain = part_of(true);
  T raw[2][4];
  auto load = [&](int row, int u) {
    if (row >= first_row + TK || row >= a.w.n_tokens || u >= last) return;
    const bool is_q = u < a.n_heads, is_v = u >= a.n_heads + a.c.n_kv;
    const int h = is_q ? u : is_v ? u - a.n_heads - a.c.n_kv : u - a.n_heads;
    const T* x = is_q ? (const T*)a.q + row * a.ldq : is_v ? (const T*)a.v + row * a.ldv : (const T*)a.k + row * a.ldk;
    const Part p = is_v ? plain : turning;
    x += (int64_t)h * d;
    load4(x + p.at0, p.n0, raw[0]);
    load4(x + p.at1, p.n1, raw[1]);
  };
  int row = first_row, u = blockIdx.y * a.units + (int)threadIdx.x / LG;
  auto next = [&](int& row, int& u) {
    u += GROUPS;
    while (TK > 1 && u >= all) u -= all, ++row;
  };
  while (TK > 1 && u >= all) u -= all, ++row;
  load(row, u);
  // the weights of this lane's values
  float qw[8], kw[8];
  if (a.q_weight) {
    load4(a.q_weight, a.w_dtype, turning.at0, turning.n0, qw);
    load4(a.q_weight, a.w_dtype, turning.at1, turning.n1, qw + 4);
  }
  if (a.k_weight) {
    load4(a.k_weight, a.w_dtype, turning.at0, turning.n0, kw);
    load4(a.k_weight, a.w_dtype, turning.at1, turning.n1, kw + 4);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(a.w, 0x7FFFFFFF, 256);
  const int wave = threadIdx.x >> 6;
  int my_key = -1, my_page = -1, my_slot = 0;
  if (TK == 1 || wave < TK) {
    const int mine = first_row + (TK == 1 ? 0 : wave);
    const Seq q = mine < a.w.n_tokens ? seq_of(a.w, mine, 0x7FFFFFFF) : Seq{0, 0, 0, 0};
    if (q.tokens > 0) {
      my_key = q.ctx + mine - q.start;
      my_page = a.w.pages[q.s * a.w.ld_pages + my_key / a.c.page_size];
      my_slot = my_key % a.c.page_size;
      if (my_page < 0 || my_page >= a.c.n_pages) {
        my_page = -1;
        if (blockIdx.y == 0 && (threadIdx.x & 63) == 0) atomicOr(a.w.err, MOE_ERR_PAGE);
      }
    }
    if (TK > 1 && (threadIdx.x & 63) == 0) s_place[wave][0] = my_key, s_place[wave][1] = my_page, s_place[wave][2] = my_slot;
  }
  if constexpr (TK > 1) __syncthreads();
  else if (my_key < 0) return;
  for (int i = threadIdx.x; i < TK * half; i += 256) {
    const int t = TK == 1 ? 0 : i / half, p = i - t * half, key = TK == 1 ? my_key : s_place[t][0];
    if (key < 0) continue;
    double c, s;
    turn64((double)(a.w.pos ? a.w.pos[first_row + t] : key) * (double)a.freq[p], c, s);
    s_turn[t][p][0] = a.amp * c;
    s_turn[t][p][1] = a.amp * s;
  }
  __syncthreads();
  for (; row < first_row + TK && u < last; next(row, u)) {
    const bool is_q = u < a.n_heads, is_v = u >= a.n_heads + a.c.n_kv;
    const int t = row - first_row;
    const int page = TK == 1 ? my_page : s_place[t][1], slot = TK == 1 ? my_slot : s_place[t][2];
    const bool page_ok = page >= 0;
    const int h = is_q ? u : is_v ? u - a.n_heads - a.c.n_kv : u - a.n_heads;
    const Part p = is_v ? plain : turning;
    double y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (double)to_f(raw[e / 4][e % 4]);
    {
      int r = row, v = u;
      next(r, v);
      load(r, v);
    }
    if (TK > 1 && s_place[t][0] < 0) continue;   // a row of no sequence
    if (is_q ? a.q_weight != nullptr : !is_v && a.k_weight) {
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fma(y[e], y[e], sum);
      const double rinv = inverse_sqrt64(__builtin_fma(lanes_sum<LG>(sum), 1.0 / d, (double)a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rinv * (double)(is_q ? qw[e] : kw[e]);
    }
    if (p.turns) {
      double z[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = 4 * l + e < half;   // past the last pair zeros, which stay
        const double c = in ? s_turn[t][4 * l + e][0] : 1.0, s = in ? s_turn[t][4 * l + e][1] : 0.0;
        const double p0 = p.halves ? y[e] : y[2 * e], p1 = p.halves ? y[4 + e] : y[2 * e + 1];
        const double r0 = __builtin_fma(p0, c, -(p1 * s)), r1 = __builtin_fma(p1, c, p0 * s);
        // by selects: an index that differs from lane to lane would put y into memory
        y[e] = p.halves ? r0 : y[e];
        y[4 + e] = p.halves ? r1 : y[4 + e];
        z[2 * e] = r0, z[2 * e + 1] = r1;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = p.halves ? y[e] : z[e];
    }
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)y[e];
    auto put = [&](auto* o, const float* f) {
      store4(o + p.at0, p.n0, f);
      store4(o + p.at1, p.n1, f + 4);
    };
    if (is_q) {
      on_type(a.o_dtype, [&](auto t) {
        auto* o = (decltype(t)*)a.q_out + row * a.ldo + (int64_t)h * d;
        put(o, f);
      });
      continue;
    }
    const int64_t at = page * a.c.page + h * a.c.head + slot * a.c.slot;
    uint8_t* pool = is_v ? a.c.v : a.c.k;
    if (a.c_dtype != MOE_I8) {
      if (!page_ok) continue;
      a.c_dtype == MOE_BF16 ? put((bf16_t*)pool + at, f) : put((f16_t*)pool + at, f);
      continue;
    }
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool there = e < 4 ? e < p.n0 : e - 4 < p.n1;
      most = max(most, there ? __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu : 0u);
    }
    most = lanes_max<LG>(most);
    const bool finite = most < 0x7F800000u;
    const QScale s = q_scale(__builtin_bit_cast(float, most));
    uint32_t codes[2] = {0, 0};
    if (finite && s.d != 0.0f) codes8(f, s, codes);
    if (!page_ok) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = i ? p.n1 : p.n0;
      int8_t* o = (int8_t*)pool + at + (i ? p.at1 : p.at0);
      if (n >= 4) {
        __builtin_memcpy(o, &codes[i], 4);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < n) o[e] = (int8_t)(codes[i] >> (8 * e));
      }
    }
    if (l == 0)
      (is_v ? a.c.vs : a.c.ks)[((int64_t)page * a.c.n_kv + h) * a.c.page_size + slot] = finite ? s.d : __builtin_nanf("");
  }
}

// ------------------------------------------------------------------ attention ---------------
//
// The keys of a sequence are cut into runs (run_of), a workgroup takes one run of one cache head for a tile of rows (the
// window's tokens times the query heads that share the cache head), and k_attend_join adds the runs of a row up. A wave takes
// 64 of every 256 keys, 32 at a time. All products are transposed: scores are K . Q^T, so that a lane has four neighbouring keys
// of one row and the row's factors are the lane's own, and K's rows go from memory straight into the matrix instruction's
// lanes; the exponentials are already where V^T . P^T takes them (which key is which place of the sum over keys is free, as
// long as V agrees), and a lane loads the same eight neighbouring values of eight keys, from which a byte permutation
// makes the eight rows of V^T. Without WIDE there is no LDS until the waves join.
// Bound by the cache's bytes up to some 32 rows a cache head: 4 tokens x 8 heads over 131072 keys 55 us (4.9 TB/s) and 5 to
// join, one token 50 us (5.3 TB/s); 64 sequences x 4 tokens of 512 to 8192 keys, int8 137 us (4.4 TB/s) and 8, bf16 231
// (4.9 TB/s). One token over 4096 keys takes 11 us and 4 to join: 64 workgroups, whose waves walk two steps of loads
// that wait for each other (lengths, pages, keys). Trees of 64 tokens x 8 heads over 4096 to 8100 keys 220 us (0.44 PFLOP/s)
// and 24: counted over the launch, 328 vector and 115 scalar instructions for every 32 matrix instructions (a step), which
// two waves a SIMD overlap only in part; some 180 scalars are spilled to lanes. Their runs' results are 104 MB written and
// read back where the case itself has 207. Registers: two tiles of 128 wide 16-bit heads spill 5 (16 bytes of scratch a
// lane), two of 144 to 256 values 133 (380 bytes, one wave a SIMD): 4 tokens x 8 heads of 256 over 131072 keys 133 us
// (4.0 TB/s).
// Tried and slower: keys and values of two steps in registers (145 us for the int8 batch where this takes 136), three
// waves a SIMD (spills; 158), values read from the ring when they are needed (265 us for the trees where this takes 219).

struct AttendArgs {
  CacheArgs c;
  WindowArgs w;
  const void* q;
  void* out;
  float *lse, *part, *part_ml;   // of runs: [row][head][max_runs] head_dim values, and (maximum, sum)
  int64_t ldq, ldo;
  int n_heads, max_runs, least_run;
  float scale;
};

// Keys of a run: `least` (by the call's sizes), or what makes kMaxRuns of the sequence's keys.
__host__ __device__ __forceinline__ int run_of(int keys, int least) { return max(least, ((keys >> 6) + 256) & ~255); }
__host__ __device__ __forceinline__ int runs_of(int keys, int least) {
  const int run = run_of(keys, least);
  return (int)(((int64_t)keys + run - 1) / run);
}
constexpr int kMaxRuns = 64;   // runs_of of any count

// s_waitcnt vmcnt(n), the other counters left alone (n < 64; vmcnt in bits 3:0 and 15:14)
#define MOE_VM(n) (((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))
// Every LDS access of the wave has finished, then the workgroup meets; loads stay on their way.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <typename T>
struct Mat;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <>
struct Mat<bf16_t> {
  static constexpr float kBoost = 0.0f;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});
  }
  static constexpr uint32_t kOne = 0x3F80u;
  static __device__ __forceinline__ uint32_t odd(uint32_t x) {   // of two values, bit 0 / bit 16: not finite
    return ((x & 0x00007F80u) == 0x00007F80u ? 1u : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0x10000u : 0u);
  }
};
template <>
struct Mat<f16_t> {
  static constexpr float kBoost = 14.0f;   // weights up to 2^14, so that small ones stay normal numbers
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{(_Float16)a, (_Float16)b});
  }
  static constexpr uint32_t kOne = 0x3C00u;
  static __device__ __forceinline__ uint32_t odd(uint32_t x) {
    return ((x & 0x00007C00u) == 0x00007C00u ? 1u : 0u) | ((x & 0x7C000000u) == 0x7C000000u ? 0x10000u : 0u);
  }
};

// Over the four lanes of a row (lane, and 16, 32, 48 on).
__device__ __forceinline__ float max4(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
}
__device__ __forceinline__ float sum4(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}

// 32 keys of a head as they are loaded: of keys 16 t + lane % 16 the values that the matrix instruction takes from this lane, and
// of keys 16 t + 4 (lane / 16) + i this lane's neighbouring values.
template <bool I8, int HD>
struct Keys {
  static constexpr int KL = I8 ? HD / 64 : HD / 32, VD = I8 ? HD / 64 : HD / 32;
  u32x4 k[2][KL];
  uint32_t v[8][VD];
  f32x4 ks[2], vs[2];
};

// The log of a sum of 2^(x - best), in natural units.
__device__ __forceinline__ float lse_of(float best, float sum) {
  return sum == 0.0f ? -__builtin_inff() : (best + __builtin_log2f(sum)) * 0.69314718055994530942f;
}

constexpr uint32_t kNowhere = 0x80000000u;   // an offset past any buffer: the load gives 0 and touches nothing

// HD: 64, 128 or 256, the least that holds head_dim. NT: a wave's tiles of 16 rows. WIDE: the waves share the keys, which
// then go through LDS (a ring of stages of 32 keys, loaded straight into it), and have rows of their own; otherwise they
// share the rows, and a wave takes 64 of every 256 keys. The next keys are loaded as soon as these are multiplied, the
// next values as soon as these are.
constexpr int ring_bytes(int hd, bool i8) {   // three stages, or two large ones
  return 64 * hd * (i8 ? 1 : 2) * (hd * (i8 ? 1 : 2) > 256 ? 2 : 3);
}
constexpr int kAttendWaves(int hd) { return hd < 256 ? 2 : 1; }   // of a SIMD: what their registers leave room for
template <typename T, bool I8, int HD, int NT, bool WIDE>
__global__ __launch_bounds__(256, kAttendWaves(HD)) void k_attend(AttendArgs a) {
  using M = Mat<T>;
  using KV = Keys<I8, HD>;
  // In front of V a weight is rounded to T, which costs bits: the error of bfloat16 outputs of 1 x 4 tokens over 131072 keys
  // against 64 bits is 2.1e-3 instead of 1.7e-3. (Two parts of 8 bits each, two products: as fast there, but 8 x 64 bf16
  // 258 us instead of 219.) Over an int8 cache a weight has its value's scale in it, of float32's range and any size next
  // to the others', and is bfloat16 whatever T: float16 under a common power of two lost the rows whose scales are small.
  // It is in two parts there (64 x 4 of 8192: 2.4e-3 and 1.7e-3, 136 us and 137), but for bfloat16 queries of many rows,
  // which the products bound (8 x 64: 261 us, in two parts 290 to 303).
  using MV = Mat<std::conditional_t<I8, bf16_t, T>>;
  constexpr bool PARTS = I8 && (!WIDE || std::is_same_v<T, f16_t>);
  constexpr int ROWS = 16 * NT * (WIDE ? 4 : 1), KS = HD / 32, E0 = HD < 128 ? 4 : 8, NH = HD < 128 ? 1 : HD / 128, DT = E0 * NH;
  constexpr int SIZE = I8 ? 1 : 2, STRIDE = HD + 4;
  __shared__ float s_m[4][WIDE ? 1 : ROWS], s_l[4][WIDE ? 1 : ROWS], s_o[4][WIDE ? 1 : 16 * STRIDE];
  constexpr bool Q_LDS = !WIDE && NT == 2;
  __shared__ u32x4 s_q[Q_LDS ? NT : 1][Q_LDS ? KS : 1][Q_LDS ? 64 : 1];
  __shared__ int s_wave[4];
  // the ring: rows of 16-byte chunks, chunk c of row r at place c ^ swizzle(r), so that neighbouring lanes meet other banks
  constexpr int CR = HD * SIZE / 16, HALF = 32 * HD * SIZE, STAGE = 2 * HALF, STAGES = ring_bytes(HD, I8) / STAGE;
  constexpr int RPI = 64 / CR, NI = 32 / RPI, PER = NI / 2;   // rows a load instruction has, loads of K, loads a wave makes
  // static, the compiler would have reads wait for the loads on their way
  extern __shared__ __align__(16) uint8_t s_ring[];
  int* const s_end = (int*)(s_ring + (WIDE ? STAGES * STAGE : 0));   // [n_seqs]: items of the sequences up to this one
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, col = lane & 15, quad = lane >> 4;
  const int G = a.n_heads / a.c.n_kv, d = a.c.d;
  auto items_of = [&](int start, int end, int ctx) {
    if (!seq_ok(a.w, start, end, ctx, a.w.max_window)) {
      if (blockIdx.x == 0) atomicOr(a.w.err, MOE_ERR_WINDOW);
      return 0;
    }
    return end > start ? ((end - start) * G + ROWS - 1) / ROWS * runs_of(ctx + end - start, a.least_run) * a.c.n_kv : 0;
  };
  auto scan = [&](int n) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int up = __shfl_up(n, o);
      if (lane >= o) n += up;
    }
    return n;
  };
  auto largest = [&](int n) {   // of the lanes before this one
#pragma unroll
    for (int o = 1; o < 64; o *= 2) n = max(n, __shfl_up(n, o));
    n = __shfl_up(n, 1);
    return lane > 0 ? n : (int)0x80000000;
  };
  // items of the sequences up to each: in the lanes of every wave, or, of more than 64, in LDS
  int total = 0, my_start = 0, my_end = 0, my_ctx = 0, my_items = 0;
  const bool few = a.w.n_seqs <= 64;
  if (few) {
    int n = 0;
    if (lane < a.w.n_seqs) {
      my_start = a.w.row_start[lane], my_end = a.w.row_start[lane + 1], my_ctx = a.w.ctx_len[lane];
      n = items_of(my_start, my_end, my_ctx);
    }
    if (__ballot(my_end < my_start)) {   // the list goes back
      const int earlier = largest(my_start);
      if (earlier > my_start) n = 0;
    }
    my_items = scan(n);
    total = __builtin_amdgcn_readlane(my_items, 63);
  } else {
    bool back = false;
    int top = (int)0x80000000;   // the largest start of the sequences before these 256, from the first that goes back on
    for (int i0 = 0; i0 < a.w.n_seqs; i0 += 256) {
      const int i = i0 + tid;
      int n = 0, start = top, end = top;
      if (i < a.w.n_seqs) {
        start = a.w.row_start[i], end = a.w.row_start[i + 1];
        n = items_of(start, end, a.w.ctx_len[i]);
      }
      if (__syncthreads_or(end < start)) back = true;
      if (back) {
        int earlier = largest(start);
        if (lane == 63) s_wave[wave] = max(earlier, start);
        earlier = max(earlier, top);
        __syncthreads();
        for (int w = 0; w < 4; ++w) {
          if (w < wave) earlier = max(earlier, s_wave[w]);
          top = max(top, s_wave[w]);
        }
        if (earlier > start) n = 0;
        __syncthreads();
      }
      n = scan(n);
      if (lane == 63) s_wave[wave] = n;
      __syncthreads();
      for (int w = 0; w < wave; ++w) n += s_wave[w];
      if (i < a.w.n_seqs) s_end[i] = total + n;
      total += s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3];
      __syncthreads();
    }
    total = __builtin_amdgcn_readfirstlane(total);
  }
  auto swizzle = [](int r) { return CR == 4 ? r >> 1 & 3 : r & (CR < 16 ? CR - 1 : 15); };
  if constexpr (WIDE) {
    if (d < HD) {   // places that no load reaches
      for (int i = tid; i < STAGES * STAGE / 16; i += 256) ((u32x4*)s_ring)[i] = u32x4{0, 0, 0, 0};
      __syncthreads();
    }
  }
  // neighbouring items, the tiles of one run among them, on one die
  const int first = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const float c = a.scale == 0.0f ? 1.0f : __builtin_fabsf(a.scale) * 1.44269504088896340736f;
  const int64_t slot_bytes = a.c.slot * SIZE;
  for (int item = first; item < total; item += gridDim.x) {
    int s = 0, rest, start, tokens, ctx;
    if (few) {
      s = __popcll(__ballot(my_items <= item));   // the first whose end is past the item
      rest = item - (s > 0 ? __builtin_amdgcn_readlane(my_items, s - 1) : 0);
      start = __builtin_amdgcn_readlane(my_start, s);
      tokens = __builtin_amdgcn_readlane(my_end, s) - start;
      ctx = __builtin_amdgcn_readlane(my_ctx, s);
    } else {
      for (int n = a.w.n_seqs; n > 0;) {
        const int mid = n >> 1;
        if (s_end[s + mid] <= item) s += mid + 1, n -= mid + 1;
        else n = mid;
      }
      s = __builtin_amdgcn_readfirstlane(s);
      rest = item - __builtin_amdgcn_readfirstlane(s > 0 ? s_end[s - 1] : 0);
      start = __builtin_amdgcn_readfirstlane(a.w.row_start[s]);
      tokens = __builtin_amdgcn_readfirstlane(a.w.row_start[s + 1]) - start;
      ctx = __builtin_amdgcn_readfirstlane(a.w.ctx_len[s]);
    }
    const int keys = ctx + tokens, rows = tokens * G;
    const int tiles = (rows + ROWS - 1) / ROWS, run = run_of(keys, a.least_run), runs = runs_of(keys, a.least_run);
    const int tile = rest % tiles;
    rest /= tiles;
    const int part = rest % runs, head = rest / runs;   // of the cache
    const int key0 = part * run, len = min(run, keys - key0);
    const int steps = WIDE ? (len + 31) >> 5 : 2 * (len >> 8) + min(2, max(0, (len & 255) - 64 * wave + 31) >> 5);
    // a step's first key, from the run's first: past the run's end it still counts in 32 bits, the key itself may not
    auto rel_of = [&](int step) { return WIDE ? step * 32 : (step >> 1) * 256 + wave * 64 + (step & 1) * 32; };
    auto key_of = [&](int step) { return key0 + rel_of(step); };

    // rows: this lane's row of each tile of 16, its token's mask, and its part of Q^T
    uint64_t seen[NT];
    u32x4 q[Q_LDS ? 1 : NT][Q_LDS ? 1 : KS];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = tile * ROWS + 16 * ((WIDE ? wave * NT : 0) + t) + col, j = r / G;
      const bool row = r < rows;
      const int64_t at = start + (row ? j : 0);
      uint64_t mask = ~0ull >> (63 - (row ? j : 0));
      if (a.w.seen) mask = a.w.seen[at];
      seen[t] = row ? mask & (~0ull >> (64 - tokens)) : 0;
      const T* x = (const T*)a.q + at * a.ldq + (int64_t)(head * G + r % G) * d;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int i = I8 ? (k >> 1) * 64 + quad * 16 + (k & 1) * 8 : k * 32 + quad * 8;
        if (Q_LDS && (k & 3) != wave) continue;
        u32x4 v = {0, 0, 0, 0};
        if (row && i < d && a.scale != 0.0f) __builtin_memcpy(&v, x + i, 16);
        if (a.scale < 0.0f) v ^= 0x80008000u;
        if constexpr (Q_LDS) s_q[t][k][lane] = v;
        else q[t][k] = v;
      }
    }
    if constexpr (Q_LDS) __syncthreads();
    float m[NT], l[NT];
    f32x4 acc[NT][DT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -__builtin_inff();
      l[t] = 0.0f;
#pragma unroll
      for (int x = 0; x < DT; ++x) acc[t][x] = f32x4{0, 0, 0, 0};
    }

    // Lane i: where tile i of 16 keys (of the wave's from the batch on) is, in bytes from the head's first page, and its scales;
    // `there`: the tiles that are.
    uint32_t at_lo = 0, at_hi = 0, sc_lo = 0, sc_hi = 0;
    uint64_t there = 0;
    auto pages = [&](int batch) {
      const int rel = rel_of(batch + (lane >> 1)) + 16 * (lane & 1), key = key0 + (rel < len ? rel : 0);
      int page = -1, slot = 0;
      if (rel < len) {
        page = a.w.pages[s * a.w.ld_pages + key / a.c.page_size];
        slot = key % a.c.page_size;
        if (page < 0 || page >= a.c.n_pages) {
          atomicOr(a.w.err, MOE_ERR_PAGE);
          page = -1;
        }
      }
      there = __ballot(page >= 0);
      const int64_t at = page >= 0 ? (page * a.c.page + slot * a.c.slot) * SIZE : 0;
      at_lo = (uint32_t)at, at_hi = (uint32_t)(at >> 32);
      if constexpr (I8) {
        const int64_t sc = page >= 0 ? (((int64_t)page * a.c.n_kv + head) * a.c.page_size + slot) * 4 : 0;
        sc_lo = (uint32_t)sc, sc_hi = (uint32_t)(sc >> 32);
      }
    };
    const uint64_t k_head = (uint64_t)(a.c.k + head * a.c.head * SIZE), v_head = (uint64_t)(a.c.v + head * a.c.head * SIZE);
    auto lane64 = [](uint32_t lo, uint32_t hi, int i) {
      return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)lo, i) |
             (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, i) << 32;
    };
    auto buffer = [](uint64_t at, bool live) {
      return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, live ? 0x7FFFFFFF : 0, 0x00027000);
    };
    auto four = [&](const float* scales, uint64_t at, bool live) {
      const auto from = buffer((uint64_t)scales + at, live);
      return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, quad * 16, 0, 0));
    };
    auto scales = [&](KV& kv, int step, bool k, bool v) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int i = 2 * (step & 31) + t;
        const bool live = step < steps && (there >> i & 1);
        const uint64_t at = lane64(sc_lo, sc_hi, i);
        if (k) kv.ks[t] = four(a.c.ks, at, live);
        if (v) kv.vs[t] = four(a.c.vs, at, live);
      }
    };

    // Keys straight into registers. Lane offsets; of what is past head_dim, nowhere.
    uint32_t k_off[KV::KL], v_off[NH];
#pragma unroll
    for (int u = 0; u < KV::KL; ++u) {
      const uint32_t byte = u * 64 + quad * 16;
      k_off[u] = byte < (uint32_t)(d * SIZE) ? (uint32_t)(col * slot_bytes) + byte : kNowhere;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int e = h * 128 + col * E0;
      v_off[h] = e < d ? (uint32_t)(4 * quad * slot_bytes) + (uint32_t)(e * SIZE) : kNowhere;
    }
    auto load = [&](KV& kv, int step, bool want_k, bool want_v) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int at = 2 * (step & 31) + t;
        const bool live = step < steps && (there >> at & 1);
        const uint64_t off = lane64(at_lo, at_hi, at);
        const auto kr = buffer(k_head + off, live), vr = buffer(v_head + off, live);
#pragma unroll
        for (int u = 0; want_k && u < KV::KL; ++u)
          kv.k[t][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(kr, k_off[u], 0, 0));
#pragma unroll
        for (int i = 0; want_v && i < 4; ++i)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            constexpr int W = E0 * SIZE / 4;
            uint32_t* to = &kv.v[4 * t + i][h * W];
            const int slot = (int)(i * slot_bytes);
            if constexpr (W == 4) {
              const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(vr, v_off[h], slot, 0));
              to[0] = x[0], to[1] = x[1], to[2] = x[2], to[3] = x[3];
            } else if constexpr (W == 2) {
              const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(vr, v_off[h], slot, 0));
              to[0] = x[0], to[1] = x[1];
            } else {
              to[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(vr, v_off[h], slot, 0);
            }
          }
      }
      if constexpr (I8) scales(kv, step, want_k, want_v);
    };

    // Through LDS: a wave's share of a step's rows on the way to the ring, and a step's values from there.
    uint32_t s_off[WIDE ? PER : 1];
    if constexpr (WIDE) {
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int r = (wave + 4 * x) % NI * RPI + lane / CR, byte = ((lane % CR) ^ swizzle(r)) * 16;
        s_off[x] = byte < d * SIZE ? (uint32_t)((r & 15) * slot_bytes) + byte : kNowhere;
      }
    }
    uint64_t lives = 0;   // of the tiles sent: bit 2 (step % 32) + t
    auto send = [&](int step, int slot) {
      const int at = 2 * (step & 31);
      lives = (lives & ~(3ull << at)) | (there & 3ull << at);
      uint8_t* const stage = s_ring + slot * STAGE;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int j = wave + 4 * x, of_v = j >= NI, row0 = (of_v ? j - NI : j) * RPI, i = at + (row0 >> 4);
        const auto from = __builtin_amdgcn_make_buffer_rsrc((void*)((of_v ? v_head : k_head) + lane64(at_lo, at_hi, i)), 0,
                                                            there >> i & 1 ? 0x7FFFFFFF : 0, 0x00027000);
        MOE_LDS void* const to = (MOE_LDS void*)(stage + of_v * HALF + row0 * (HD * SIZE));
        if (s_off[x] != kNowhere) __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 16, (int)s_off[x], 0, 0, 0);
      }
    };
    auto read = [&](KV& kv, int slot) {
      int col = lane & 15, quad = lane >> 4;   // offsets made anew each time: kept, they cost registers that the loop has not
      asm volatile("" : "+v"(col), "+v"(quad));
      const uint8_t* const stage = s_ring + slot * STAGE;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int u = 0; u < KV::KL; ++u)
          kv.k[t][u] = *(const u32x4*)(stage + (16 * t + col) * (HD * SIZE) + ((u * 4 + quad) ^ swizzle(col)) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const int byte = (h * 128 + col * E0) * SIZE, r = 4 * quad + i;
            constexpr int W = E0 * SIZE / 4;
            using Words = std::conditional_t<W == 4, u32x4, std::conditional_t<W == 2, u32x2, uint32_t>>;
            const uint8_t* const row = stage + HALF + (16 * t + r) * (HD * SIZE);
            const Words x = *(const Words*)(row + ((byte >> 4) ^ swizzle(r)) * 16 + (byte & 15));
            __builtin_memcpy(&kv.v[4 * t + i][h * W], &x, 4 * W);
          }
      }
    };

    bool odd = false;   // whether a value of a window's key is not finite
    // One step; `next` is called when the keys (true) and then the values (false) are used up.
    // Steps of the context whose pages are all there (`plain`) need no masks; a loop of their own keeps the masks' registers
    // out of it.
    auto plain = [&](int step, const bool (&live)[2]) { return rel_of(step) + 32 <= ctx - key0 && live[0] && live[1]; };
    auto use = [&](auto checked, KV& kv, int step, const bool (&live)[2], auto next) {
      constexpr bool check = checked();
      const int key = key_of(step);
      f32x4 p[2][NT];
      int q_lane = lane;   // read each time: kept, the rows cost registers that the loop has not
      if constexpr (Q_LDS) asm volatile("" : "+v"(q_lane));
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) p[t][n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        u32x4 qk[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (Q_LDS) qk[n] = s_q[n][k][q_lane];
          else qk[n] = q[n][k];
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          u32x4 f;
          if constexpr (I8) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t b = kv.k[t][k >> 1][2 * (k & 1) + (x >> 1)] >> (16 * (x & 1));
              f[x] = M::pack((float)(int8_t)b, (float)(int8_t)(b >> 8));
            }
          } else {
            f = kv.k[t][k];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) p[t][n] = M::mma(f, qk[n], p[t][n]);
        }
      }
      if constexpr (I8) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[t][n][i] *= kv.ks[t][i];
      }
      next(true);
      uint32_t sight[NT] = {};   // I8: the keys that a row sees, whose scales count though their weights may round to 0
      if constexpr (check) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rel = key + 16 * t + 4 * quad + i - ctx;
            if (rel >= tokens || !live[t]) {   // a slot past the last key may hold anything
#pragma unroll
              for (int y = 0; y < KV::VD; ++y) kv.v[4 * t + i][y] = 0;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const bool sees = live[t] && (rel < 0 || (rel < 64 && (seen[n] >> (rel & 63) & 1)));
              p[t][n][i] = sees ? p[t][n][i] : -__builtin_inff();
              if constexpr (I8) sight[n] |= sees ? 1u << (4 * t + i) : 0;
            }
          }
        // A value of a drafted token that is not finite must not reach rows that do not see it (0 times it is NaN): it
        // counts as 0 here, and add_odd adds it to the rows that do.
        if constexpr (!I8) {
          uint32_t any = 0;
#pragma unroll
          for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < KV::VD; ++y) {
              const uint32_t o = key + 16 * (x >> 2) + 4 * quad + (x & 3) >= ctx ? M::odd(kv.v[x][y]) : 0;
              any |= o;
              kv.v[x][y] &= ~(o * 0xFFFFu);
            }
          odd |= __ballot(any != 0) != 0;
        }
      }
      float top[NT];
      bool grows = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x = m[n];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) x = __builtin_fmaxf(x, p[t][n][i]);
        top[n] = max4(x);
        grows |= top[n] > m[n];
      }
      if (__ballot(grows)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float ref = top[n] == -__builtin_inff() ? 0.0f : top[n];
          const float keep = __builtin_amdgcn_exp2f((m[n] - ref) * c);
          l[n] *= keep;
#pragma unroll
          for (int x = 0; x < DT; ++x) acc[n][x] *= keep;
          m[n] = top[n];
        }
      }
      u32x4 w[NT], w_lo[PARTS ? NT : 1];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float mc = (m[n] == -__builtin_inff() ? 0.0f : m[n]) * c - MV::kBoost;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[t][n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[t][n][i], c, -mc));
          sum += (p[t][n][0] + p[t][n][1]) + (p[t][n][2] + p[t][n][3]);
          f32x4 y = p[t][n];
          if constexpr (I8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = check && !(sight[n] >> (4 * t + i) & 1) ? 0.0f : y[i] * kv.vs[t][i];
          }
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const uint32_t hi = MV::pack(y[i], y[i + 1]);
            w[n][2 * t + i / 2] = hi;
            if constexpr (PARTS)
              w_lo[n][2 * t + i / 2] = MV::pack(y[i] - __builtin_bit_cast(float, hi << 16),
                                                y[i + 1] - __builtin_bit_cast(float, hi & 0xFFFF0000u));
          }
        }
        l[n] += sum;
      }
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e8 = 0; e8 < E0; ++e8) {
          u32x4 f;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if constexpr (I8) {
              constexpr int W = E0 / 4;
              const uint32_t lo = kv.v[2 * y][h * W + e8 / 4] >> (8 * (e8 & 3));
              const uint32_t hi = kv.v[2 * y + 1][h * W + e8 / 4] >> (8 * (e8 & 3));
              f[y] = MV::pack((float)(int8_t)lo, (float)(int8_t)hi);
            } else {
              constexpr int W = E0 / 2;
              f[y] = __builtin_amdgcn_perm(kv.v[2 * y + 1][h * W + e8 / 2], kv.v[2 * y][h * W + e8 / 2],
                                           e8 & 1 ? 0x07060302u : 0x05040100u);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][h * E0 + e8] = MV::mma(f, w[n], acc[n][h * E0 + e8]);
            if constexpr (PARTS) acc[n][h * E0 + e8] = MV::mma(f, w_lo[n], acc[n][h * E0 + e8]);
          }
        }
      next(false);
    };
    auto add_odd = [&]() {
      if constexpr (!I8) {
        for (int step = 0; step < steps; ++step)
          for (int k = 0; k < 32; ++k) {
            const int key = key_of(step) + k;
            if (key < ctx || key >= keys) continue;
            const int page = a.w.pages[s * a.w.ld_pages + key / a.c.page_size];
            if (page < 0 || page >= a.c.n_pages) continue;
            const T* v = (const T*)v_head + page * a.c.page + key % a.c.page_size * a.c.slot;
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = x / E0 * 128 + (4 * quad + i) * E0 + x % E0;
                const float f = to_f(v[e < d ? e : 0]);
                const bool counts = (e < d) & !(__builtin_fabsf(f) < __builtin_inff());
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][x][i] += counts & (bool)(seen[n] >> (key - ctx) & 1) ? f : 0.0f;
              }
          }
      }
    };

    if constexpr (WIDE) {
      KV x, ahead;
      bool live[2];
      pages(0);
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i)
        if (i < steps) send(i, i);
      if constexpr (I8) scales(ahead, 0, true, true);
      auto arrive = [&](int i) {
        // this step has landed: all but the loads of the steps behind it
        if (i + STAGES - 2 < steps) __builtin_amdgcn_s_waitcnt(MOE_VM(PER * (STAGES - 2)));
        else __builtin_amdgcn_s_waitcnt(MOE_VM(0));
        meet();   // all waves', and the stage before it is free
        live[0] = lives >> (2 * (i & 31)) & 1, live[1] = lives >> (2 * (i & 31) + 1) & 1;
      };
      auto step = [&](auto checked, int i, int slot) {
        const int next = i + STAGES - 1;
        if constexpr (I8) {
#pragma unroll
          for (int t = 0; t < 2; ++t) x.ks[t] = ahead.ks[t], x.vs[t] = ahead.vs[t];
          if (STAGES > 2 && i + 1 < steps) scales(ahead, i + 1, true, true);   // while its pages are there
        }
        if (next < steps) {
          if ((next & 31) == 0) pages(next);
          send(next, slot == 0 ? STAGES - 1 : slot - 1);
          if constexpr (I8 && STAGES == 2) scales(ahead, next, true, true);
        }
        read(x, slot);
        use(checked, x, i, live, [](bool) {});
      };
      int i = 0, slot = 0;
      for (; i < steps; ++i, slot = slot + 1 == STAGES ? 0 : slot + 1) {
        arrive(i);
        if (!plain(i, live)) break;
        step(std::false_type{}, i, slot);
      }
      while (i < steps) {
        step(std::true_type{}, i, slot);
        ++i, slot = slot + 1 == STAGES ? 0 : slot + 1;
        if (i < steps) arrive(i);
      }
    }
    for (int batch = 0; !WIDE && batch < steps; batch += 32) {
      pages(batch);
      const int last = min(batch + 32, steps);
      KV x;
      load(x, batch, true, false);
      __builtin_amdgcn_sched_barrier(0);   // in this order, so that the loop waits for the keys alone
      load(x, batch, false, true);
      int i = batch;
      auto step = [&](auto checked, const bool (&live)[2]) {
        use(checked, x, i, live, [&](bool keys_done) { load(x, i + 1 < last ? i + 1 : steps, keys_done, !keys_done); });
      };
      for (; i < last; ++i) {
        const bool live[2] = {(bool)(there >> (2 * (i & 31)) & 1), (bool)(there >> (2 * (i & 31) + 1) & 1)};
        if (!plain(i, live)) break;
        step(std::false_type{}, live);
      }
      for (; i < last; ++i) {
        const bool live[2] = {(bool)(there >> (2 * (i & 31)) & 1), (bool)(there >> (2 * (i & 31) + 1) & 1)};
        step(std::true_type{}, live);
      }
    }
    if (odd) add_odd();

    if constexpr (WIDE) {   // a lane has neighbouring values of its rows
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float sum = sum4(l[n]);
        const int r = tile * ROWS + 16 * (wave * NT + n) + col;
        if (r >= rows) continue;
        const float best = m[n] == -__builtin_inff() ? 0.0f : m[n];
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t row = start + r / G;
        const int qh = head * G + r % G;
        const int64_t idx = (row * a.n_heads + qh) * a.max_runs + part;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = h * 128 + (4 * quad + i) * E0;
            if (at >= d) continue;
            float o[E0];
#pragma unroll
            for (int x = 0; x < E0; ++x) o[x] = acc[n][h * E0 + x][i];
            if (runs == 1) {
              T y[E0];
#pragma unroll
              for (int x = 0; x < E0; ++x) y[x] = from_f<T>(sum == 0.0f ? 0.0f : o[x] * inv);
              __builtin_memcpy((T*)a.out + row * a.ldo + (int64_t)qh * d + at, y, sizeof y);
            } else {
              __builtin_memcpy(a.part + idx * d + at, o, sizeof o);
            }
          }
        if (quad == 0 && runs == 1 && a.lse)
          a.lse[row * a.n_heads + qh] = lse_of(best * c - MV::kBoost, sum);
        if (quad == 0 && runs > 1) {
          a.part_ml[2 * idx] = sum == 0.0f ? -__builtin_inff() : best * c - MV::kBoost;
          a.part_ml[2 * idx + 1] = sum;
        }
      }
      meet();
      continue;
    }
    if constexpr (!WIDE) {
      // the waves' results, in their order
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float sum = sum4(l[n]);
        if (quad == 0) {
          s_m[wave][16 * n + col] = m[n];
          s_l[wave][16 * n + col] = sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        auto best_of = [&](int r) {
          const float x = __builtin_fmaxf(__builtin_fmaxf(s_m[0][r], s_m[1][r]), __builtin_fmaxf(s_m[2][r], s_m[3][r]));
          return x == -__builtin_inff() ? 0.0f : x;
        };
        const float f = __builtin_amdgcn_exp2f((m[n] - best_of(16 * n + col)) * c);
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e4 = 0; e4 < E0; e4 += 4) {
              f32x4 y;
#pragma unroll
              for (int x = 0; x < 4; ++x) y[x] = acc[n][h * E0 + e4 + x][i] * f;
              *(f32x4*)&s_o[wave][col * STRIDE + h * 128 + (4 * quad + i) * E0 + e4] = y;
            }
        __syncthreads();
        const int rr = tid >> 4, at = (tid & 15) * (HD / 16), r = tile * ROWS + 16 * n + rr;
        if (r < rows && at < d) {
          const float best = best_of(16 * n + rr);
          float sum = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum += s_l[w][16 * n + rr] * __builtin_amdgcn_exp2f((s_m[w][16 * n + rr] - best) * c);
          const int64_t row = start + r / G;
          const int qh = head * G + r % G;
          float o[HD / 16];
#pragma unroll
          for (int x = 0; x < HD / 16; x += 4) {
            f32x4 y = *(const f32x4*)&s_o[0][rr * STRIDE + at + x];
#pragma unroll
            for (int w = 1; w < 4; ++w) y += *(const f32x4*)&s_o[w][rr * STRIDE + at + x];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[x + i] = y[i];
          }
          if (runs == 1) {
            T* out = (T*)a.out + row * a.ldo + (int64_t)qh * d + at;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            T y[HD / 16];
#pragma unroll
            for (int x = 0; x < HD / 16; ++x) y[x] = from_f<T>(sum == 0.0f ? 0.0f : o[x] * inv);
            __builtin_memcpy(out, y, sizeof y);
            if (a.lse && at == 0)
              a.lse[row * a.n_heads + qh] = lse_of(best * c - MV::kBoost, sum);
          } else {
            const int64_t idx = (row * a.n_heads + qh) * a.max_runs + part;
            __builtin_memcpy(a.part + idx * d + at, o, sizeof o);
            if (at == 0) {
              a.part_ml[2 * idx] = sum == 0.0f ? -__builtin_inff() : best * c - MV::kBoost;
              a.part_ml[2 * idx + 1] = sum;
            }
          }
        }
        __syncthreads();
      }
    }
  }
}

// The runs of a row and head, by W waves. Lanes side by side take four neighbouring values, and the groups of lanes every
// 4 W / (2 W, W)-th run of head_dim up to 64 (128, 256), always in the same order.
template <typename T, int W>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
  __shared__ float s_w[4 / W][kMaxRuns];
  __shared__ f32x4 s_o[W > 1 ? 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, team = tid / (64 * W), d = a.c.d;
  const int64_t item = (int64_t)blockIdx.x * (4 / W) + team;
  const bool there = item < (int64_t)a.w.n_tokens * a.n_heads;
  const int row = there ? (int)(item / a.n_heads) : 0, head = there ? (int)(item % a.n_heads) : 0;
  const int64_t idx = there ? item * a.max_runs : 0;
  // asked for before it is known how many there are
  float best = -__builtin_inff(), l = 0.0f;
  if (lane < a.max_runs) best = a.part_ml[2 * (idx + lane)], l = a.part_ml[2 * (idx + lane) + 1];
  const Seq q = seq_of(a.w, row, a.w.max_window);
  const int runs = there && q.tokens > 0 ? runs_of(q.ctx + q.tokens, a.least_run) : 0;
  if (runs <= 1) return;   // W > 1: the whole workgroup
  if (lane >= runs) best = -__builtin_inff(), l = 0.0f;
  const float m = best;
#pragma unroll
  for (int o = 32; o; o /= 2) best = __builtin_fmaxf(best, __shfl_xor(best, o));
  const float w = lane < runs ? __builtin_amdgcn_exp2f(m - (best == -__builtin_inff() ? 0.0f : best)) : 0.0f;
  float sum = l * w;
#pragma unroll
  for (int o = 32; o; o /= 2) sum += __shfl_xor(sum, o);
  if (W == 1 || tid < 64) s_w[team][lane] = w;
  if constexpr (W > 1) __syncthreads();
  else __builtin_amdgcn_wave_barrier();
  const int wide = d <= 64 ? 16 : d <= 128 ? 32 : 64, mine = tid % (64 * W), at = (mine % wide) * 4, groups = 64 * W / wide;
  f32x4 o = {0, 0, 0, 0};
  if (at < d) {
    const float* p = a.part + idx * d + at;
#pragma unroll 4
    for (int r = mine / wide; r < runs; r += groups) {
      const f32x4 x = *(const f32x4*)(p + (int64_t)r * d);
      const float f = s_w[team][r];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], f, o[i]);
    }
  }
  if constexpr (W > 1) {
    s_o[tid] = o;
    __syncthreads();
    if (tid < wide)
      for (int g = 1; g < groups; ++g) o += s_o[g * wide + tid];
  } else {
    for (int step = wide; step < 64; step *= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], step);
  }
  if (mine < wide && at < d) {
    T* out = (T*)a.out + row * a.ldo + (int64_t)head * d + at;
    T y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = from_f<T>(sum == 0.0f ? 0.0f : o[i] / sum);
    __builtin_memcpy(out, y, sizeof y);
    if (a.lse && at == 0)
      a.lse[(int64_t)row * a.n_heads + head] = lse_of(best, sum);
  }
}

// ------------------------------------------------------------------ log probabilities -------
//
// A row is cut into pieces of 256 lanes times EL values (by the row's length alone, so that its sums have one order).
// k_scores takes a piece into registers, reads it once, and leaves its maximum, its sums of e = exp(z) and of e z, and the best
// tokens among which the row's k best must be; k_scores_join puts the pieces of a row together. The pieces' bound for the best
// is the k-th largest of 64 maxima of four lanes each (of its first 16 bits); k of them are at least that, and few values
// are above it. (Float32 rows far from 0 share these bits: 257 x 50021 with 20 best 25 us, plus 1000 155, as pieces of more
// than kListed candidates take one best after the other.) 1024 x 131072 bf16: 62 us for k = 8 (4.4 TB/s), 47 for none; the
// join 7 and 5. Slower: workgroups that go on to further pieces with the next one's values on their way (75; 55 for none).

struct ScoreArgs {
  const void* logits;
  const int32_t* tokens;
  float *logp, *entropy, *top_logp;
  int32_t* top_ids;
  float* stats;       // [row][piece] maximum, sums of e and of e z without the maxima, how many best and (from bit 16) maxima
  uint64_t* best;     // [row][piece][kKept] their keys
  int64_t ld;
  int n, given, k, pieces;
  float scale;
};

constexpr int kKept = 64;     // best tokens that a piece hands on
constexpr int kListed = 512;  // and those it can choose them from

__device__ __forceinline__ float masked_logit(float x) {   // NaN is -infinity, infinity the largest number
  return __builtin_fminf(__builtin_fmaxf(x, -__builtin_inff()), 0x1.fffffep127f);
}
// Ordered as the values are, -0 as 0; kMasked and below: -infinity.
constexpr uint32_t kMasked = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __builtin_bit_cast(float, order >> 31 ? order ^ 0x80000000u : ~order);
}
// Larger values first, then lower ids.
__device__ __forceinline__ uint64_t key_of(float x, int id) { return (uint64_t)order_of(masked_logit(x)) << 32 | (uint32_t)~id; }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max64(uint64_t v) {
  const uint64_t u = (uint64_t)dpp0<CTRL, ROWS>((uint32_t)v) | (uint64_t)dpp0<CTRL, ROWS>((uint32_t)(v >> 32)) << 32;
  return u > v ? u : v;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  v = dpp_max64<0x111, 0xF>(v);
  v = dpp_max64<0x112, 0xF>(v);
  v = dpp_max64<0x114, 0xF>(v);
  v = dpp_max64<0x118, 0xF>(v);
  v = dpp_max64<0x142, 0xA>(v);
  v = dpp_max64<0x143, 0xC>(v);
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63) << 32;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int o = 32; o; o /= 2) v += __shfl_xor(v, o);
  return v;
}

// The k best of `list` (n keys that differ, n <= 64 PER) into out, largest first, 0 where there are none left; by one wave.
template <int PER, typename F>
__device__ __forceinline__ void choose(const uint64_t* list, int n, int k, F out) {
  const int lane = threadIdx.x & 63;
  uint64_t v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = i * 64 + lane < n ? list[i * 64 + lane] : 0;
  for (int c = 0; c < k; ++c) {
    uint64_t mine = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mine = v[i] > mine ? v[i] : mine;
    const uint64_t top = wave_max64(mine);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = v[i] == top ? 0 : v[i];
    out(c, top);
  }
}

// z = x c - r in units of log 2, with c the float32 unit and r its reference: the float32 product top c, whose rounding
// the join makes good, or the product itself where that is large.
constexpr float kFused = 0x1p20f;
__device__ __forceinline__ float unit_of(float scale) { return scale * 1.44269504088896340736f; }
__device__ __forceinline__ double reference(float top, float c) {
  const float tc = top * c;
  return __builtin_fabsf(tc) < kFused ? (double)tc : (double)top * (double)c;
}

// Eight neighbouring values as they are in memory.
template <typename T>
struct Eight {
  static constexpr int W = sizeof(T) * 2;
  uint32_t w[W];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[e]);
    else return to_f(__builtin_bit_cast(T, (uint16_t)(w[e / 2] >> (16 * (e & 1)))));
  }
  static __device__ __forceinline__ uint32_t bits_of(float x) {   // of a word of it: one or two of them
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(uint32_t, x);
    else return (uint32_t)__builtin_bit_cast(uint16_t, from_f<T>(x)) * 0x10001u;
  }
  static __device__ __forceinline__ uint32_t none() { return bits_of(-__builtin_inff()); }
  // Values of the bits of `top` become -infinity; returns `bits` and the bits of these values.
  __device__ __forceinline__ int take_out(float top, int bits) {
    const uint32_t t = bits_of(top);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t d = w[i] ^ t;
      uint32_t m;
      if constexpr (sizeof(T) == 4) m = (uint32_t)((int32_t)((d >> 1 | (d & 1)) - 1) >> 31);
      else m = ((uint32_t)((int32_t)((d & 0xFFFFu) - 1) >> 31) & 0xFFFFu) |
               ((uint32_t)((int32_t)((d >> 16) - 1) >> 31) & 0xFFFF0000u);
      w[i] = (w[i] & ~m) | (none() & m);
      bits += __builtin_popcount(m);
    }
    return bits;
  }
  // What follows converts anew rather than keep a register for each value.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
  }
};

template <typename T, int EL>
__global__ __launch_bounds__(256) void k_scores(ScoreArgs a) {
  constexpr int PIECES = EL / 8;
  __shared__ uint32_t s_top[256];
  __shared__ uint64_t s_list[kListed];
  __shared__ float s_sum[2][4];
  __shared__ uint64_t s_key[4];
  __shared__ int s_count, s_tops;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int64_t row = blockIdx.x / a.pieces;
  const int piece = blockIdx.x % a.pieces, from = piece * (256 * EL);
  const T* x = (const T*)a.logits + row * a.ld;
  Eight<T> raw[PIECES];
  if (from + 256 * EL <= a.n) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) __builtin_memcpy(raw[p].w, x + from + p * 2048 + tid * 8, sizeof raw[p].w);
  } else {   // the row's end: eight values that it cuts are loaded one by one, and past it all are -infinity
    const int cut = a.n & ~7;
    Eight<T> last;
    T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_f<T>(-__builtin_inff());
    if (((cut - from) / 8 & 255) == tid) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (cut + e < a.n) v[e] = x[cut + e];
    }
    __builtin_memcpy(last.w, v, sizeof v);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int i = from + p * 2048 + tid * 8;
      if (i < cut) {
        __builtin_memcpy(raw[p].w, x + i, sizeof raw[p].w);
      } else {
#pragma unroll
        for (int w = 0; w < Eight<T>::W; ++w) raw[p].w[w] = i == cut ? last.w[w] : Eight<T>::none();
      }
    }
  }
  if (tid == 0) s_count = s_tops = 0;
  float mine = -__builtin_inff();
#pragma unroll
  for (int p = 0; p < PIECES; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) mine = __builtin_fmaxf(mine, raw[p].at(e));
  mine = __builtin_fminf(mine, 0x1.fffffep127f);
  const uint32_t my_order = order_of(mine);
  s_top[tid] = my_order;
  __syncthreads();
  const uint32_t four = max(max(s_top[lane], s_top[64 + lane]), max(s_top[128 + lane], s_top[192 + lane]));
  const uint32_t most = wave_max(four);
  const bool none = most <= kMasked;
  const float top = none ? 0.0f : value_of(most);

  // Infinity counts as the largest number. (In 16 bits that number is infinity, which the next step takes out.)
  if constexpr (sizeof(T) == 4) {
    if (top == 0x1.fffffep127f) {
#pragma unroll
      for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[p].w[e] = raw[p].w[e] == 0x7F800000u ? 0x7F7FFFFFu : raw[p].w[e];
    }
  }

  // A row that is sure of a token has a sum of 1 and little more, and that little is what its entropy hangs on: the lanes
  // that have the maximum take it out (any number of times; +0 for -0 stays, with which nothing is lost), and
  // the join counts the maxima. Without branches or masks, which cost registers: 53 us for the 1024 x 131072 without
  // this, 62 with it, 82 by a second pass over the lane's values.
  if (mine == top && !none) {
    int bits = 0;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) bits = raw[p].take_out(top, bits);
    atomicAdd(&s_tops, bits / (8 * (int)sizeof(T)));
  }

  // below -200 (masked tokens too) z counts as that, and e is 0
  const float c = unit_of(a.scale), tc = top * c;
  float sum = 0.0f, dot = 0.0f;
  if (__builtin_fabsf(tc) < kFused) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      raw[p].forget();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = __builtin_fmaxf(__builtin_fmaf(raw[p].at(e), c, -tc), -200.0f);
        const float y = __builtin_amdgcn_exp2f(z);
        sum += y;
        dot = __builtin_fmaf(y, z, dot);
      }
    }
  } else {   // the rounding of tc counts, or it is out of range: the difference first
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      raw[p].forget();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = __builtin_fmaxf((masked_logit(raw[p].at(e)) - top) * c, -200.0f);
        const float y = __builtin_amdgcn_exp2f(z);
        sum += y;
        dot = __builtin_fmaf(y, z, dot);
      }
    }
  }
  sum = wave_sum_f(sum);
  dot = wave_sum_f(dot);
  if (lane == 0) s_sum[0][wave] = sum, s_sum[1][wave] = dot;

  uint32_t bound = kMasked >> 16;
  if (a.k > 0 && !none) {
    uint32_t t = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
      const uint32_t next = (t | 1u << b) << 16;
      if (__popcll(__ballot(four >= next)) >= a.k) t |= 1u << b;
    }
    bound = max(t, (kMasked >> 16) + 1);
    // the values of the lanes that have some, a lane's by the wave, four lanes at a time
    for (uint64_t hot = __ballot(my_order >> 16 >= bound); hot;) {
      float v[4];
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = hot ? __builtin_ctzll(hot) : 0;
        id[j] = from + (lane >> 3) * 2048 + (wave * 64 + h) * 8 + (lane & 7);
        const bool in = hot && lane < EL && id[j] < a.n;
        v[j] = in ? to_f(x[id[j]]) : -__builtin_inff();
        hot &= hot - 1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t key = key_of(v[j], id[j]);
        if (key >> 48 >= bound) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kListed) s_list[at] = key;
        }
      }
    }
  }
  __syncthreads();
  float* stats = a.stats + (int64_t)blockIdx.x * 4;
  uint64_t* best = a.best + (int64_t)blockIdx.x * kKept;
  const int count = s_count;
  if (tid == 0) {
    stats[0] = none ? -__builtin_inff() : top;
    stats[1] = none ? 0.0f : (s_sum[0][0] + s_sum[0][1]) + (s_sum[0][2] + s_sum[0][3]);
    stats[2] = none ? 0.0f : (s_sum[1][0] + s_sum[1][1]) + (s_sum[1][2] + s_sum[1][3]);
    stats[3] = __builtin_bit_cast(float, (count <= kKept ? count : a.k) | s_tops << 16);
  }
  if (count <= kKept) {
    if (tid < count) best[tid] = s_list[tid];
  } else if (count <= kListed) {
    if (wave == 0) choose<kListed / 64>(s_list, count, a.k, [&](int i, uint64_t key) {
      if (lane == 0) best[i] = key;
    });
  } else {   // many equal values: one after the other
    uint64_t last = ~0ull;
    for (int i = 0; i < a.k; ++i) {
      uint64_t next = 0;
      for (int at = from + tid; at < min(a.n, from + 256 * EL); at += 256) {
        const uint64_t key = key_of(to_f(x[at]), at);
        if (key < last && key > next) next = key;
      }
      next = wave_max64(next);
      if (lane == 0) s_key[wave] = next;
      __syncthreads();
      last = max(max(s_key[0], s_key[1]), max(s_key[2], s_key[3]));
      __syncthreads();
      if (tid == 0) best[i] = last;
    }
  }
}

// A wave a row.
template <typename T>
__global__ __launch_bounds__(64) void k_scores_join(ScoreArgs a) {
  __shared__ uint64_t s_list[kListed + 64];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x;
  const T* x = (const T*)a.logits + row * a.ld;
  const float* stats = a.stats + row * a.pieces * 4;
  const float c = unit_of(a.scale);
  float top = -__builtin_inff();
  for (int p = lane; p < a.pieces; p += 64) top = __builtin_fmaxf(top, stats[4 * p]);
#pragma unroll
  for (int o = 32; o; o /= 2) top = __builtin_fmaxf(top, __shfl_xor(top, o));
  const bool none = top == -__builtin_inff();
  const double ref = none ? 0.0 : reference(top, c), ln2 = 0.6931471805599453;
  double sum = 0.0, dot = 0.0;
  for (int p = lane; p < a.pieces; p += 64) {
    const float m = stats[4 * p];
    if (m == -__builtin_inff()) continue;
    // the maxima's z, which the rounding of the reference leaves a little off 0, and their share
    const double off = (double)m * (double)c - reference(m, c);
    const double tops = (double)(__builtin_bit_cast(int, stats[4 * p + 3]) >> 16) * exp64(off * ln2);
    const double z = reference(m, c) - ref, f = exp64(z * ln2), s = (double)stats[4 * p + 1] + tops;
    sum = __builtin_fma(s, f, sum);
    dot = __builtin_fma(f, __builtin_fma(s, f > 0.0 ? z : 0.0, __builtin_fma(tops, off, (double)stats[4 * p + 2])), dot);
  }
  sum = wave_sum(sum);
  dot = wave_sum(dot);
  const double log_sum = none ? 0.0 : log(sum), base = none ? 0.0 : (double)top;
  const double rest = ((base * (double)c) - ref) * ln2 - log_sum;
  // rest may be 2^-53 above 0
  auto logp_of = [&](float v) { return (float)__builtin_fmin(((double)v - base) * (double)a.scale + rest, 0.0); };
  if (lane == 0 && a.entropy) a.entropy[row] = none ? 0.0f : (float)__builtin_fmax(log_sum - dot / sum * ln2, 0.0);
  if (lane < a.given) {
    const int id = a.tokens[row * a.given + lane];
    a.logp[row * a.given + lane] = logp_of(id >= 0 && id < a.n ? masked_logit(to_f(x[id])) : -__builtin_inff());
  }
  if (a.k == 0) return;
  // the pieces' best, eight pieces at a time
  int have = 0;
  uint64_t mine = 0;   // of the k best, lane by lane
  auto choose_from = [&]() {
    mine = 0;
    auto take = [&](int i, uint64_t key) { mine = lane == i ? key : mine; };
    __syncthreads();
    if (have <= 64) choose<1>(s_list, have, a.k, take);
    else if (have <= 128) choose<2>(s_list, have, a.k, take);
    else if (have <= 256) choose<4>(s_list, have, a.k, take);
    else choose<(kListed + 64) / 64>(s_list, have, a.k, take);
    __syncthreads();
    if (lane < a.k) s_list[lane] = mine;
    have = __popcll(__ballot(lane < a.k && mine != 0));
  };
  for (int p0 = 0; p0 < a.pieces; p0 += 64) {
    const int counts = p0 + lane < a.pieces ? __builtin_bit_cast(int, stats[4 * (p0 + lane) + 3]) & 0xFFFF : 0;
    const uint64_t* best = a.best + (row * a.pieces + p0) * kKept;
    for (int p = 0; p < 64 && p0 + p < a.pieces; p += 8) {
      uint64_t key[8];
      int count[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        count[i] = __builtin_amdgcn_readlane(counts, p + i);
        key[i] = lane < count[i] ? best[(p + i) * kKept + lane] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (have + count[i] > kListed + 64) choose_from();
        if (lane < count[i]) s_list[have + lane] = key[i];
        have += count[i];
      }
    }
  }
  choose_from();
  __syncthreads();
  if (lane < have) {
    const uint64_t key = s_list[lane];
    a.top_ids[row * a.k + lane] = (int)~(uint32_t)key;
    a.top_logp[row * a.k + lane] = logp_of(value_of((uint32_t)(key >> 32)));
  }
  for (int i = 0; have < a.k && i < a.n; i += 64) {   // then masked tokens, lowest id first
    const bool masked = i + lane < a.n && order_of(masked_logit(to_f(x[i + lane < a.n ? i + lane : 0]))) <= kMasked;
    const uint64_t all = __ballot(masked);
    const int at = have + __popcll(all & ((1ull << lane) - 1));
    if (masked && at < a.k) {
      a.top_ids[row * a.k + at] = i + lane;
      a.top_logp[row * a.k + at] = -__builtin_inff();
    }
    have += __popcll(all);
  }
}

// ------------------------------------------------------------------ host checks -------------

constexpr float kMaxScale = 0x1p127f;   // times log2(e), the unit of the exponentials, still a float32

// Rows of a cache in memory, in bytes from k: whether they lie apart, and the bytes from the first to the last.
struct Extent {
  bool ok;
  int64_t bytes;
};
Extent cache_extent(const moe_kv_cache& c) {
  const int size = c.dtype == MOE_I8 ? 1 : 2;
  const uintptr_t k = (uintptr_t)c.k, v = (uintptr_t)c.v;
  const int64_t apart = (int64_t)(v > k ? v - k : k - v);
  struct {
    int64_t count, step;
  } dim[] = {{c.n_pages, c.page_stride}, {c.n_kv, c.head_stride}, {c.page_size, c.slot_stride}};
  for (auto& x : dim) {
    if (x.count == 1) x.step = 0;
    else if (x.step < 16 || x.step % 16 || x.step > MOE_MAX_SPAN / x.count) return {false, 0};
    x.step *= size;
  }
  std::sort(dim, dim + 3, [](auto& a, auto& b) { return a.step < b.step; });
  // each stride past all that the smaller ones span; so is the way from k to v, wherever it comes among them
  int64_t span = (int64_t)c.head_dim * size;
  bool both = false;
  for (auto& x : dim) {
    if (x.count == 1) continue;
    if (!both && apart < x.step) {
      if (apart < span) return {false, 0};
      span += apart;
      both = true;
    }
    if (x.step < span) return {false, 0};
    span += (x.count - 1) * x.step;
  }
  if (!both) {
    if (apart < span) return {false, 0};
    return {true, span};
  }
  return {true, span - apart};   // of k alone, and of v alone
}

int check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_E_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_F16 && c->dtype != MOE_I8) return MOE_E_ARG;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size > MOE_MAX_PAGE || c->page_size % 16 || c->n_kv < 1 ||
      c->n_kv > MOE_MAX_HEADS || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
    return MOE_E_SHAPE;
  if (c->page_size > 1 && c->slot_stride > 1 << 24) return MOE_E_SHAPE;   // 16 rows within 32 bits of bytes
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16) || !cache_extent(*c).ok) return MOE_E_ARG;
  if (c->dtype == MOE_I8) {
    if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return MOE_E_ARG;
    const int64_t n = (int64_t)c->n_pages * c->n_kv * c->page_size;
    const int64_t bytes = cache_extent(*c).bytes;
    const Rows apart[] = {rows_of(c->k_scale, 1, n, n, 4), rows_of(c->v_scale, 1, n, n, 4), rows_of(c->k, 1, bytes, bytes, 1),
                          rows_of(c->v, 1, bytes, bytes, 1)};
    for (int i = 1; i < 4; ++i)   // k and v may share their span (cache_extent has looked at their rows)
      for (int j = 0; j < std::min(i, 2); ++j)
        if (overlap(apart[i], apart[j])) return MOE_E_ARG;
  } else if (c->k_scale || c->v_scale) {
    return MOE_E_ARG;
  }
  return MOE_OK;
}

int check_window(const moe_window* w, const moe_kv_cache& c) {
  if (!w || w->n_seqs < 0 || w->n_tokens < 0) return MOE_E_ARG;
  if (w->n_seqs > MOE_MAX_SEQS || w->n_tokens > MOE_MAX_ROWS) return MOE_E_SHAPE;
  if (w->n_seqs == 0 || w->n_tokens == 0) return MOE_OK;
  if (w->max_window < 1 || w->max_pages < 1 || (int64_t)w->max_pages * c.page_size > 0x7FFFFFFF) return MOE_E_SHAPE;
  if (!w->row_start || !w->ctx_len || !w->pages || !w->err || bad_stride(w->ld_pages, w->max_pages, w->n_seqs)) return MOE_E_ARG;
  if (!aligned(w->row_start, 4) || !aligned(w->ctx_len, 4) || !aligned(w->pages, 4) || !aligned(w->pos, 4) ||
      !aligned(w->seen, 8) || !aligned(w->err, 4))
    return MOE_E_ARG;
  return MOE_OK;
}

constexpr int kCacheSpans = 4;
void cache_spans(const moe_kv_cache& c, Rows (&out)[kCacheSpans]) {
  const int64_t bytes = cache_extent(c).bytes, scales = (int64_t)c.n_pages * c.n_kv * c.page_size;
  out[0] = rows_of(c.k, 1, bytes, bytes, 1);
  out[1] = rows_of(c.v, 1, bytes, bytes, 1);
  out[2] = rows_of(c.k_scale, 1, scales, scales, 4);
  out[3] = rows_of(c.v_scale, 1, scales, scales, 4);
}
constexpr int kWindowSpans = 6;
void window_spans(const moe_window& w, Rows (&out)[kWindowSpans]) {
  out[0] = rows_of(w.row_start, 1, w.n_seqs + 1, 0, 4);
  out[1] = rows_of(w.ctx_len, 1, w.n_seqs, 0, 4);
  out[2] = rows_of(w.pages, w.n_seqs, w.max_pages, w.ld_pages, 4);
  out[3] = rows_of(w.pos, 1, w.n_tokens, 0, 4);
  out[4] = rows_of(w.seen, 1, w.n_tokens, 0, 8);
  out[5] = rows_of(w.err, 1, 1, 0, 4);
}
template <int N>
bool over(const Rows& r, const Rows (&all)[N]) {
  for (const Rows& x : all)
    if (overlap(r, x)) return true;
  return false;
}

CacheArgs cache_args(const moe_kv_cache& c) {
  return CacheArgs{(uint8_t*)c.k, (uint8_t*)c.v, c.k_scale, c.v_scale, c.page_stride, c.head_stride, c.slot_stride,
                   c.n_pages, c.page_size, c.n_kv, c.head_dim};
}
WindowArgs window_args(const moe_window& w, const moe_kv_cache& c) {
  return WindowArgs{w.row_start, w.ctx_len, w.pages, w.pos, w.seen, w.err, w.ld_pages, w.n_seqs, w.n_tokens, w.max_window,
                    w.max_pages * c.page_size};
}

// Rows that share a cache head, at most.
int most_rows(const moe_kv_cache& c, const moe_window& w, int n_heads) { return w.max_window * (n_heads / c.n_kv); }
// The least keys of a run, by how many sequences, cache heads and tiles of 128 rows there are to spread over the card. Launches
// and kernels, us in runs of 256 / 512 / 1024 (2048), bf16. One token, four or eight query heads a cache head: 16 units over
// 1000 keys 14.0 / 16.2 / 16.7, over 16000 32.0 / 29.6 / 29.7; 32 units 13.9 / 16.1 / 16.5 and 52 / 49 / 49; 48 units
// 14.2 / 16.5 / 16.6 and 90 / 84 / 90; 128 units 21.7 / 21.5 / 18.5 and 224 / 204 / 197; 192 units 29.6 / 27.1 / 22.0 and
// 330 / 302 / 291. Trees of 64 tokens x 8 heads: 32 units 31 / 38 / 57 and 126 / 98 / 83 (103); 128 units 65 / 53 / 65 and
// 520 / 361 / 287 (257); 256 units 96 / 93 / 88 (60) and 991 / 709 / 574 (504). So it leans to short contexts: long ones, of
// trees above all, would take longer runs, whose results are fewer.
int least_run(const moe_kv_cache& c, const moe_window& w, int n_heads) {
  const int64_t units = (int64_t)w.n_seqs * c.n_kv * ((most_rows(c, w, n_heads) + 127) / 128);
  return units <= 32 ? 256 : units <= 128 ? 512 : 1024;
}
int max_runs(const moe_kv_cache& c, const moe_window& w, int n_heads) {
  const int least = least_run(c, w, n_heads);
  return (int)std::min<int64_t>(((int64_t)w.max_pages * c.page_size + least - 1) / least, kMaxRuns);
}

// Tokens whose heads are spread over several workgroups (above: four tokens a workgroup). A sequence of 32 + 2 x 8 heads of 128,
// bf16, launch and kernel: 512 tokens 10.8 us spread, 19.7 by fours; 1024 16.6, 20.6; 1536 23.2, 25.9; 2048 30.7, 27.2; 8192
// 101, 62. Of 8 + 2 x 1 heads: 1024 6.6, 9.0; 1536 9.6, 10.0; 2048 10.7, 10.4. Tokens that are sequences of their own, where
// each workgroup looks for its sequence: 640 15.0, 22.0; 1024 23.5, 24.3; 1500 34.3, 29.7.
constexpr int kAppendFew = 1536;
// Rows and heads whose runs are joined by four waves each, above by one: 32 rows of 63 runs 4.9 us by four, 6.1 by one; 512 of 64
// 6.5, 6.7; 1024 8.8, 8.5; 8192 of some 6 16.4, 8.4.
constexpr int kJoinWide = 1024;

// Attention's sizes beside those of the cache and the window, for the call and for the size of its workspace.
int check_attend(const moe_kv_cache& c, const moe_window& w, int n_heads) {
  if (n_heads < 1 || n_heads > MOE_MAX_HEADS || n_heads % c.n_kv) return MOE_E_SHAPE;
  if (w.n_seqs == 0 || w.n_tokens == 0) return MOE_OK;
  if (w.max_window > MOE_MAX_WINDOW) return MOE_E_SHAPE;
  if (max_runs(c, w, n_heads) > 1 && (int64_t)w.n_tokens * n_heads > MOE_MAX_JOIN) return MOE_E_SHAPE;
  return MOE_OK;
}
static_assert(MOE_MAX_JOIN / 4 * 256ll <= kLaunchThreads && MOE_MAX_JOIN % 4 == 0 && kJoinWide * 256ll <= kLaunchThreads);

template <typename T, bool I8, int HD, int NT, bool WIDE>
int launch_attend(hipStream_t st, const AttendArgs& a) {
  constexpr int ROWS = 16 * NT * (WIDE ? 4 : 1);
  const int64_t tiles = ((int64_t)a.w.max_window * (a.n_heads / a.c.n_kv) + ROWS - 1) / ROWS;
  const int64_t items = tiles * a.max_runs * a.c.n_kv * a.w.n_seqs;   // at most 2048 * 64 * 4096
  const int grid = (int)std::min<int64_t>(256 * kAttendWaves(HD), (items + 7) & ~7ll);
  const int lds = (WIDE ? ring_bytes(HD, I8) : 0) + 4 * a.w.n_seqs;
  const auto kern = k_attend<T, I8, HD, NT, WIDE>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return hip_fail(e, "moe_window_attention");
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(256), lds, st, a);
  if (const int rc = launched("moe_window_attention")) return rc;
  if (a.max_runs > 1) {
    const int64_t rows = (int64_t)a.w.n_tokens * a.n_heads;
    if (rows <= kJoinWide) hipLaunchKernelGGL((k_attend_join<T, 4>), dim3((unsigned)rows), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_attend_join<T, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
    return launched("moe_window_attention");
  }
  return MOE_OK;
}
template <typename T>
int run_attend(hipStream_t st, const AttendArgs& a, bool i8) {
  const int rows = a.w.max_window * (a.n_heads / a.c.n_kv);
  auto tiles = [&](auto i, auto hd) {
    constexpr bool I8 = decltype(i)::value;
    constexpr int HD = decltype(hd)::value;
    // Launches and kernels, us of 32 sequences over 4000 keys, bf16 and int8. 16 rows a cache head: one tile a wave 50 and 34,
    // two 52 and 40. 20 rows: two tiles 54 and 41, one in two workgroups 65 and 54 (of one sequence over 60000 keys 34, 33). 40
    // rows: wide 65 and 76, two tiles in two workgroups 76 and 72 (one sequence 47, 37). 64 rows: wide of one tile 72 and 82,
    // of two 83 and 96; 128 rows: wide of two 105 and 114, of one 127 and 151. 32 rows of heads of 256 over 2000 keys: two
    // tiles 91, one in two workgroups 80.
    constexpr int MOST = HD == 256 && !I8 ? 1 : 2;   // tiles that a wave of the wide kernel has registers for
    if (rows > 32) return rows <= 64 ? launch_attend<T, I8, HD, 1, true>(st, a) : launch_attend<T, I8, HD, MOST, true>(st, a);
    return rows <= 16 ? launch_attend<T, I8, HD, 1, false>(st, a) : launch_attend<T, I8, HD, 2, false>(st, a);
  };
  auto width = [&](auto i) {
    using std::integral_constant;
    if (a.c.d <= 64) return tiles(i, integral_constant<int, 64>{});
    if (a.c.d <= 128) return tiles(i, integral_constant<int, 128>{});
    return tiles(i, integral_constant<int, 256>{});
  };
  return i8 ? width(std::true_type{}) : width(std::false_type{});
}

// Values of a lane: 32 spread short rows over more workgroups. Launches and kernels with 8 best, us by 32 and by 64: 1024 rows of
// bf16 20000 21.2, 24.0; 50021 35.1, 37.0; 65536 37.5, 36.6; 80000 45.0, 42.2; 131072 63.9, 59.1; one row of 32000 9.8, 10.5;
// 262144 13.7, 12.2. float32: 1024 x 50021 43.4, 50.0; 1024 x 131072 104, 112; 64 x 262144 25.8, 24.1; one row of
// 262144 13.9, 13.0.
constexpr int kShortRow = 65536, kLongEl = 64;
int pieces_of(int n) { return n <= kShortRow ? (n + 8191) / 8192 : (n + 256 * kLongEl - 1) / (256 * kLongEl); }
// The sizes of log probabilities, for the call and for the size of its workspace.
int check_scores(int rows, int n) {
  if (rows > MOE_MAX_ROWS || n < 1 || n > MOE_MAX_VOCAB || (int64_t)rows * pieces_of(n) > MOE_MAX_PIECES) return MOE_E_SHAPE;
  return MOE_OK;
}
static_assert(MOE_MAX_PIECES * 256ll <= kLaunchThreads);

}  // namespace moe

using namespace moe;

// ------------------------------------------------------------------ C ABI -------------------

extern "C" {

int moe_window_append(void* stream, const moe_kv_cache* C, const moe_window* W, int dtype, const void* q, int64_t ldq,
                      const void* k, int64_t ldk, const void* v, int64_t ldv, int n_heads, int w_dtype, const void* q_weight,
                      const void* k_weight, float eps, const float* freq, int n_rot, int layout, double amp, int o_dtype,
                      void* q_out, int64_t ldqo) {
  if (const int rc = check_cache(C)) return rc;
  if (const int rc = check_window(W, *C)) return rc;
  if (!type_ok(dtype) || !q != !q_out || (q && !type_ok(o_dtype))) return MOE_E_ARG;
  if ((q_weight || k_weight) && (!type_ok(w_dtype) || !(eps > 0.0f) || !(eps < __builtin_inff()))) return MOE_E_ARG;
  if (!(__builtin_fabs(amp) < __builtin_inff()) || (layout != MOE_ROPE_HALF && layout != MOE_ROPE_PAIRS)) return MOE_E_ARG;
  const int d = C->head_dim, n = W->n_tokens;
  if (n_rot < 0 || n_rot > d || n_rot % 2) return MOE_E_SHAPE;
  if (q && (n_heads < 1 || n_heads > MOE_MAX_HEADS || n_heads % C->n_kv)) return MOE_E_SHAPE;
  if (W->n_seqs == 0 || n == 0) return MOE_OK;
  const int64_t wide = (int64_t)n_heads * d, kv = (int64_t)C->n_kv * d;
  if (!k || !v || (n_rot && !freq) || bad_stride(ldk, kv, n) || bad_stride(ldv, kv, n)) return MOE_E_ARG;
  if (q && (bad_stride(ldq, wide, n) || bad_stride(ldqo, wide, n))) return MOE_E_ARG;
  const int sz = type_size(dtype), szo = type_size(o_dtype), szw = type_size(w_dtype);
  if (!aligned(q, sz) || !aligned(k, sz) || !aligned(v, sz) || (q_weight && !aligned(q_weight, szw)) ||
      (k_weight && !aligned(k_weight, szw)) || !aligned(freq, 4) || (q && !aligned(q_out, szo)))
    return MOE_E_ARG;
  Rows spans[kCacheSpans], window[kWindowSpans];
  cache_spans(*C, spans);
  window_spans(*W, window);
  const Rows in[] = {rows_of(q, n, wide, ldq, sz), rows_of(k, n, kv, ldk, sz), rows_of(v, n, kv, ldv, sz),
                     rows_of(q_weight, 1, d, d, szw), rows_of(k_weight, 1, d, d, szw), rows_of(freq, 1, n_rot / 2, 0, 4)};
  const Rows out = rows_of(q_out, n, wide, ldqo, szo);
  for (int i = 0; i < 6; ++i) {
    if (over(in[i], spans) || overlap(in[i], window[5])) return MOE_E_ARG;
    if (overlap(out, in[i]) && !(i == 0 && q_out == q && out.step == in[0].step && o_dtype == dtype)) return MOE_E_ARG;
  }
  if (over(out, spans) || over(out, window)) return MOE_E_ARG;
  for (const Rows& r : window)
    if (over(r, spans)) return MOE_E_ARG;
  for (int i = 0; i < 5; ++i)
    if (overlap(window[i], window[5])) return MOE_E_ARG;
  const int heads = q ? n_heads : 0, all = heads + 2 * C->n_kv;
  const int lanes = std::max((d + 7) / 8, (n_rot + 7) / 8 + (d - n_rot + 7) / 8);
  const int lg = lanes <= 8 ? 8 : lanes <= 16 ? 16 : lanes <= 32 ? 32 : 64;
  const int units = n <= kAppendFew ? 256 / lg : all;
  const AppendArgs a{cache_args(*C), window_args(*W, *C), q, k, v, q_weight, k_weight, freq, q_out, ldq, ldk, ldv, ldqo,
                     heads, n_rot, layout, w_dtype, o_dtype, C->dtype, units, eps, amp};
  with_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto l) {
      constexpr int LG = decltype(l)::value;
      const hipStream_t st = (hipStream_t)stream;
      const int parts = (all + units - 1) / units;
      if (n <= kAppendFew) hipLaunchKernelGGL((k_window_append<T, LG, 1>), dim3(n, parts), dim3(256), 0, st, a);
      else hipLaunchKernelGGL((k_window_append<T, LG, 4>), dim3((n + 3) / 4), dim3(256), 0, st, a);
    };
    using std::integral_constant;
    if (lg == 8) go(integral_constant<int, 8>{});
    else if (lg == 16) go(integral_constant<int, 16>{});
    else if (lg == 32) go(integral_constant<int, 32>{});
    else go(integral_constant<int, 64>{});
  });
  return launched("moe_window_append");
}

size_t moe_window_attention_bytes(const moe_kv_cache* C, const moe_window* W, int n_heads) {
  if (check_cache(C) || check_window(W, *C) || check_attend(*C, *W, n_heads)) return 0;
  const size_t runs = W->n_seqs && W->n_tokens ? max_runs(*C, *W, n_heads) : 1;
  return runs == 1 ? 16 : ((size_t)W->n_tokens * n_heads * runs * (C->head_dim + 2) * 4 + 15) & ~(size_t)15;
}

int moe_window_attention(void* stream, const moe_kv_cache* C, const moe_window* W, int dtype, const void* q, int64_t ldq,
                         int n_heads, float scale, void* out, int64_t ldo, float* lse, void* workspace, size_t ws_bytes) {
  if (const int rc = check_cache(C)) return rc;
  if (const int rc = check_window(W, *C)) return rc;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_E_ARG;
  if ((C->dtype != MOE_I8 && C->dtype != dtype) || !(__builtin_fabsf(scale) <= kMaxScale)) return MOE_E_ARG;
  if (const int rc = check_attend(*C, *W, n_heads)) return rc;
  const int n = W->n_tokens;
  if (W->n_seqs == 0 || n == 0) return MOE_OK;
  const int64_t wide = (int64_t)n_heads * C->head_dim;
  if (!q || !out || bad_stride(ldq, wide, n) || bad_stride(ldo, wide, n)) return MOE_E_ARG;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4)) return MOE_E_ARG;
  const size_t need = moe_window_attention_bytes(C, W, n_heads);
  if (!workspace || ws_bytes < need || !aligned(workspace, 16)) return MOE_E_WS;
  Rows spans[kCacheSpans], window[kWindowSpans];
  cache_spans(*C, spans);
  window_spans(*W, window);
  const Rows in = rows_of(q, n, wide, ldq, 2);
  const Rows outs[] = {rows_of(out, n, wide, ldo, 2), rows_of(lse, 1, (int64_t)n * n_heads, 0, 4),
                       rows_of(workspace, 1, (int64_t)need, 0, 1), window[5]};
  for (int i = 0; i < 4; ++i) {
    if (overlap(outs[i], in) || over(outs[i], spans)) return MOE_E_ARG;
    for (int j = 0; j < 5; ++j)
      if (overlap(outs[i], window[j])) return MOE_E_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_E_ARG;
  }
  const int runs = max_runs(*C, *W, n_heads);
  AttendArgs a{cache_args(*C), window_args(*W, *C), q, out, lse, (float*)workspace, nullptr, ldq, ldo, n_heads, runs,
               least_run(*C, *W, n_heads), scale};
  a.part_ml = a.part + (int64_t)n * n_heads * runs * C->head_dim;
  return dtype == MOE_BF16 ? run_attend<bf16_t>((hipStream_t)stream, a, C->dtype == MOE_I8)
                           : run_attend<f16_t>((hipStream_t)stream, a, C->dtype == MOE_I8);
}

size_t moe_token_logprobs_bytes(int rows, int n, int k) {
  if (rows < 1 || k < 0 || k > 32 || k > n || check_scores(rows, n)) return 0;
  return (size_t)rows * pieces_of(n) * (16 + (k ? 8 * kKept : 0));
}

int moe_token_logprobs(void* stream, int dtype, const void* logits, int64_t ld, int rows, int n, float scale,
                       const int32_t* tokens, int given, float* logp, float* entropy, int k, int32_t* top_ids,
                       float* top_logp, void* workspace, size_t ws_bytes) {
  if (!type_ok(dtype) || rows < 0 || given < 0 || given > 64 || k < 0 || k > 32 || !(scale > 0.0f) || !(scale <= kMaxScale))
    return MOE_E_ARG;
  if (const int rc = check_scores(rows, n)) return rc;
  if (k > n) return MOE_E_ARG;
  if (rows == 0) return MOE_OK;
  if (!logits || bad_stride(ld, n, rows) || !tokens != !given || !logp != !given || !top_ids != !k || !top_logp != !k ||
      (!given && !entropy && !k))
    return MOE_E_ARG;
  if (!aligned(logits, type_size(dtype)) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return MOE_E_ARG;
  const size_t need = moe_token_logprobs_bytes(rows, n, k);
  if (!workspace || ws_bytes < need || !aligned(workspace, 16)) return MOE_E_WS;
  const Rows in[] = {rows_of(logits, rows, n, ld, type_size(dtype)), rows_of(tokens, 1, (int64_t)rows * given, 0, 4)};
  const Rows outs[] = {rows_of(logp, 1, (int64_t)rows * given, 0, 4), rows_of(entropy, 1, rows, 0, 4),
                       rows_of(top_ids, 1, (int64_t)rows * k, 0, 4), rows_of(top_logp, 1, (int64_t)rows * k, 0, 4),
                       rows_of(workspace, 1, (int64_t)need, 0, 1)};
  for (int i = 0; i < 5; ++i) {
    if (over(outs[i], in)) return MOE_E_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_E_ARG;
  }
  const int pieces = pieces_of(n);
  const int64_t blocks = (int64_t)rows * pieces;
  float* const stats = (float*)workspace;
  const ScoreArgs a{logits, tokens, logp, entropy, top_logp, top_ids, stats, (uint64_t*)(stats + 4 * blocks), ld, n, given, k,
                    pieces, scale};
  with_type(dtype, [&](auto t) {
    using T = decltype(t);
    if (n <= kShortRow) hipLaunchKernelGGL((k_scores<T, 32>), dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL((k_scores<T, kLongEl>), dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
    hipLaunchKernelGGL(k_scores_join<T>, dim3(rows), dim3(64), 0, (hipStream_t)stream, a);
  });
  return launched("moe_token_logprobs");
}

}  // extern "C"
