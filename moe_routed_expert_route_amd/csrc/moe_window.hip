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
// The sequence that a row is of (the last that starts at or before it: one without tokens is passed over); tokens = 0:
// none, or one that is left out. Uniform over the wave: a lane looks at one start in 64.
__device__ __forceinline__ Seq seq_of(const WindowArgs& w, int row, int most) {
  int n = 0;
  for (int i = 0; i < w.n_seqs; i += 64) {
    const int at = i + (int)(threadIdx.x & 63);
    n += __popcll(__ballot(at < w.n_seqs && w.row_start[at < w.n_seqs ? at : 0] <= row));
  }
  n = __builtin_amdgcn_readfirstlane(n);
  if (n == 0) return Seq{0, 0, 0, 0};
  const int start = w.row_start[n - 1], end = w.row_start[n], ctx = w.ctx_len[n - 1];
  if (row >= end || !seq_ok(w, start, end, ctx, most)) return Seq{0, 0, 0, 0};
  return Seq{n - 1, start, end - start, ctx};
}
// One workgroup of a launch looks at every sequence.
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
  float eps, amp;
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

// A head's row is with LG neighbouring lanes, eight values each: four pairs (of MOE_ROPE_HALF: four values and their
// four partners), or eight values that do not turn.
template <typename T, int LG>
__global__ __launch_bounds__(256) void k_window_append(AppendArgs a) {
  constexpr int GROUPS = 256 / LG;
  __shared__ double s_turn[128][2];
  const int row = blockIdx.x, l = threadIdx.x % LG, d = a.c.d;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(a.w, 0x7FFFFFFF, 256);
  const Seq q = seq_of(a.w, row, 0x7FFFFFFF);
  if (q.tokens == 0) return;
  const int key = q.ctx + row - q.start, slot = key % a.c.page_size;
  const int page = a.w.pages[q.s * a.w.ld_pages + key / a.c.page_size];
  const bool page_ok = page >= 0 && page < a.c.n_pages;
  if (!page_ok && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.w.err, MOE_ERR_PAGE);
  const int half = a.n_rot / 2;
  if ((int)threadIdx.x < half) {
    double c, s;
    turn64((double)(a.w.pos ? a.w.pos[row] : key) * (double)a.freq[threadIdx.x], c, s);
    s_turn[threadIdx.x][0] = (double)a.amp * c;
    s_turn[threadIdx.x][1] = (double)a.amp * s;
  }
  __syncthreads();
  const int first = blockIdx.y * a.units, last = min(first + a.units, a.n_heads + 2 * a.c.n_kv);
  for (int u = first + (int)threadIdx.x / LG; u < last; u += GROUPS) {
    const bool is_q = u < a.n_heads, is_v = u >= a.n_heads + a.c.n_kv;
    const int h = is_q ? u : (u - a.n_heads) % a.c.n_kv;
    const T* x = is_q ? (const T*)a.q + row * a.ldq : is_v ? (const T*)a.v + row * a.ldv : (const T*)a.k + row * a.ldk;
    x += (int64_t)h * d;
    // this lane's values: n0 from at0 on, n1 from at1 on
    const int rot = is_v ? 0 : a.n_rot, turning = (rot + 7) / 8;
    const bool turns = l < turning, halves = turns && a.layout == MOE_ROPE_HALF;
    const int at0 = halves ? 4 * l : turns ? 8 * l : rot + 8 * (l - turning);
    const int at1 = halves ? half + 4 * l : at0 + 4, end = turns ? rot : d;
    const int n0 = (halves ? half : end) - at0, n1 = end - at1;
    T raw[2][4];
    load4(x + at0, n0, raw[0]);
    load4(x + at1, n1, raw[1]);
    double y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (double)to_f(raw[e / 4][e % 4]);
    const void* weight = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
    if (weight) {
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fma(y[e], y[e], sum);
#pragma unroll
      for (int o = LG / 2; o; o /= 2) sum += __shfl_xor(sum, o);
      const double rinv = 1.0 / __builtin_sqrt(sum / d + (double)a.eps);
      float w[8];
      load4(weight, a.w_dtype, at0, n0, w);
      load4(weight, a.w_dtype, at1, n1, w + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rinv * (double)w[e];
    }
    if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (4 * l + e >= half) break;
        const double c = s_turn[4 * l + e][0], s = s_turn[4 * l + e][1];
        double &u0 = halves ? y[e] : y[2 * e], &u1 = halves ? y[4 + e] : y[2 * e + 1];
        const double p = u0, r = u1;
        u0 = __builtin_fma(p, c, -(r * s));
        u1 = __builtin_fma(r, c, p * s);
      }
    }
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)y[e];
    if (is_q) {
      on_type(a.o_dtype, [&](auto t) {
        auto* o = (decltype(t)*)a.q_out + row * a.ldo + (int64_t)h * d;
        store4(o + at0, n0, f);
        store4(o + at1, n1, f + 4);
      });
      continue;
    }
    const int64_t at = page * a.c.page + h * a.c.head + slot * a.c.slot;
    uint8_t* pool = is_v ? a.c.v : a.c.k;
    if (a.c_dtype != MOE_I8) {
      if (!page_ok) continue;
      auto put = [&](auto t) {
        auto* o = (decltype(t)*)pool + at;
        store4(o + at0, n0, f);
        store4(o + at1, n1, f + 4);
      };
      a.c_dtype == MOE_BF16 ? put(bf16_t{}) : put(f16_t{});
      continue;
    }
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, (e < 4 ? e < n0 : e - 4 < n1) ? __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu : 0u);
#pragma unroll
    for (int o = LG / 2; o; o /= 2) most = max(most, (uint32_t)__shfl_xor((int)most, o));
    const bool finite = most < 0x7F800000u;
    const QScale s = q_scale(__builtin_bit_cast(float, most));
    uint32_t codes[2] = {0, 0};
    if (finite && s.d != 0.0f) codes8(f, s, codes);
    if (!page_ok) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = i ? n1 : n0;
      int8_t* o = (int8_t*)pool + at + (i ? at1 : at0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) o[e] = (int8_t)(codes[i] >> (8 * e));
    }
    if (l == 0)
      (is_v ? a.c.vs : a.c.ks)[((int64_t)page * a.c.n_kv + h) * a.c.page_size + slot] = finite ? s.d : __builtin_nanf("");
  }
}

// ------------------------------------------------------------------ attention ---------------

struct AttendArgs {
  CacheArgs c;
  WindowArgs w;
  const void* q;
  void* out;
  float* lse;
  int64_t ldq, ldo;
  int n_heads;
  float scale;
};

// A wave for each row and head: 64 keys at a time, one a lane.
template <typename T, typename K>
__global__ __launch_bounds__(64) void k_attend_rows(AttendArgs a) {
  __shared__ float s_q[256], s_p[64];
  const int row = blockIdx.x / a.n_heads, head = blockIdx.x % a.n_heads, lane = threadIdx.x, d = a.c.d;
  const int h = head / (a.n_heads / a.c.n_kv);
  if (blockIdx.x == 0) check_seqs(a.w, a.w.max_window, 64);
  const Seq q = seq_of(a.w, row, a.w.max_window);
  if (q.tokens == 0) return;
  const int j = row - q.start, keys = q.ctx + q.tokens;
  const uint64_t seen = a.w.seen ? a.w.seen[row] : ~0ull >> (63 - j);
  for (int i = lane; i < d; i += 64) s_q[i] = to_f(((const T*)a.q)[row * a.ldq + (int64_t)head * d + i]);
  __syncthreads();
  float top = -__builtin_inff(), sum = 0.0f, acc[4] = {};
  for (int base = 0; base < keys; base += 64) {
    const int key = base + lane;
    bool sees = key < keys && (key < q.ctx || (seen >> (key - q.ctx) & 1));
    int64_t at = 0, sc = 0;
    if (sees) {
      const int page = a.w.pages[q.s * a.w.ld_pages + key / a.c.page_size], slot = key % a.c.page_size;
      sees = page >= 0 && page < a.c.n_pages;
      if (!sees) atomicOr(a.w.err, MOE_ERR_PAGE);
      at = page * a.c.page + h * a.c.head + slot * a.c.slot;
      sc = ((int64_t)page * a.c.n_kv + h) * a.c.page_size + slot;
    }
    float s = -__builtin_inff(), vs = 0.0f;
    if (sees) {
      const K* k = (const K*)a.c.k + at;
      float dot = 0.0f;
      for (int i = 0; i < d; ++i) dot = __builtin_fmaf(s_q[i], (float)to_f(k[i]), dot);
      if constexpr (sizeof(K) == 1) dot *= a.c.ks[sc], vs = a.c.vs[sc];
      s = dot * a.scale;
    }
    float most = s;
    for (int o = 32; o; o /= 2) most = __builtin_fmaxf(most, __shfl_xor(most, o));
    const float now = __builtin_fmaxf(top, most), ref = now == -__builtin_inff() ? 0.0f : now;
    const float p = sees ? expf(s - ref) : 0.0f, keep = expf(top - ref);
    top = now;
    float ps = p;
    for (int o = 32; o; o /= 2) ps += __shfl_xor(ps, o);
    sum = sum * keep + ps;
    s_p[lane] = sizeof(K) == 1 ? p * vs : p;
    const uint64_t live = __ballot(sees);
    __syncthreads();
    for (int x = 0; x < 4; ++x) acc[x] *= keep;
    for (int i = 0; i < 64; ++i) {
      if (!(live >> i & 1)) continue;
      const int64_t from = __shfl(at, i);
      for (int x = 0; x < 4; ++x)
        if (x * 64 + lane < d) acc[x] = __builtin_fmaf(s_p[i], (float)to_f(((const K*)a.c.v)[from + x * 64 + lane]), acc[x]);
    }
    __syncthreads();
  }
  for (int x = 0; x < 4; ++x)
    if (x * 64 + lane < d)
      ((T*)a.out)[row * a.ldo + (int64_t)head * d + x * 64 + lane] = from_f<T>(sum == 0.0f ? 0.0f : acc[x] / sum);
  if (a.lse && lane == 0) a.lse[(int64_t)row * a.n_heads + head] = sum == 0.0f ? -__builtin_inff() : top + logf(sum);
}

// ------------------------------------------------------------------ log probabilities -------

struct ScoreArgs {
  const void* logits;
  const int32_t* tokens;
  float *logp, *entropy, *top_logp;
  int32_t* top_ids;
  int64_t ld;
  int n, given, k, dtype;
  float scale;
};

__device__ __forceinline__ float masked_logit(float x) {   // NaN is -infinity, infinity the largest number
  x = x == x ? x : -__builtin_inff();
  return __builtin_fminf(x, 0x1.fffffep127f);
}

// A workgroup a row, which goes over it once for the maximum, once for the sums and once for each of the k best.
template <typename T>
__global__ __launch_bounds__(256) void k_logprobs_rows(ScoreArgs a) {
  __shared__ double s_red[3][4];
  __shared__ uint64_t s_key[4];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)a.logits + row * a.ld;
  const int wave = threadIdx.x >> 6;
  // larger logits first, then lower ids
  auto key_of = [&](int i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, masked_logit(to_f(x[i])) + 0.0f);
    return (uint64_t)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (uint32_t)~i;
  };
  double log_sum = 0.0, mean = 0.0;
  float top = 0.0f;
  bool none = true;
  uint64_t bound = ~0ull;
  for (int c = 0; c < (a.k > 0 ? a.k : 1); ++c) {
    uint64_t best = 0;
    for (int i = threadIdx.x; i < a.n; i += 256) {
      const uint64_t key = key_of(i);
      if (key < bound && key > best) best = key;
    }
    for (int o = 32; o; o /= 2) best = max(best, (uint64_t)__shfl_xor((unsigned long long)best, o));
    if ((threadIdx.x & 63) == 0) s_key[wave] = best;
    __syncthreads();
    best = max(max(s_key[0], s_key[1]), max(s_key[2], s_key[3]));
    bound = best;
    const int id = (int)~(uint32_t)best;
    const float v = masked_logit(to_f(x[id]));
    if (c == 0) {
      none = v == -__builtin_inff();
      top = none ? 0.0f : v;
      double sum = 0.0, dot = 0.0;
      for (int i = threadIdx.x; i < a.n; i += 256) {
        const double z = ((double)masked_logit(to_f(x[i])) - (double)top) * (double)a.scale;
        const double e = exp64(z);
        sum += e;
        if (e > 0.0) dot = __builtin_fma(e, z, dot);
      }
      sum = wave_sum(sum);
      dot = wave_sum(dot);
      if ((threadIdx.x & 63) == 0) s_red[0][wave] = sum, s_red[1][wave] = dot;
      __syncthreads();
      sum = s_red[0][0] + s_red[0][1] + s_red[0][2] + s_red[0][3];
      dot = s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3];
      log_sum = none ? 0.0 : log(sum);
      mean = none ? 0.0 : dot / sum;
    }
    if (threadIdx.x == 0 && a.k > 0) {
      a.top_ids[row * a.k + c] = id;
      a.top_logp[row * a.k + c] = (float)(((double)v - (double)top) * (double)a.scale - log_sum);
    }
    __syncthreads();
  }
  if ((int)threadIdx.x < a.given) {
    const int id = a.tokens[row * a.given + threadIdx.x];
    const float v = id >= 0 && id < a.n ? masked_logit(to_f(x[id])) : -__builtin_inff();
    a.logp[row * a.given + threadIdx.x] = (float)(((double)v - (double)top) * (double)a.scale - log_sum);
  }
  if (threadIdx.x == 0 && a.entropy) a.entropy[row] = (float)(log_sum - mean);
}

// ------------------------------------------------------------------ host checks -------------

// Rows of a cache in memory, in bytes from k: whether they lie apart, and the bytes from the first to the last.
struct Extent {
  bool ok;
  int64_t bytes;
};
Extent cache_extent(const moe_kv_cache& c) {
  const int size = c.dtype == MOE_I8 ? 1 : 2;
  const int64_t apart = (int64_t)((uintptr_t)c.v > (uintptr_t)c.k ? (uintptr_t)c.v - (uintptr_t)c.k : (uintptr_t)c.k - (uintptr_t)c.v);
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
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16) || !cache_extent(*c).ok) return MOE_E_ARG;
  if (c->dtype == MOE_I8) {
    if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return MOE_E_ARG;
    const int64_t n = (int64_t)c->n_pages * c->n_kv * c->page_size;
    if (overlap(rows_of(c->k_scale, 1, n, n, 4), rows_of(c->v_scale, 1, n, n, 4))) return MOE_E_ARG;
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
  if (!aligned(w->row_start, 4) || !aligned(w->ctx_len, 4) || !aligned(w->pages, 4) || !aligned(w->pos, 4) || !aligned(w->seen, 8) ||
      !aligned(w->err, 4))
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

}  // namespace moe

using namespace moe;

// ------------------------------------------------------------------ C ABI -------------------

extern "C" {

int moe_window_append(void* stream, const moe_kv_cache* C, const moe_window* W, int dtype, const void* q, int64_t ldq,
                      const void* k, int64_t ldk, const void* v, int64_t ldv, int n_heads, int w_dtype, const void* q_weight,
                      const void* k_weight, float eps, const float* freq, int n_rot, int layout, float amp, int o_dtype,
                      void* q_out, int64_t ldqo) {
  if (const int rc = check_cache(C)) return rc;
  if (const int rc = check_window(W, *C)) return rc;
  if (!type_ok(dtype) || !q != !q_out || (q && !type_ok(o_dtype))) return MOE_E_ARG;
  if ((q_weight || k_weight) && (!type_ok(w_dtype) || !(eps > 0.0f) || !(eps < __builtin_inff()))) return MOE_E_ARG;
  if (!(__builtin_fabsf(amp) < __builtin_inff()) || (layout != MOE_ROPE_HALF && layout != MOE_ROPE_PAIRS)) return MOE_E_ARG;
  const int d = C->head_dim, n = W->n_tokens;
  if (n_rot < 0 || n_rot > d || n_rot % 2 || (q && (n_heads < 1 || n_heads > MOE_MAX_HEADS || n_heads % C->n_kv))) return MOE_E_SHAPE;
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
  const int heads = q ? n_heads : 0, units = heads + 2 * C->n_kv;
  const AppendArgs a{cache_args(*C), window_args(*W, *C), q, k, v, q_weight, k_weight, freq, q_out, ldq, ldk, ldv, ldqo,
                     heads, n_rot, layout, w_dtype, o_dtype, C->dtype, units, eps, amp};
  const int lanes = std::max((d + 7) / 8, (n_rot + 7) / 8 + (d - n_rot + 7) / 8);
  with_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(n), dim3(256), 0, (hipStream_t)stream, a); };
    if (lanes <= 8) go(k_window_append<T, 8>);
    else if (lanes <= 16) go(k_window_append<T, 16>);
    else if (lanes <= 32) go(k_window_append<T, 32>);
    else go(k_window_append<T, 64>);
  });
  return launched("moe_window_append");
}

size_t moe_window_attention_bytes(const moe_kv_cache* C, const moe_window* W, int n_heads) {
  if (check_cache(C) || check_window(W, *C) || n_heads < 1 || n_heads > MOE_MAX_HEADS || n_heads % C->n_kv ||
      W->max_window > MOE_MAX_WINDOW)
    return 0;
  return 16;
}

int moe_window_attention(void* stream, const moe_kv_cache* C, const moe_window* W, int dtype, const void* q, int64_t ldq,
                         int n_heads, float scale, void* out, int64_t ldo, float* lse, void* workspace, size_t ws_bytes) {
  if (const int rc = check_cache(C)) return rc;
  if (const int rc = check_window(W, *C)) return rc;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_E_ARG;
  if ((C->dtype != MOE_I8 && C->dtype != dtype) || !(__builtin_fabsf(scale) < __builtin_inff())) return MOE_E_ARG;
  if (n_heads < 1 || n_heads > MOE_MAX_HEADS || n_heads % C->n_kv) return MOE_E_SHAPE;
  const int n = W->n_tokens;
  if (W->n_seqs == 0 || n == 0) return MOE_OK;
  if (W->max_window > MOE_MAX_WINDOW) return MOE_E_SHAPE;
  const int64_t wide = (int64_t)n_heads * C->head_dim;
  if (!q || !out || bad_stride(ldq, wide, n) || bad_stride(ldo, wide, n) || !aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4))
    return MOE_E_ARG;
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
  const AttendArgs a{cache_args(*C), window_args(*W, *C), q, out, lse, ldq, ldo, n_heads, scale};
  const int64_t blocks = (int64_t)n * n_heads;
  if (blocks * 64 > kLaunchThreads) return MOE_E_SHAPE;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64), 0, (hipStream_t)stream, a); };
  if (dtype == MOE_BF16) C->dtype == MOE_I8 ? go(k_attend_rows<bf16_t, int8_t>) : go(k_attend_rows<bf16_t, bf16_t>);
  else C->dtype == MOE_I8 ? go(k_attend_rows<f16_t, int8_t>) : go(k_attend_rows<f16_t, f16_t>);
  return launched("moe_window_attention");
}

size_t moe_token_logprobs_bytes(int rows, int n, int k) {
  if (rows < 0 || rows > MOE_MAX_ROWS || n < 1 || n > MOE_MAX_VOCAB || k < 0 || k > 32 || k > n) return 0;
  return 0;
}

int moe_token_logprobs(void* stream, int dtype, const void* logits, int64_t ld, int rows, int n, float scale,
                       const int32_t* tokens, int given, float* logp, float* entropy, int k, int32_t* top_ids,
                       float* top_logp, void* workspace, size_t ws_bytes) {
  if (!type_ok(dtype) || rows < 0 || given < 0 || given > 64 || k < 0 || k > 32 || !(scale > 0.0f) || !(scale < __builtin_inff()))
    return MOE_E_ARG;
  if (rows > MOE_MAX_ROWS || n < 1 || n > MOE_MAX_VOCAB) return MOE_E_SHAPE;
  if (k > n) return MOE_E_ARG;
  if (rows == 0) return MOE_OK;
  if (!logits || bad_stride(ld, n, rows) || !tokens != !given || !logp != !given || !top_ids != !k || !top_logp != !k ||
      (!given && !entropy && !k))
    return MOE_E_ARG;
  if (!aligned(logits, type_size(dtype)) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return MOE_E_ARG;
  const size_t need = moe_token_logprobs_bytes(rows, n, k);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 16))) return MOE_E_WS;
  const Rows in[] = {rows_of(logits, rows, n, ld, type_size(dtype)), rows_of(tokens, 1, (int64_t)rows * given, 0, 4)};
  const Rows outs[] = {rows_of(logp, 1, (int64_t)rows * given, 0, 4), rows_of(entropy, 1, rows, 0, 4),
                       rows_of(top_ids, 1, (int64_t)rows * k, 0, 4), rows_of(top_logp, 1, (int64_t)rows * k, 0, 4),
                       rows_of(workspace, need ? 1 : 0, (int64_t)need, 0, 1)};
  for (int i = 0; i < 5; ++i) {
    if (over(outs[i], in)) return MOE_E_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_E_ARG;
  }
  const ScoreArgs a{logits, tokens, logp, entropy, top_logp, top_ids, ld, n, given, k, dtype, scale};
  with_type(dtype, [&](auto t) {
    hipLaunchKernelGGL(k_logprobs_rows<decltype(t)>, dim3(rows), dim3(256), 0, (hipStream_t)stream, a);
  });
  return launched("moe_token_logprobs");
}

}  // extern "C"
