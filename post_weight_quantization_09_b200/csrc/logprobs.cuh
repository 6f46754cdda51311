// Log probabilities of given tokens with entropy and the top alternatives,
// and their gradient: what the logits of a quantised output layer are scored
// by (perplexity is exp of minus the mean log probability).
//
// For a row x of V logits, in base 2 with t = x log2 e and T the row's
// largest t:
//   s = sum 2^(t - T),  w = sum 2^(t - T) (t - T)
//   lse = ln 2 (T + log2 s),  logprob = ln 2 ((t_tok - T) - log2 s),
//   entropy = -sum p ln p = ln 2 (log2 s - w / s).
// (T, s, w) of two parts of a row combine by scaling both to the larger T,
// so one pass over the logits is enough.  All three are fp32; t - T is one
// fused multiply-add, so its error is half a step of the difference and
// |x| 2^-26 from log2 e's own rounding.
#pragma once

#include <type_traits>

#include <cooperative_groups.h>

#include "common.cuh"

namespace quip {
namespace lp {

namespace cg = cooperative_groups;

constexpr int NT = 256;            // threads per CTA
constexpr int GROUPS = 64;         // groups of threads whose maxima bound the k-th value; >= MAX_K
constexpr int MAX_K = QUIP_LOGPROBS_MAX_TOP;
constexpr int CAP = 256;           // candidates ranked by counting; >= MAX_CLUSTER * MAX_K
constexpr int MAX_CLUSTER = 8;
constexpr int UNROLL = 4;          // 16-byte loads in flight per thread
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// fp32 <-> unsigned with the same order (-inf < ... < +inf < NaN); 0 is below
// all.  -0 counts as +0, so that equal logits stay equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// The logits of one 16-byte vector: as pairs of fp32, and their maximum
// (NaN only where every logit is).
template <typename TX> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t PAD = 0xFF800000u;                 // -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  // every logit at least `floor`; a NaN stays
  static __device__ __forceinline__ void hold(uint4& v, float floor) {
    v.x = __float_as_uint(max_nan(__uint_as_float(v.x), floor));
    v.y = __float_as_uint(max_nan(__uint_as_float(v.y), floor));
    v.z = __float_as_uint(max_nan(__uint_as_float(v.z), floor));
    v.w = __float_as_uint(max_nan(__uint_as_float(v.w), floor));
  }
  template <int K>
  static __device__ __forceinline__ float top(const uint4 (&v)[K]) {
    float t = NEG_INF;
#pragma unroll
    for (int j = 0; j < K; ++j)
      t = fmaxf(t, fmaxf(fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y)),
                         fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w))));
    return t;
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t PAD = 0xFF80FF80u;                 // -inf, -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
  static __device__ __forceinline__ void hold(uint4& v, float floor) {
    const __nv_bfloat162 f = __float2bfloat162_rn(floor);
    uint32_t* u[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r = __hmax2_nan(pair(*u[i]), f);
      *u[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  template <int K>
  static __device__ __forceinline__ float top(const uint4 (&v)[K]) {
    __nv_bfloat162 t = pair(PAD);
#pragma unroll
    for (int j = 0; j < K; ++j)
      t = __hmax2(t, __hmax2(__hmax2(pair(v[j].x), pair(v[j].y)), __hmax2(pair(v[j].z), pair(v[j].w))));
    return fmaxf(__low2float(t), __high2float(t));
  }
};

constexpr float LOW_T = 4096.f;

// (T, s, w) of a part of a row.  T = -inf: no logit that 2^(t - T) can serve
// (none above LEAST_T, Running below), s = w = 0, or NaN
// where it met one.
struct Part {
  float T, s, w;
  __device__ __forceinline__ void raise(float to) {     // to >= T
    // 2^-200 is 0 in fp32; a longer way down times s may leave fp32
    const float d = T == NEG_INF ? 0.f : max_nan(T - to, -200.f);
    const float f = ex2(d);
    w = f * fmaf(d, s, w);
    s *= f;
    T = to;
  }
};
__device__ __forceinline__ Part no_part() { return Part{NEG_INF, 0.f, 0.f}; }

// The combination of the 32 lanes' parts, in every lane.
__device__ __forceinline__ Part warp_combine(Part p) {
  // an ordered key for redux.sync; a maximum is never NaN
  p.raise(key_value(__reduce_max_sync(0xffffffffu, order_key(p.T))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
    p.w += __shfl_xor_sync(0xffffffffu, p.w, o);
  }
  return p;
}

// A thread's running part, with the largest logit m itself.  T follows the
// maximum only once that is SLACK above it (2^(t - T) has room; the entropy's
// log2 s and w / s then share up to SLACK, half a step of which is small):
// most rounds then cost a comparison.
//
// T does not follow a maximum of LEAST_T and below (masks of large finite
// values): the rounding of such a T is no longer small beside 1 (half a step
// of 2^31 is 128, and 2^128 is infinite).  Those logits are held as those of
// -inf are, and count 0 beside any other; a row of nothing else is sum_low's.
constexpr float SLACK = 8.f, LEAST_T = -1e6f;
struct Running {
  float m = NEG_INF;
  Part p{NEG_INF, 0.f, 0.f};
  float raise_at = LEAST_T;
  // A logit of -inf (a barred token, padding) has e = 0, but t - T = -inf
  // would make e (t - T) NaN: logits are held at a value whose exponential is
  // 0 in fp32, at least 100 below T's after its rounding to bf16 too
  // (lower by 1 / 64 where that is more).
  float floor = -200.f, ref = 0.f;
  // `top` is the maximum of the logits about to be added
  __device__ __forceinline__ void raise(float top) {
    m = fmaxf(m, top);
    if (m * LOG2E > raise_at) {
      p.raise(m * LOG2E);
      raise_at = p.T + SLACK;
      floor = m - fmaxf(200.f, fabsf(m) * 0.015625f);
      ref = -p.T;
    }
  }
  // N more logits, held at floor
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = fmaf(x[i], LOG2E, ref), e = ex2(d);
      p.s += e;
      p.w = fmaf(e, d, p.w);
    }
  }
};

// The part of a row that a CTA handles: logits [v0, v1), of which the first
// `head` come before the first 16-byte boundary and `tail` after the last
// vector.  Thread t reads vectors t, t + NT, ... and edge logits t.
template <typename TX>
struct Slice {
  const TX* x;                     // the row
  int v0, v1, head, nvec, tail;
  __device__ __forceinline__ Slice(const TX* row, int a, int b) : x(row), v0(a), v1(b) {
    constexpr int N = Vec<TX>::N;
    const int off = (int)((reinterpret_cast<uintptr_t>(row + a) / sizeof(TX)) % N);
    head = min(off ? N - off : 0, b - a);
    nvec = (b - a - head) / N;
    tail = b - a - head - nvec * N;
  }
  __device__ __forceinline__ const uint4* vecs() const { return reinterpret_cast<const uint4*>(x + v0 + head); }
  // the logit before (thread < head) or after (thread < tail) the vectors
  __device__ __forceinline__ int edge(int which, int tid) const {
    if (which == 0) return tid < head ? v0 + tid : -1;
    return tid < tail ? v1 - tail + tid : -1;
  }
  __device__ __forceinline__ bool mine(int tid) const { return tid < nvec || tid < head || tid < tail; }
  // fn(logit, index) for those of thread t's logits that are not below
  // `least` (all NaN among them), of step c: its c-th vector, or past the
  // last its edge logits
  __device__ __forceinline__ int steps() const { return (nvec + NT - 1) / NT + 1; }
  template <typename Fn>
  __device__ __forceinline__ void step(int t, int c, float least, Fn fn) const {
    constexpr int N = Vec<TX>::N;
    const int i = t + c * NT;
    if (c == steps() - 1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int v = edge(e, t);
        if (v >= 0 && !(to_f32(x[v]) < least)) fn(to_f32(x[v]), v);
      }
    } else if (i < nvec) {
      float f[N];
      Vec<TX>::unpack(__ldg(vecs() + i), f);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (!(f[j] < least)) fn(f[j], v0 + head + i * N + j);
    }
  }
};

// What the threads that stream a row's slice leave for the rest.
struct RowShared {
  Part part[NT / 32];                          // per warp
  uint32_t gmax[GROUPS];                       // order_key of the groups' maxima, 0: none
};
// Choosing the top alternatives.
struct TopShared {
  uint32_t tau;
  int count, owners;
  int owner[NT];
  // (order_key << 32) | ~index: larger = earlier
  alignas(16) unsigned long long cand[CAP];
  alignas(16) unsigned long long best[MAX_K];  // the slice's k largest, in order
  unsigned long long red[NT / 32];
};

__device__ __forceinline__ unsigned long long cand_key(float x, int v) {
  return ((unsigned long long)order_key(x) << 32) | (uint32_t)~(uint32_t)v;
}

// How many of list[0 .. count) are above c; list is 16-byte aligned.
__device__ __forceinline__ int count_above(const unsigned long long* list, int count, unsigned long long c) {
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(list);
  int above = 0;
#pragma unroll 8
  for (int i = 0; i < count / 2; ++i) {
    const ulonglong2 v = two[i];
    above += (v.x > c ? 1 : 0) + (v.y > c ? 1 : 0);
  }
  if (count & 1) above += list[count - 1] > c ? 1 : 0;
  return above;
}

// A barrier of the NT threads that read logits.
__device__ __forceinline__ void team_sync() { asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory"); }

// The k largest (value, then lowest index) logits of a slice into tp.best, in
// order; keys of 0 where the slice has fewer.  tid: the thread's number in
// the team.
//
// The k-th largest of the groups' maxima is at most the k-th largest logit,
// and few logits are above it (about 64 ln(64 / (64 - k)) of a random row),
// all in threads whose own maximum is: those threads' logits are read again
// (from L2) and the ones not below are ranked by counting.  Where more than
// CAP pass (many equal maxima, or most of them in one thread), k rounds of a
// maximum over all logits below the one before find the same.
template <typename TX>
__device__ __forceinline__ void choose_top(TopShared& tp, const RowShared& rs, const Slice<TX>& sl, float tmax, int k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    // the k-th largest of the 64, two per lane: the largest leaves k times
    uint32_t hi = rs.gmax[lane], lo = rs.gmax[lane + 32], top = 0u;
    if (lo > hi) { const uint32_t c = hi; hi = lo, lo = c; }
    for (int j = 0; j < k; ++j) {
      top = __reduce_max_sync(0xffffffffu, hi);
      if (lane == __ffs(__ballot_sync(0xffffffffu, hi == top)) - 1) hi = lo, lo = 0u;
    }
    if (lane == 0) tp.tau = top;
  }
  team_sync();
  const uint32_t tau = tp.tau;
  if (sl.mine(tid) && order_key(tmax) >= tau) tp.owner[atomicAdd(&tp.owners, 1)] = tid;
  team_sync();
  const int steps = sl.steps();
  const float least = tau ? key_value(tau) : NEG_INF;
  for (int i = warp; i < tp.owners; i += NT / 32)
    for (int c = lane; c < steps; c += 32)
      sl.step(tp.owner[i], c, least, [&](float f, int v) {
        const int at = atomicAdd(&tp.count, 1);
        if (at < CAP) tp.cand[at] = cand_key(f, v);
      });
  team_sync();
  const int count = tp.count;
  if (count <= CAP) {
    for (int i = tid; i < count; i += NT) {
      const unsigned long long c = tp.cand[i];
      const int above = count_above(tp.cand, count, c);
      if (above < k) tp.best[above] = c;
    }
    team_sync();
    return;
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < k; ++j) {
    unsigned long long top = 0ull;
    for (int c = 0; c < steps; ++c)
      sl.step(tid, c, NEG_INF, [&](float f, int v) {
        const unsigned long long key = cand_key(f, v);
        if (key < last && key > top) top = key;
      });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long c = __shfl_xor_sync(0xffffffffu, top, o);
      top = c > top ? c : top;
    }
    if (lane == 0) tp.red[warp] = top;
    team_sync();
    top = 0ull;
    for (int i = 0; i < NT / 32; ++i) top = tp.red[i] > top ? tp.red[i] : top;
    if (tid == 0) tp.best[j] = top;
    last = top;
    team_sync();
  }
}

// For the rows whose largest |t| is LOW_T or more, where half a step of T no
// longer is small (and of a maximum of the type's lowest value, -inf or +inf): their maximum m, and the sums of exp and
// of exp (x - m) with the differences in natural units, held at -200; one
// warp.
template <typename TX>
__device__ __noinline__ Part sum_low(const TX* x, int V) {
  float m = NEG_INF;
  for (int v = threadIdx.x % 32; v < V; v += 32) m = fmaxf(m, to_f32(x[v]));
  m = warp_max(m);
  const float ref = m == NEG_INF ? 0.f : m;
  Part p{m, 0.f, 0.f};
  for (int v = threadIdx.x % 32; v < V; v += 32) {
    const float d = max_nan(to_f32(x[v]) - ref, -200.f), e = ex2(d * LOG2E);
    p.s += e;
    p.w = fmaf(e, d, p.w);
  }
  p.s = warp_sum(p.s), p.w = warp_sum(p.w);
  return p;
}

struct Args {
  int64_t ld;
  int V, k;
  int64_t T;
  const int32_t* tokens;
  float *logprob, *entropy, *lse, *top_values;
  int32_t* top_ids;
};

// A row's outputs from its parts' combination, and the log probability of a
// logit of the row.
template <typename TX>
struct Finish {
  const TX* x;
  Part p;
  float log_s;                 // in the units of p: base 2, or natural for a row of sum_low
  bool low;
  // every thread of a warp; p from warp_combine
  __device__ __forceinline__ Finish(const TX* x_, int V, Part p_) : x(x_), p(p_), low(!(fabsf(p_.T) < LOW_T)) {
    if (low) p = sum_low(x, V);
    log_s = low ? logf(p.s) : log2f(p.s);
  }
  __device__ __forceinline__ bool empty() const { return p.T == NEG_INF && p.s == 0.f; }   // no logit above -inf
  __device__ __forceinline__ float given(float f) const {
    if (low) return empty() ? NEG_INF : (f - p.T) - log_s;
    if (f < -1e38f) return f - LN2 * (p.T + log_s);      // times log2 e it may leave fp32
    return LN2 * (fmaf(f, LOG2E, -p.T) - log_s);
  }
  __device__ __forceinline__ void write(const Args& a, int64_t row) const {
    const float unit = low ? 1.f : LN2;
    if (a.lse) a.lse[row] = empty() ? NEG_INF : unit * (p.T + log_s);
    if (a.entropy) a.entropy[row] = empty() ? 0.f : unit * (log_s - p.w / p.s);
    if (a.tokens) {
      const int tok = a.tokens[row];
      if (tok >= a.V || tok < -1) record_status(QUIP_ERR_ARG);
      a.logprob[row] = tok >= 0 && tok < a.V ? given(to_f32(x[tok])) : 0.f;
    }
  }
  __device__ __forceinline__ void write_top(const Args& a, int64_t row, int at, unsigned long long c) const {
    a.top_ids[row * a.k + at] = (int)~(uint32_t)c;
    a.top_values[row * a.k + at] = given(key_value((uint32_t)(c >> 32)));
  }
};

template <typename TX, int K>
__device__ __forceinline__ void consume(Running& r, uint4 (&u)[K]) {
  constexpr int N = Vec<TX>::N;
  r.raise(Vec<TX>::top(u));
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float f[N];
    Vec<TX>::hold(u[j], r.floor);
    Vec<TX>::unpack(u[j], f);
    r.add(f);
  }
}
// This thread's vectors (every NT-th) of the `n` at v, CHUNK at most.
constexpr int CHUNK = UNROLL * NT;
template <typename TX>
__device__ __forceinline__ void consume_chunk(Running& r, const uint4* v, int n, int tid) {
  if (n >= CHUNK) {
    uint4 u[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) u[j] = v[tid + j * NT];
    consume<TX>(r, u);
  } else {
    uint4 u[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      constexpr uint32_t P = Vec<TX>::PAD;
      u[j] = tid + j * NT < n ? v[tid + j * NT] : make_uint4(P, P, P, P);
    }
    consume<TX>(r, u);
  }
}
// The thread's edge logits, then its and its warp's part into rs.
template <typename TX, bool TOP>
__device__ __forceinline__ void close_row(Running& r, const Slice<TX>& sl, RowShared& rs, TopShared& tp, int tid) {
  if (TOP && tid == 0) tp.count = 0, tp.owners = 0;
  const int a = sl.edge(0, tid), b = sl.edge(1, tid);
  if (a >= 0 || b >= 0) {
    float f[2] = {a >= 0 ? to_f32(sl.x[a]) : NEG_INF, b >= 0 ? to_f32(sl.x[b]) : NEG_INF};
    r.raise(fmaxf(f[0], f[1]));
      f[0] = max_nan(f[0], r.floor), f[1] = max_nan(f[1], r.floor);
    r.add(f);
  }
  if (TOP && sl.mine(tid)) atomicMax(&rs.gmax[tid % GROUPS], order_key(r.m));
  const Part p = warp_combine(r.p);
  if (tid % 32 == 0) rs.part[tid / 32] = p;
}

// One cluster per row (one CTA where the rows fill the GPU, up to 8 where
// they do not), each CTA a slice of it; the first CTA combines.
// 4096 x 32000 bf16: 52 us, 5.0 TB/s, 63 us with five alternatives; 2047 x
// 50257 fp32: 74 us, 5.6 TB/s; 64 x 128000 bf16: 7.3 us, 13.7 us with twenty
// (a chain of barriers and L2 loads); one row of 32000: 6.1 us.  A bf16 logit
// costs six to seven instructions and an ex2, which with the loads' latency
// bound it; 256 threads with five CTAs an SM were as fast as 128 with ten, and
// resident CTAs behind a ring of bulk copies slower by 3 us (no alternatives)
// to 20 us.
template <typename TX, bool TOP>
__global__ void __launch_bounds__(NT, 5) k_logprobs(const TX* __restrict__ logits, const __grid_constant__ Args a) {
  constexpr int N = Vec<TX>::N;
  __shared__ RowShared rs;
  __shared__ TopShared tp;
  __shared__ Part cta;                         // read by the other CTAs of the cluster, as tp.best
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
  const int64_t row = blockIdx.x / nc;
  const TX* x = logits + row * a.ld;
  // slices of whole 16-byte vectors' worth of logits
  const int per = ((a.V + nc - 1) / nc + N - 1) / N * N;
  const Slice<TX> sl(x, min(a.V, rank * per), min(a.V, (rank + 1) * per));
  if (TOP) {
    if (tid < GROUPS) rs.gmax[tid] = 0u;
    if (tid < MAX_K) tp.best[tid] = 0ull;
    __syncthreads();
  }
  Running r;
  for (int i = 0; i < sl.nvec; i += CHUNK) consume_chunk<TX>(r, sl.vecs() + i, sl.nvec - i, tid);
  close_row<TX, TOP>(r, sl, rs, tp, tid);
  __syncthreads();
  if (warp == NT / 32 - 1) {
    const Part p = warp_combine(lane < NT / 32 ? rs.part[lane] : no_part());
    if (lane == 0) cta = p;
  }
  if constexpr (TOP) choose_top(tp, rs, sl, r.m, k);
  if (nc > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0) {
    const Finish<TX> fin(x, a.V, warp_combine(lane < nc ? *cluster.map_shared_rank(&cta, lane) : no_part()));
    if (tid == 0) fin.write(a, row);
    if constexpr (TOP) {
      if (nc == 1) {
        if (tid < k) fin.write_top(a, row, tid, tp.best[tid]);
      } else {
        // the nc lists of k keys, ranked by counting; a key of 0 is none
        const int total = nc * k;
        for (int i = tid; i < total; i += NT) tp.cand[i] = cluster.map_shared_rank(tp.best, i / k)[i % k];
        __syncthreads();
        for (int i = tid; i < total; i += NT) {
          const unsigned long long c = tp.cand[i];
          if (c == 0ull) continue;
          const int above = count_above(tp.cand, total, c);
          if (above < k) fin.write_top(a, row, above, c);
        }
      }
    }
  }
  if (nc > 1) cluster.sync();      // the others' shared memory is read until here
}

// d_logits[v] = g (1[v = tok] - p_v) - ge p_v (ln p_v + H), p_v = exp(x_v - lse).
// Elementwise: one read and one write per logit bound it (4096 x 32000 bf16:
// 84.5 us, 6.2 TB/s; with the token's and the entropy's terms in every element
// 91 us).  A row with g = 0
// (or no token) and ge = 0 is 0 without its logits being looked at, as is a
// row with no logit above -inf.  A row whose lse is far from 0 (FAR_LSE) is
// one CTA's, which reads it three times (4096 x 32000 bf16, all rows so:
// 113 us; 64 x 32000 fp32: 17 us for 3.7).
template <typename TX>
__device__ __forceinline__ TX from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// What rounding took from a row's log-sum-exp: (max - lse) + ln sum exp(x -
// max), from the row again; the whole CTA.  exp(x - lse) carries half a step
// of lse, and where |lse| is FAR_LSE or more that is more than the other
// roundings: 2^-16 of p at 256, all of p at 2^24.  An lse that is no rounding
// of this row's (of a vocabulary in shards) is taken as it stands: 0.
constexpr float FAR_LSE = 256.f;
template <typename TX>
__device__ __noinline__ float lse_rest(const TX* x, int V, float lse) {
  constexpr int N = Vec<TX>::N;
  __shared__ float sums[2][NT / 32];
  const int tid = threadIdx.x;
  const Slice<TX> sl(x, 0, V);
  const int a = sl.edge(0, tid), b = sl.edge(1, tid);
  const float f0 = a >= 0 ? to_f32(x[a]) : NEG_INF, f1 = b >= 0 ? to_f32(x[b]) : NEG_INF;
  float m = fmaxf(f0, f1), s = 0.f;
#pragma unroll 4
  for (int i = tid; i < sl.nvec; i += NT) {
    const uint4 v[1] = {sl.vecs()[i]};
    m = fmaxf(m, Vec<TX>::top(v));
  }
  m = warp_max(m);
  if (tid % 32 == 0) sums[0][tid / 32] = m;
  __syncthreads();
  for (int i = 0; i < NT / 32; ++i) m = fmaxf(m, sums[0][i]);
  if (a >= 0) s += ex2((f0 - m) * LOG2E);
  if (b >= 0) s += ex2((f1 - m) * LOG2E);
#pragma unroll 4
  for (int i = tid; i < sl.nvec; i += NT) {
    float f[N];
    Vec<TX>::unpack(sl.vecs()[i], f);
#pragma unroll
    for (int j = 0; j < N; ++j) s += ex2((f[j] - m) * LOG2E);
  }
  s = warp_sum(s);
  if (tid % 32 == 0) sums[1][tid / 32] = s;
  __syncthreads();                             // past it every logit has been read
  s = 0.f;
  for (int i = 0; i < NT / 32; ++i) s += sums[1][i];
  const float rest = (m - lse) + logf(s);
  return fabsf(rest) <= fabsf(lse) * 0x1p-21f ? rest : 0.f;
}

constexpr int GRAD_VECS = 4;       // 16-byte vectors per thread
template <typename TX> __host__ __device__ constexpr int grad_cols() { return NT * GRAD_VECS * Vec<TX>::N; }

template <typename TX>
__global__ void __launch_bounds__(NT)
    k_logprobs_grad(const TX* logits, int64_t ld, int V, const int32_t* __restrict__ tokens,
                    const float* __restrict__ lse, const float* __restrict__ entropy,
                    const float* __restrict__ g_logprob, const float* __restrict__ g_entropy, TX* d_logits,
                    int64_t ldd, int nseg) {
  constexpr int N = Vec<TX>::N;
  const int64_t row = blockIdx.x / nseg;
  const int seg = blockIdx.x % nseg;
  const TX* x = logits + row * ld;
  TX* d = d_logits + row * ldd;
  int tok = tokens ? tokens[row] : -1;
  if (tok >= V || tok < -1) {
    if (seg == 0 && threadIdx.x == 0) record_status(QUIP_ERR_ARG);
    tok = -1;
  }
  const float g = g_logprob && tok >= 0 ? g_logprob[row] : 0.f;
  const float ge = g_entropy ? g_entropy[row] : 0.f;
  const float l = lse[row];
  const float H = ge != 0.f ? entropy[row] : 0.f;
  int v0 = seg * grad_cols<TX>(), v1 = min(V, v0 + grad_cols<TX>());
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(d)) & 15) == 0;
  if ((g == 0.f && ge == 0.f) || l == NEG_INF) {
    for (int v = v0 + N * threadIdx.x; v < v1; v += N * NT) {
      if (vec && v + N <= v1) *reinterpret_cast<uint4*>(d + v) = make_uint4(0u, 0u, 0u, 0u);
      else
        for (int i = v; i < min(v + N, v1); ++i) d[i] = from_f32<TX>(0.f);
    }
    return;
  }
  // -g p - ge p (ln p + H) = p (c0 + c1 ln p); without an entropy gradient
  // (c1 = 0) p alone, and no care for p = 0 times ln p = -inf
  const float c0 = -g - ge * H, c1 = -ge;
  float rest = 0.f;
  auto write = [&](auto entropy_too, auto far) {
    auto one = [&](float f) {
      const float d = decltype(far)::value ? (f - l) - rest : f - l;
      if constexpr (decltype(entropy_too)::value) {
        const float lnp = max_nan(d, -200.f);              // p = 0 below
        return ex2(lnp * LOG2E) * fmaf(c1, lnp, c0);
      } else {
        return ex2(d * LOG2E) * c0;
      }
    };
    auto scalar = [&](int v) { d[v] = from_f32<TX>(one(to_f32(x[v])) + (v == tok ? g : 0.f)); };
    if (!vec) {
      // rows whose logits and gradients do not both start on 16 bytes
      for (int v = v0 + threadIdx.x; v < v1; v += NT) scalar(v);
      return;
    }
    uint4 u[GRAD_VECS];
#pragma unroll
    for (int j = 0; j < GRAD_VECS; ++j) {
      const int v = v0 + (threadIdx.x + j * NT) * N;
      u[j] = v + N <= v1 ? *reinterpret_cast<const uint4*>(x + v) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < GRAD_VECS; ++j) {
      const int v = v0 + (threadIdx.x + j * NT) * N;
      if (v + N <= v1) {
        float f[N];
        alignas(16) TX o[N];
        Vec<TX>::unpack(u[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = one(f[i]);
        if ((unsigned)(tok - v) < (unsigned)N) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (v + i == tok) f[i] += g;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = from_f32<TX>(f[i]);
        *reinterpret_cast<uint4*>(d + v) = *reinterpret_cast<const uint4*>(o);
      } else {
        for (int i = v; i < v1; ++i) scalar(i);
      }
    }
  };
  if (fabsf(l) >= FAR_LSE && fabsf(l) < -NEG_INF) {
    if (seg > 0) return;
    rest = lse_rest(x, V, l);
    for (v0 = 0; v0 < V; v0 += grad_cols<TX>()) {
      v1 = min(V, v0 + grad_cols<TX>());
      if (ge != 0.f) write(std::true_type{}, std::true_type{});
      else write(std::false_type{}, std::true_type{});
    }
    return;
  }
  if (ge != 0.f) write(std::true_type{}, std::false_type{});
  else write(std::false_type{}, std::false_type{});
}

}  // namespace lp
}  // namespace quip
