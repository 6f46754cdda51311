// Log probabilities of given tokens with entropy and the top alternatives,
// and their gradient: what the logits of a quantised output layer are scored
// by (perplexity is exp of minus the mean log probability).
//
// For a row x of V logits, in base 2 with t = x log2 e and T = max t:
//   s = sum 2^(t - T),  w = sum 2^(t - T) (t - T)
//   lse = ln 2 (T + log2 s),  logprob = ln 2 ((t_tok - T) - log2 s),
//   entropy = -sum p ln p = ln 2 (log2 s - w / s).
// (T, s, w) of two parts of a row combine by scaling both to the larger T,
// so one pass over the logits is enough.  T, s and w are fp32.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace quip {
namespace lp {

namespace cg = cooperative_groups;

constexpr int NT = 256;            // threads per CTA
constexpr int GROUPS = 64;         // groups of threads whose maxima bound the k-th value; >= MAX_K
constexpr int MAX_K = 32;
constexpr int CAP = NT;            // candidates ranked in one step
constexpr int MAX_CLUSTER = 8;
constexpr int UNROLL = 4;          // 16-byte loads in flight per thread
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

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
constexpr float NEG_INF = -__builtin_huge_valf();

// fp32 -> unsigned with the same order (-inf < ... < +inf < NaN); 0 is below all.
// -0 counts as +0, so that equal logits stay equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x == 0.f) x = 0.f;
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The logits of one 16-byte vector as fp32.
template <typename TX> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t PAD = 0xFF800000u;                 // -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
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
};

// Running (T, s, w) of a part of a row.
struct Part {
  float T = NEG_INF, s = 0.f, w = 0.f;
  // scale to the maximum T2 >= T.  A part without a finite logit (T = -inf)
  // has s = w = 0, or NaN where it met one: kept as it is.
  __device__ __forceinline__ void raise(float T2) {
    const float d = T == NEG_INF ? 0.f : T - T2;
    const float f = ex2(d);
    w = f * fmaf(d, s, w);
    s *= f;
    T = T2;
  }
  __device__ __forceinline__ void add(Part o) {
    const float T2 = fmaxf(T, o.T);
    raise(T2);
    o.raise(T2);
    s += o.s, w += o.w;
  }
};

// N more logits.  A -inf logit (and padding) counts 0: its exponent is held
// at -200, where 2^x is 0 in fp32; max.NaN lets a NaN through.
template <int N>
__device__ __forceinline__ void accumulate(Part& p, const float (&f)[N]) {
  float top = f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
  p.raise(fmaxf(p.T, top * LOG2E));
  const float T = p.T == NEG_INF ? 0.f : p.T;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = max_nan(fmaf(f[i], LOG2E, -T), -200.f);
    const float e = ex2(d);
    p.s += e;
    p.w = fmaf(e, d, p.w);
  }
}

// The part of a row that a CTA handles: logits [v0, v1), of which the first
// `head` come before the first 16-byte boundary and `tail` after the last.
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
};

struct Shared {
  Part part[NT / 32];
  Part cta;                        // read by the other CTAs of the cluster
  uint32_t gmax[GROUPS];
  uint32_t tau;
  int count;
  unsigned long long cand[CAP];    // (order_key << 32) | ~index: larger = earlier
  unsigned long long best[MAX_K];  // the CTA's k largest, in order; read by the cluster
  unsigned long long red[NT / 32];
};

__device__ __forceinline__ unsigned long long cand_key(float x, int v) {
  return ((unsigned long long)order_key(x) << 32) | (uint32_t)~(uint32_t)v;
}

// Calls fn(logit, index) for every logit of the slice that thread `owner`
// read, the lanes of the calling warp sharing its vectors.
template <typename TX, typename Fn>
__device__ __forceinline__ void warp_for_owner(const Slice<TX>& sl, int owner, int lane, Fn fn) {
  constexpr int N = Vec<TX>::N;
  for (int i = owner + lane * NT; i < sl.nvec; i += 32 * NT) {
    float f[N];
    Vec<TX>::unpack(sl.vecs()[i], f);
#pragma unroll
    for (int j = 0; j < N; ++j) fn(f[j], sl.v0 + sl.head + i * N + j);
  }
  if (lane < 2) {
    const int v = sl.edge(lane, owner);
    if (v >= 0) fn(to_f32(sl.x[v]), v);
  }
}

// The k largest (value, then lowest index) logits of the CTA's slice into
// sh.best, in order; keys of 0 where the slice has fewer.  tmax is the
// largest logit the thread read (-inf if none).
//
// The k-th largest of the 64 groups' maxima is at most the k-th largest
// logit, and few logits are above it (about 64 ln(64 / (64 - k)) of a random
// row), all in threads whose own maximum is: those threads' logits are read
// again (from L2) and the ones not below are ranked by counting.  Where more
// than CAP pass (many equal maxima, or most of them in one thread), k rounds
// of a maximum over all logits below the one before do the same.
template <typename TX>
__device__ void cta_top(Shared& sh, const Slice<TX>& sl, float tmax, bool any, int k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < GROUPS) sh.gmax[tid] = 0u;
  if (tid < MAX_K) sh.best[tid] = 0ull;
  if (tid == 0) sh.count = 0, sh.tau = 0u;
  __syncthreads();
  const uint32_t mine = any ? order_key(tmax) : 0u;
  if (any) atomicMax(&sh.gmax[tid % GROUPS], mine);
  __syncthreads();
  if (tid < GROUPS) {
    const uint32_t g = sh.gmax[tid];
    int above = 0;
    for (int i = 0; i < GROUPS; ++i) {
      const uint32_t o = sh.gmax[i];
      above += (o > g || (o == g && i < tid)) ? 1 : 0;
    }
    if (above == k - 1) sh.tau = g;
  }
  __syncthreads();
  const uint32_t tau = sh.tau;
  unsigned todo = __ballot_sync(0xffffffffu, any && mine >= tau);
  while (todo) {
    const int b = __ffs(todo) - 1;
    todo &= todo - 1;
    warp_for_owner(sl, warp * 32 + b, lane, [&](float f, int v) {
      if (order_key(f) >= tau) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < CAP) sh.cand[at] = cand_key(f, v);
      }
    });
  }
  __syncthreads();
  const int count = sh.count;
  if (count <= CAP) {
    if (tid < count) {
      const unsigned long long c = sh.cand[tid];
      int above = 0;
      for (int i = 0; i < count; ++i) above += sh.cand[i] > c ? 1 : 0;
      if (above < k) sh.best[above] = c;
    }
    __syncthreads();
    return;
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < k; ++j) {
    unsigned long long top = 0ull;
    for (int own = 0; own < 32; ++own)
      warp_for_owner(sl, warp * 32 + own, lane, [&](float f, int v) {
        const unsigned long long c = cand_key(f, v);
        if (c < last && c > top) top = c;
      });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long c = __shfl_xor_sync(0xffffffffu, top, o);
      top = c > top ? c : top;
    }
    if (lane == 0) sh.red[warp] = top;
    __syncthreads();
    top = 0ull;
    for (int i = 0; i < NT / 32; ++i) top = sh.red[i] > top ? sh.red[i] : top;
    if (tid == 0) sh.best[j] = top;
    last = top;
    __syncthreads();
  }
}

// One cluster per row (one CTA where the rows fill the GPU, up to 8 where
// they do not), each CTA a slice of it; the first CTA combines.
template <typename TX, bool TOP>
__global__ void __launch_bounds__(NT, 4)
    k_logprobs(const TX* __restrict__ logits, int64_t ld, int V, const int32_t* __restrict__ tokens,
               float* __restrict__ logprob, float* __restrict__ entropy, float* __restrict__ lse, int k,
               float* __restrict__ top_values, int32_t* __restrict__ top_ids) {
  constexpr int N = Vec<TX>::N;
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / nc;
  const TX* x = logits + row * ld;
  // slices of whole 16-byte vectors' worth of logits
  const int per = ((V + nc - 1) / nc + N - 1) / N * N;
  const Slice<TX> sl(x, min(V, rank * per), min(V, (rank + 1) * per));

  Part p;
  float tmax = NEG_INF;
  const uint4* vecs = sl.vecs();
  for (int i = tid; i < sl.nvec; i += UNROLL * NT) {
    uint4 u[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      constexpr uint32_t P = Vec<TX>::PAD;
      u[j] = i + j * NT < sl.nvec ? __ldg(vecs + i + j * NT) : make_uint4(P, P, P, P);
    }
    float f[UNROLL * N];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) Vec<TX>::unpack(u[j], f + j * N);
    if (TOP) {
#pragma unroll
      for (int j = 0; j < UNROLL * N; ++j) tmax = fmaxf(tmax, f[j]);
    }
    accumulate(p, f);
  }
  {
    const int a = sl.edge(0, tid), b = sl.edge(1, tid);
    const float f[2] = {a >= 0 ? to_f32(x[a]) : NEG_INF, b >= 0 ? to_f32(x[b]) : NEG_INF};
    if (a >= 0 || b >= 0) {
      tmax = fmaxf(tmax, fmaxf(f[0], f[1]));
      accumulate(p, f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Part q;
    q.T = __shfl_xor_sync(0xffffffffu, p.T, o);
    q.s = __shfl_xor_sync(0xffffffffu, p.s, o);
    q.w = __shfl_xor_sync(0xffffffffu, p.w, o);
    p.add(q);
  }
  if (lane == 0) sh.part[warp] = p;
  if constexpr (TOP) cta_top(sh, sl, tmax, tid < sl.nvec || tid < sl.head || tid < sl.tail, k);
  __syncthreads();
  if (tid == 0) {
    Part c = sh.part[0];
    for (int i = 1; i < NT / 32; ++i) c.add(sh.part[i]);
    sh.cta = c;
  }
  if (nc > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0) {
    Part c = sh.cta;
    for (int i = 1; i < nc; ++i) c.add(*cluster.map_shared_rank(&sh.cta, i));
    const float l2 = log2f(c.s);
    const bool empty = c.s == 0.f;                       // no logit above -inf
    const float T = c.T == NEG_INF ? 0.f : c.T;
    if (tid == 0) {
      if (lse) lse[row] = empty ? NEG_INF : LN2 * (T + l2);
      if (entropy) entropy[row] = empty ? 0.f : LN2 * (l2 - c.w / c.s);
      if (tokens) {
        const int tok = tokens[row];
        float v = 0.f;
        if (tok >= V || tok < -1) record_status(QUIP_ERR_ARG);
        else if (tok >= 0) v = empty ? NEG_INF : LN2 * (fmaf(to_f32(x[tok]), LOG2E, -T) - l2);
        logprob[row] = v;
      }
    }
    if constexpr (TOP) {
      // the nc lists of k keys, ranked by counting
      const int total = nc * k;
      if (nc > 1) {
        if (tid < total) sh.cand[tid] = cluster.map_shared_rank(sh.best, tid / k)[tid % k];
        __syncthreads();
      }
      const unsigned long long* list = nc > 1 ? sh.cand : sh.best;
      if (tid < total) {
        const unsigned long long c = list[tid];
        int above = tid;
        if (nc > 1) {
          above = 0;
          for (int i = 0; i < total; ++i) above += (list[i] > c || (list[i] == c && i < tid)) ? 1 : 0;
        }
        if (above < k) {
          const int v = (int)~(uint32_t)c;
          top_ids[row * k + above] = v;
          top_values[row * k + above] = empty ? NEG_INF : LN2 * (fmaf(to_f32(x[v]), LOG2E, -T) - l2);
        }
      }
    }
  }
  if (nc > 1) cluster.sync();      // the others' shared memory is read until here
}

// d_logits[v] = g (1[v = tok] - p_v) - ge p_v (ln p_v + H), p_v = exp(x_v - lse).
// Elementwise: one read and one write per logit bound it.  A row with g = 0
// (or no token) and ge = 0 is 0 without its logits being looked at, as is a
// row with no logit above -inf.
template <typename TX>
__device__ __forceinline__ TX from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

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
  const bool zero = (g == 0.f && ge == 0.f) || l == NEG_INF;
  // -g p - ge p (ln p + H) = p (c0 + c1 ln p)
  const float c0 = -g - ge * H, c1 = -ge;
  auto one = [&](float f, int v) {
    const float lnp = max_nan(f - l, -200.f);            // p = 0 below
    float r = ex2(lnp * LOG2E) * fmaf(c1, lnp, c0);
    if (v == tok) r += g;
    return r;
  };
  const int v0 = seg * grad_cols<TX>(), v1 = min(V, v0 + grad_cols<TX>());
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(d)) & 15) == 0;
  if (vec) {
    uint4 u[GRAD_VECS];
#pragma unroll
    for (int j = 0; j < GRAD_VECS; ++j) {
      const int v = v0 + (threadIdx.x + j * NT) * N;
      u[j] = v + N <= v1 && !zero ? *reinterpret_cast<const uint4*>(x + v) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < GRAD_VECS; ++j) {
      const int v = v0 + (threadIdx.x + j * NT) * N;
      if (v + N <= v1) {
        float f[N];
        alignas(16) TX o[N];
        Vec<TX>::unpack(u[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = from_f32<TX>(zero ? 0.f : one(f[i], v + i));
        *reinterpret_cast<uint4*>(d + v) = *reinterpret_cast<const uint4*>(o);
      } else {
        for (int i = v; i < v1; ++i) d[i] = from_f32<TX>(zero ? 0.f : one(to_f32(x[i]), i));
      }
    }
  } else {
    // rows whose logits and gradients do not both start on 16 bytes
    for (int v = v0 + threadIdx.x; v < v1; v += NT) d[v] = from_f32<TX>(zero ? 0.f : one(to_f32(x[v]), v));
  }
}

}  // namespace lp
}  // namespace quip
