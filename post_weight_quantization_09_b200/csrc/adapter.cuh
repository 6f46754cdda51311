// Low-rank adapters beside a shared (quantised) projection: every token of a
// batch names one of `count` adapters, or none,
//   h_t = P_l x_t          (P: r x n, "shrink")
//   y_t = base_t + s_l Q_l^T h_t   (Q: r x m, "expand"),  l = ids_t.
// Both factors are stored as r rows of the layer's width, so the gradient's
// products dh_t = s_l up_l dy_t and dx_t = base_t + down_l^T dh_t are the same
// kernel with P = up, Q = down, and the two weight gradients
//   d_down_l = sum_t dh_t x_t^T,  d_up_l = s_l sum_t h_t dy_t^T
// are one kernel for an outer product summed over an adapter's tokens.
//
// Forward and gradient of the activations take 2 T r (n + m) flops each, the
// weight gradients as much; at ranks up to 64 the bytes of x, y and dy are the
// floor of all of them (rank 64 does 64 flops a byte, the GPU 250).  What
// bounds each kernel as built stands there.
//
// By the number of tokens (adapter_direct in quip_api.cu): few go straight
// from ids, a cluster per token; more are grouped by adapter first (the plan)
// and taken in tiles of 128 tokens on the tensor cores.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace quip {
namespace adapter {

namespace cg = cooperative_groups;

constexpr int MAX_COUNT = QUIP_ADAPTER_MAX_COUNT;
constexpr int MAX_RANK = QUIP_ADAPTER_MAX_RANK;

// ---------------------------------------------------------------- plan
// The batch's tokens grouped by adapter (int32 words, device memory):
//   header  HEAD words
//   start   count + 2: where adapter l's tokens begin in `order`; entry
//           `count` is the tokens without an adapter, entry count + 1 is T
//   order   T: the tokens, by adapter, within one in their own order
//   tiles   (adapter, first position in order) of up to TILE tokens of one
//           adapter each, those without an adapter last (adapter `count`)
//   small   the same for SMALL tokens
//   chunks  the same for CHUNK tokens, for the sums over an adapter's tokens:
//           every adapter has one at least; (adapter, first, slot, sub), slot =
//           -1 for an adapter's only chunk, else its place among the partial
//           sums; sub: the number of its first SUB tokens among all runs of SUB
//   parts   (first slot, number of slots) per adapter, 0 slots with one chunk
constexpr int HEAD = 16, TILE = 128, SMALL = 8, CHUNK = 1024, SUB = 64;
enum { H_MAGIC, H_T, H_COUNT, H_TILES, H_SMALL, H_CHUNKS };
constexpr int MAGIC = 0x51AD;

struct PlanView {
  int32_t *head, *start, *order;
  int2 *tiles, *small;
  int4* chunks;
  int2* parts;
};
__host__ __device__ inline int64_t max_tiles(int64_t T, int64_t count, int size) { return T / size + count + 1; }
// Chunks that belong to adapters of several: fewer than 2 T / CHUNK.
__host__ __device__ inline int64_t max_slots(int64_t T) { return 2 * (T / CHUNK); }
__host__ __device__ inline int64_t up4(int64_t v) { return (v + 3) / 4 * 4; }
__host__ __device__ inline int64_t plan_words(int64_t T, int64_t count) {
  return HEAD + up4(count + 2) + up4(T) + up4(2 * max_tiles(T, count, TILE)) + up4(2 * max_tiles(T, count, SMALL)) +
         4 * max_tiles(T, count, CHUNK) + up4(2 * count);
}
__host__ __device__ inline PlanView plan_view(void* plan, int64_t T, int64_t count) {
  int32_t* p = static_cast<int32_t*>(plan);
  PlanView v;
  v.head = p;
  v.start = p + HEAD;
  v.order = v.start + up4(count + 2);
  v.tiles = reinterpret_cast<int2*>(v.order + up4(T));
  v.small = reinterpret_cast<int2*>(reinterpret_cast<int32_t*>(v.tiles) + up4(2 * max_tiles(T, count, TILE)));
  v.chunks = reinterpret_cast<int4*>(reinterpret_cast<int32_t*>(v.small) + up4(2 * max_tiles(T, count, SMALL)));
  v.parts = reinterpret_cast<int2*>(v.chunks + max_tiles(T, count, CHUNK));
  return v;
}

// Latency bound (7 us for 4096 tokens, 11 for 8192); a model makes it once per
// batch for all its layers.
// One CTA of 32 warps: a stable counting sort of the tokens by adapter, each
// warp a contiguous share of the tokens with counters of its own (a warp's
// equal ids are ranked by match.any), then the tables.  Shared memory:
// 32 x (count + 1) counters (later 7 numbers per adapter).
constexpr int PLAN_WARPS = 32;
inline size_t plan_smem(int64_t count) { return (size_t)PLAN_WARPS * (count + 1) * sizeof(int); }

// Exclusive sums of N numbers over 1024 threads, and their totals.
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&total)[N], int (*warp_sums)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] += u;
    }
    if (lane == 31) warp_sums[warp][k] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int s = warp_sums[lane][k];
    int scan = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += u;
    }
    total[k] = __shfl_sync(0xffffffffu, scan, 31);
    v[k] = __shfl_sync(0xffffffffu, scan - s, warp) + inc[k] - v[k];
  }
}

__global__ void __launch_bounds__(PLAN_WARPS * 32)
    k_adapter_plan(const int32_t* __restrict__ ids, int T, int count, void* plan) {
  extern __shared__ int counters[];            // [warp][count + 1]
  enum { FIRST, TILES, SMALLS, CHUNKS, SLOTS, SUBS, SCANS };
  __shared__ int warp_sums[32][SCANS];
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, T, count);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = count + 1;
  int* mine = counters + warp * nb;
  for (int i = lane; i < nb; i += 32) mine[i] = 0;
  __syncwarp();
  const int per = (T + PLAN_WARPS * 32 - 1) / (PLAN_WARPS * 32) * 32;
  const int t0 = min(T, warp * per), t1 = min(T, t0 + per);
  auto bucket = [&](int t, bool report) {
    int b = ids[t];
    if (b >= count && report) record_status(QUIP_ERR_ARG);
    return b < 0 || b >= count ? count : b;
  };
  constexpr int AHEAD = 8;                     // rounds whose ids are loaded together
  for (int t = t0; t < t1; t += 32 * AHEAD) {
    int b[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) b[k] = t + 32 * k + lane < t1 ? bucket(t + 32 * k + lane, true) : -1;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (t + 32 * k >= t1) break;
      const unsigned same = __match_any_sync(0xffffffffu, b[k]);
      if (b[k] >= 0 && lane == __ffs(same) - 1) mine[b[k]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // per bucket: the warps' counts to offsets within it
  int total = 0, counts[PLAN_WARPS];
  if (tid < count) {
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) counts[w] = counters[w * nb + tid];
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) total += counts[w];
  }
  const int my_chunks = tid < count ? max(1, (total + CHUNK - 1) / CHUNK) : 0;
  const int my_slots = my_chunks > 1 ? my_chunks : 0;
  int v[SCANS] = {total, (total + TILE - 1) / TILE, (total + SMALL - 1) / SMALL, my_chunks, my_slots, (total + SUB - 1) / SUB};
  int all[SCANS];
  block_scan(v, all, warp_sums);
  const int with = all[FIRST], ntile = all[TILES], nsmall = all[SMALLS], nchunk = all[CHUNKS];
  if (tid < count) {
    pv.start[tid] = v[FIRST];
    pv.parts[tid] = make_int2(v[SLOTS], my_slots);
    int at = v[FIRST];
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) {
      counters[w * nb + tid] = at;
      at += counts[w];
    }
  }
  if (tid == 0) {
    int at = with;                             // the tokens without an adapter come last
    for (int w = 0; w < PLAN_WARPS; ++w) {
      const int c = counters[w * nb + count];
      counters[w * nb + count] = at;
      at += c;
    }
    pv.start[count] = with;
    pv.start[count + 1] = T;
    pv.head[H_MAGIC] = MAGIC;
    pv.head[H_T] = T;
    pv.head[H_COUNT] = count;
    pv.head[H_TILES] = ntile + (T - with + TILE - 1) / TILE;
    pv.head[H_SMALL] = nsmall + (T - with + SMALL - 1) / SMALL;
    pv.head[H_CHUNKS] = nchunk;
  }
  __syncthreads();
  for (int t = t0; t < t1; t += 32 * AHEAD) {
    int b[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) b[k] = t + 32 * k + lane < t1 ? bucket(t + 32 * k + lane, false) : -1;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (t + 32 * k >= t1) break;
      const unsigned same = __match_any_sync(0xffffffffu, b[k]);
      if (b[k] >= 0) pv.order[mine[b[k]] + __popc(same & ((1u << lane) - 1u))] = t + 32 * k + lane;
      __syncwarp();
      if (b[k] >= 0 && lane == __ffs(same) - 1) mine[b[k]] += __popc(same);
      __syncwarp();
    }
  }
  // the tables, a warp per adapter: thread l's numbers go through shared memory
  __syncthreads();
  if (tid < count) {
    int* c = counters + tid * 7;
    c[0] = v[FIRST], c[1] = total, c[2] = v[TILES], c[3] = v[SMALLS], c[4] = v[CHUNKS];
    c[5] = my_slots ? v[SLOTS] : -1, c[6] = v[SUBS];
  }
  __syncthreads();
  for (int l = warp; l <= count; l += PLAN_WARPS) {
    const bool none = l == count;
    const int* n = counters + l * 7;
    const int f = none ? with : n[0], c = none ? T - with : n[1], t = none ? ntile : n[2], s = none ? nsmall : n[3];
    for (int i = lane; i * TILE < c; i += 32) pv.tiles[t + i] = make_int2(l, f + i * TILE);
    for (int i = lane; i * SMALL < c; i += 32) pv.small[s + i] = make_int2(l, f + i * SMALL);
    if (!none)
      for (int i = lane; i == 0 || i * CHUNK < c; i += 32)
        pv.chunks[n[4] + i] = make_int4(l, f + i * CHUNK, n[5] < 0 ? -1 : n[5] + i, n[6] + i * (CHUNK / SUB));
  }
}

// ---------------------------------------------------------------- helpers

// Four consecutive values as fp32; `vec`: one aligned load, else element by
// element, `left` of them there (the others 0).
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, bool vec, int left);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p, bool vec, int left) {
  if (vec && left >= 4) return __ldg(reinterpret_cast<const float4*>(p));
  return make_float4(left > 0 ? p[0] : 0.f, left > 1 ? p[1] : 0.f, left > 2 ? p[2] : 0.f, left > 3 ? p[3] : 0.f);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p, bool vec, int left) {
  if (vec && left >= 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  }
  auto at = [&](int i) { return left > i ? __bfloat162float(p[i]) : 0.f; };
  return make_float4(at(0), at(1), at(2), at(3));
}
// y[0..4) = base[0..4) + v; base may be null or y itself.
template <typename T>
__device__ __forceinline__ void put(T* y, float v);
template <>
__device__ __forceinline__ void put<float>(float* y, float v) { *y = v; }
template <>
__device__ __forceinline__ void put<__nv_bfloat16>(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
template <typename T>
__device__ __forceinline__ void add4(T* y, const T* base, float4 v, bool vec, int left) {
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec && left >= 4) {
    if constexpr (sizeof(T) == 4) {
      if (base) b = *reinterpret_cast<const float4*>(base);
      *reinterpret_cast<float4*>(y) = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
    } else {
      if (base) {
        const uint2 u = *reinterpret_cast<const uint2*>(base);
        b = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                        __uint_as_float(u.y & 0xFFFF0000u));
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(b.x + v.x, b.y + v.y), hi = __floats2bfloat162_rn(b.z + v.z, b.w + v.w);
      *reinterpret_cast<uint2*>(y) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    return;
  }
  const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) put(y + i, (base ? to_f32(base[i]) : 0.f) + w[i]);
}

template <typename TX, typename TW, typename TY>
struct ApplyArgs {
  const TX* x;                 // T x n
  int64_t ldx;
  const TW *P, *Q;             // count x r x n, count x r x m
  const float* scale;          // count, or null: 1
  const TY* base;              // T x m, null: 0; may be y
  int64_t ldb;
  TY* y;                       // T x m, null: no expand
  int64_t ldy;
  float* h;                    // T x r, or null
  int T, n, m, r, count;
  bool h_scaled;               // h gets s_l P_l x_t instead of P_l x_t
  bool vec_x, vec_p, vec_q, vec_y;   // rows that allow the kernel's vector loads
  bool fast_y;                 // 16-byte rows of base and y at equal, 32-bit offsets (in units of 16 bytes)
};

// The plan of a call must be one made for its T and count.
__device__ __forceinline__ bool plan_ok(const PlanView& pv, int T, int count) {
  const bool ok = pv.head[H_MAGIC] == MAGIC && pv.head[H_T] == T && pv.head[H_COUNT] == count;
  if (!ok && threadIdx.x == 0) record_status(QUIP_ERR_ARG);
  return ok;
}

// ---------------------------------------------------------------- single tokens
// Decode: one cluster per token, straight from ids (no plan), bound by the
// latency of its chain of loads.  The CTAs of a cluster share n and m.  All
// that does not wait for h is asked for at once: P and x for the shrink, and
// each thread's first columns of Q and the base for the expand.  Every CTA
// stores its partial h into all others' shared memory and, past one cluster
// barrier, adds them up in rank order.  fp32 on the CUDA cores; any type,
// rank and alignment.  4096 x 4096, rank 16: 5.8 us for one token (9.2 us with
// x staged in shared memory and Q asked for after h); 4096 -> 11008, 64 tokens
// over 32 adapters: 13.1 us (21.6 us; 22 MB).
constexpr int VT = 256;                        // threads per CTA
constexpr int EARLY = 16;                      // rows of Q asked for at once
constexpr int TOKEN_CTAS = 8;                  // of a cluster, at most

// Four consecutive values as they lie in memory.  CONST: nothing writes them
// while the kernel runs (base may be y itself).
template <typename T> struct Four;
template <> struct Four<float> {
  float4 v;
  template <bool CONST = true>
  __device__ __forceinline__ void load(const float* p, bool vec, int left) {
    if (!CONST && vec && left >= 4) v = *reinterpret_cast<const float4*>(p);
    else v = load4(p, vec, left);
  }
  __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct Four<__nv_bfloat16> {
  uint2 v;
  template <bool CONST = true>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec, int left) {
    if (vec && left >= 4) {
      v = CONST ? __ldg(reinterpret_cast<const uint2*>(p)) : *reinterpret_cast<const uint2*>(p);
    } else {
      auto at = [&](int i) { return i < left ? (uint32_t)__bfloat16_as_ushort(p[i]) : 0u; };
      v = make_uint2(at(0) | at(1) << 16, at(2) | at(3) << 16);
    }
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
  }
};

template <typename TX, typename TW, typename TY>
__global__ void __launch_bounds__(VT, sizeof(TW) == 2 ? 4 : 2)
    k_adapter_token(const __grid_constant__ ApplyArgs<TX, TW, TY> a, const int32_t* __restrict__ ids) {
  constexpr int R = 2;                         // rows of P per warp at once
  __shared__ float parts[TOKEN_CTAS][MAX_RANK];    // written by the cluster
  __shared__ float hs[MAX_RANK];
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = a.r;
  const int64_t token = blockIdx.x / nc;
  auto running = cluster.barrier_arrive();     // the others' shared memory may be written past this
  pdl_wait_then_release();
  int l = ids[token];
  if (l >= a.count && rank == 0 && tid == 0) record_status(QUIP_ERR_ARG);
  if (l >= a.count) l = -1;
  const int m_per = ((a.m + nc - 1) / nc + 3) / 4 * 4, m0 = min(a.m, rank * m_per), m1 = min(a.m, m0 + m_per);
  const int n_per = ((a.n + nc - 1) / nc + 3) / 4 * 4, n0 = min(a.n, rank * n_per), n1 = min(a.n, n0 + n_per);
  const TX* x = a.x + token * a.ldx;
  const TY* base = a.base ? a.base + token * a.ldb : nullptr;
  TY* y = a.y ? a.y + token * a.ldy : nullptr;
  const int c0 = m0 + 4 * tid;                 // this thread's first columns
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (l < 0) {                                 // no adapter: y = base, h = 0
    if (rank == 0 && a.h)
      for (int i = tid; i < r; i += VT) a.h[token * r + i] = 0.f;
    if (y && a.y != a.base)
      for (int c = c0; c < m1; c += 4 * VT) add4(y + c, base ? base + c : nullptr, zero, a.vec_y, m1 - c);
    cluster.barrier_wait(std::move(running));
    return;
  }
  const TW* P = a.P + (int64_t)l * r * a.n;
  const TW* Q = a.Q + (int64_t)l * r * a.m;
  Four<TW> early[EARLY];
  Four<TY> early_base;
  if (y && c0 < m1) {
#pragma unroll
    for (int j = 0; j < EARLY; ++j) early[j].load(Q + (int64_t)min(j, r - 1) * a.m + c0, a.vec_q, m1 - c0);
    if (base) early_base.template load<false>(base + c0, a.vec_y, m1 - c0);
  }
  cluster.barrier_wait(std::move(running));
  for (int j0 = R * warp; j0 < r; j0 += R * (VT / 32)) {
    float acc[R];
#pragma unroll
    for (int k = 0; k < R; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int c = n0 + 4 * lane; c < n1; c += 128) {
      Four<TX> xv;
      xv.load(x + c, a.vec_x, n1 - c);
      const float4 v = xv.get();
#pragma unroll
      for (int k = 0; k < R; ++k) {
        Four<TW> wv;
        wv.load(P + (int64_t)min(j0 + k, r - 1) * a.n + c, a.vec_p, n1 - c);
        const float4 w = wv.get();
        acc[k] = fmaf(w.x, v.x, acc[k]);
        acc[k] = fmaf(w.y, v.y, acc[k]);
        acc[k] = fmaf(w.z, v.z, acc[k]);
        acc[k] = fmaf(w.w, v.w, acc[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      acc[k] = warp_sum(acc[k]);
      if (lane < nc && j0 + k < r) *cluster.map_shared_rank(&parts[rank][j0 + k], lane) = acc[k];
    }
  }
  cluster.sync();
  const float scale = a.scale ? a.scale[l] : 1.f;
  if (tid < r) {
    float v = 0.f;
    for (int c = 0; c < nc; ++c) v += parts[c][tid];
    hs[tid] = v * scale;
    if (rank == 0 && a.h) a.h[token * r + tid] = a.h_scaled ? v * scale : v;
  }
  __syncthreads();
  if (!y) return;
  auto add = [&](float4& acc, const float4& w, float v) {
    acc.x = fmaf(w.x, v, acc.x);
    acc.y = fmaf(w.y, v, acc.y);
    acc.z = fmaf(w.z, v, acc.z);
    acc.w = fmaf(w.w, v, acc.w);
  };
  for (int c = c0; c < m1; c += 4 * VT) {
    float4 acc = zero;
    if (c != c0) {
#pragma unroll
      for (int j = 0; j < EARLY; ++j) early[j].load(Q + (int64_t)min(j, r - 1) * a.m + c, a.vec_q, m1 - c);
      if (base) early_base.template load<false>(base + c, a.vec_y, m1 - c);
    }
#pragma unroll
    for (int j = 0; j < EARLY; ++j)
      if (j < r) add(acc, early[j].get(), hs[j]);
#pragma unroll 8
    for (int j = EARLY; j < r; ++j) {
      Four<TW> w;
      w.load(Q + (int64_t)j * a.m + c, a.vec_q, m1 - c);
      add(acc, w.get(), hs[j]);
    }
    if (base) {
      const float4 b = early_base.get();
      acc = make_float4(b.x + acc.x, b.y + acc.y, b.z + acc.z, b.w + acc.w);
    }
    add4<TY>(y + c, nullptr, acc, a.vec_y, m1 - c);
  }
}

// ---------------------------------------------------------------- vectors
// For the types and ranks that the tensor-core tiles do not take: the plan's
// tiles of up to SMALL tokens of one adapter, one cluster each.  Its CTAs
// share n, exchange their partial h through distributed shared memory
// (summed in rank order by each), and share m.  fp32 on the CUDA cores; the
// factors come from L2 once per 8 tokens, which bounds it.
constexpr int NTOK = SMALL, VROWS = 4, VCOLS = 1024;   // tokens; rows of P per warp task; columns of x staged at once
inline size_t vec_smem(int r) {
  return sizeof(float) * ((size_t)NTOK * VCOLS + (size_t)(VT / 32) * NTOK * VROWS + 2 * (size_t)NTOK * up4(r));
}

template <typename TX, typename TW, typename TY>
__global__ void __launch_bounds__(VT)
    k_adapter_vec(const __grid_constant__ ApplyArgs<TX, TW, TY> a, void* plan) {
  constexpr int R = VROWS, COLS = VCOLS;
  extern __shared__ __align__(16) float sm[];
  __shared__ int tok[NTOK];
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / nc;
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, a.T, a.count);
  if (!plan_ok(pv, a.T, a.count) || unit >= pv.head[H_SMALL]) return;      // the whole cluster
  const int2 tile = pv.small[unit];
  const int l = tile.x, cnt = min(NTOK, pv.start[l + 1] - tile.y);
  if (tid < NTOK) tok[tid] = tid < cnt ? pv.order[tile.y + tid] : -1;
  __syncthreads();
  const int r = a.r, r4 = (int)up4(r);
  float* xs = sm;                              // [NTOK][COLS]
  float* parts = xs + NTOK * COLS;             // [warp][R][NTOK] of a warp's rows
  float* hpart = parts + (VT / 32) * NTOK * R; // [r4][NTOK], read by the cluster
  float* hs = hpart + NTOK * r4;               // [r4][NTOK], times the scale
  const int m_per = ((a.m + nc - 1) / nc + 3) / 4 * 4;
  const int m0 = min(a.m, rank * m_per), m1 = min(a.m, m0 + m_per);
  if (l == a.count) {                          // no adapter: y = base, h = 0
    if (rank == 0 && a.h)
      for (int i = tid; i < cnt * r; i += VT) a.h[(int64_t)tok[i / r] * r + i % r] = 0.f;
    if (a.y && a.y != a.base)
      for (int t = 0; t < cnt; ++t) {
        const int64_t row = tok[t];
        for (int c = m0 + 4 * tid; c < m1; c += 4 * VT)
          add4(a.y + row * a.ldy + c, a.base ? a.base + row * a.ldb + c : nullptr, make_float4(0.f, 0.f, 0.f, 0.f),
               a.vec_y, m1 - c);
      }
    return;
  }
  const TW* P = a.P + (int64_t)l * r * a.n;
  const TW* Q = a.Q + (int64_t)l * r * a.m;
  const float scale = a.scale ? a.scale[l] : 1.f;
  // ---- shrink: hpart[j][t] = sum over this CTA's columns of P[j][c] x[t][c]
  const int n_per = ((a.n + nc - 1) / nc + 3) / 4 * 4;
  const int n0 = min(a.n, rank * n_per), n1 = min(a.n, n0 + n_per);
  for (int i = tid; i < NTOK * r4; i += VT) hpart[i] = 0.f;
  const int tasks = (r + R - 1) / R;
  // few rows: the warps share their columns (1 to 8 of them; 8 is a multiple)
  const int share = tasks >= VT / 32 ? 1 : (VT / 32) / tasks;
  for (int c0 = n0; c0 < n1; c0 += COLS) {
    const int nc4 = (min(COLS, n1 - c0) + 3) / 4;
    __syncthreads();
    for (int i = tid; i < NTOK * nc4; i += VT) {
      const int t = i / nc4, q = i % nc4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tok[t] >= 0) v = load4(a.x + (int64_t)tok[t] * a.ldx + c0 + 4 * q, a.vec_x, n1 - c0 - 4 * q);
      reinterpret_cast<float4*>(xs + t * COLS)[q] = v;
    }
    __syncthreads();
    for (int task = warp / share; task < tasks; task += (VT / 32) / share) {
      const int j0 = task * R;
      float acc[R][NTOK];
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int t = 0; t < NTOK; ++t) acc[k][t] = 0.f;
#pragma unroll 4
        for (int q = lane + 32 * (warp % share); q < nc4; q += 32 * share) {
          const int left = n1 - c0 - 4 * q;
          float4 w[R];
#pragma unroll
          for (int k = 0; k < R; ++k)
            w[k] = j0 + k < r ? load4(P + (int64_t)(j0 + k) * a.n + c0 + 4 * q, a.vec_p, left)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int t = 0; t < NTOK; ++t) {
            const float4 v = reinterpret_cast<const float4*>(xs + t * COLS)[q];
#pragma unroll
            for (int k = 0; k < R; ++k) {
              acc[k][t] = fmaf(w[k].x, v.x, acc[k][t]);
              acc[k][t] = fmaf(w[k].y, v.y, acc[k][t]);
              acc[k][t] = fmaf(w[k].z, v.z, acc[k][t]);
              acc[k][t] = fmaf(w[k].w, v.w, acc[k][t]);
            }
          }
        }
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int t = 0; t < NTOK; ++t) acc[k][t] = warp_sum(acc[k][t]);
      if (share == 1) {
        if (lane == 0)
#pragma unroll
          for (int k = 0; k < R; ++k)
#pragma unroll
            for (int t = 0; t < NTOK; ++t)
              if (j0 + k < r) hpart[(j0 + k) * NTOK + t] += acc[k][t];
      } else if (lane == 0) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
          for (int t = 0; t < NTOK; ++t) parts[(warp * R + k) * NTOK + t] = acc[k][t];
      }
    }
    if (share > 1) {                           // one task per warp: add its sharers in order
      __syncthreads();
      for (int i = tid; i < tasks * R * NTOK; i += VT) {
        const int task = i / (R * NTOK), e = i % (R * NTOK);
        float v = 0.f;
        for (int s = 0; s < share; ++s) v += parts[(task * share + s) * R * NTOK + e];
        if (task * R + e / NTOK < r) hpart[task * R * NTOK + e] += v;
      }
    }
  }
  cluster.sync();
  for (int i = tid; i < r * NTOK; i += VT) {
    float v = 0.f;
    for (int c = 0; c < nc; ++c) v += *cluster.map_shared_rank(hpart + i, c);
    const int t = i % NTOK;
    hs[i] = v * scale;
    if (rank == 0 && a.h && t < cnt) a.h[(int64_t)tok[t] * r + i / NTOK] = a.h_scaled ? v * scale : v;
  }
  cluster.sync();                              // everybody has read hpart; hs is there
  if (!a.y) return;
  // ---- expand: y[t][c] = base[t][c] + sum_j Q[j][c] hs[j][t]
  for (int c = m0 + 4 * tid; c < m1; c += 4 * VT) {
    float4 acc[NTOK];
#pragma unroll
    for (int t = 0; t < NTOK; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < r; ++j) {
      const float4 w = load4(Q + (int64_t)j * a.m + c, a.vec_q, m1 - c);
#pragma unroll
      for (int t = 0; t < NTOK; ++t) {
        const float v = hs[j * NTOK + t];
        acc[t].x = fmaf(w.x, v, acc[t].x);
        acc[t].y = fmaf(w.y, v, acc[t].y);
        acc[t].z = fmaf(w.z, v, acc[t].z);
        acc[t].w = fmaf(w.w, v, acc[t].w);
      }
    }
#pragma unroll
    for (int t = 0; t < NTOK; ++t)
      if (t < cnt) {
        const int64_t row = tok[t];
        add4(a.y + row * a.ldy + c, a.base ? a.base + row * a.ldb + c : nullptr, acc[t], a.vec_y, m1 - c);
      }
  }
}

// ---------------------------------------------------------------- tiles on the tensor cores
// Tiles of up to 128 tokens of one adapter, in two launches.
//
// Shrink: one cluster per tile whose CTAs share n: each accumulates
// h[token][j] over its 64-column blocks with tcgen05 (M = 128 tokens, N = r,
// both operands K-major), the partial sums meet through distributed shared
// memory (each CTA adds up a share of the tokens, in rank order), h goes to
// memory.  8192 tokens of 11008 bf16 columns, rank 32: 39 us, 4.6 TB/s (27 us
// at the measured copy rate); 4096 of 8192, rank 64: 25 us, mostly the start
// and the cluster's sum.
//
// Expand: resident CTAs, each an equal run of the (tile, column block) pairs:
// D[token][column] = h Q (M = 128 tokens, N = the block's columns, K = r, Q
// MN-major as it lies in memory).  Three warps fetch Q's tiles, one multiplies; the others, in up to
// four groups of four, take a block in turn, 32 tokens (TMEM lanes) each: a warp
// brings its rows of the base to shared memory, 256 bytes at a time by 16
// neighbouring lanes, adds a row's products there, and sends the sums out as
// the base came, while the other groups' rows are on their way.  The sides
// meet at mbarriers only (tile of Q there, accumulator full, accumulator read).
// 4096 tokens x 28672 bf16 columns, rank 64: 106 us, 4.4 TB/s (72 us at the
// copy rate; 140 us with two CTAs an SM that met at every block, 200 us with
// each lane on its own row's bytes).  By clocks read in the kernel the
// multiplying warp bounds it: of 2450 clocks a block it spends 1180 on its
// eight products, 620 on the fence and the commit around them, 290 waiting;
// a group of row warps needs a block's rows for 5100 of 4 x 2450.
//
// Types: a bf16 value is one operand piece, an fp32 value three (split3), and
// the products of pieces of order 2 and below are formed: fp32 operands keep
// fp32 accuracy.  h is fed to the second product in pieces too: two for a
// bf16 output (2^-17 is left, its rounding is 2^-9), three for an fp32 one.
// The tensor core drops low bits of the running sum at every step (of 16
// products), so the 64-column blocks of n are dealt out over several
// accumulators, 1024 columns to each at most, that are added in fp32
// (ShrinkAccs).
//
// Loads are gathered by token into shared memory with the 128-byte swizzle,
// by cp.async where bf16 rows allow 16-byte copies (CP), else through
// registers, which also cuts fp32 values into pieces and takes any alignment.
// Each stage has warps of its own that fill it, wait for it and hand it on.
template <typename T> __host__ __device__ constexpr int pieces() { return sizeof(T) == 2 ? 1 : 3; }
template <typename TY> __host__ __device__ constexpr int h_pieces() { return sizeof(TY) == 2 ? 2 : 3; }
constexpr int XT_BYTES = TILE * 128;           // one piece of 128 tokens x 64 columns

template <typename TX, typename TW>
__host__ __device__ inline int shrink_stage(int r16) { return pieces<TX>() * XT_BYTES + pieces<TW>() * r16 * 128; }
// Warps per stage (four where registers are between), and threads: four stages
// and a warp to multiply.
template <bool CP> __host__ __device__ constexpr int stage_warps() { return CP ? 2 : 4; }
template <bool CP> __host__ __device__ constexpr int stage_threads() { return 32 * (4 * stage_warps<CP>() + 1); }
// four, but three where that lets two CTAs on an SM (bf16, ranks above 64) or
// one at all
__host__ __device__ inline int shrink_stages(int stage) {
  return stage <= 24 * 1024 || (stage > 32 * 1024 && stage <= 55 * 1024) ? 4 : 3;
}
template <typename TX, typename TW>
__host__ __device__ inline int shrink_smem(int r16) {
  const int stage = shrink_stage<TX, TW>(r16);
  int s = shrink_stages(stage) * stage;
  const int hp = TILE * (r16 + 4) * 4;         // the partial h, in the stages' place
  if (hp > s) s = hp;
  s += 1024;
  // at most two CTAs on an SM, which hold 2 x 256 TMEM columns (bf16; with an
  // fp32 operand the stages take 168 KB and more: one, with 512), so no CTA
  // of a cluster ever waits for TMEM while its peers wait for it
  return s < 78 * 1024 ? 78 * 1024 : s;
}
// A block of the expand step is 256 bytes of y's rows; Q's tiles in flight and
// groups with a block's rows, as many as fit.
template <typename TY> __host__ __device__ constexpr int expand_cols() { return 256 / (int)sizeof(TY); }
constexpr int EW = 16, QW = 3, ET = 32 * (EW + QW + 1);    // warps: rows of y, tiles of Q, multiply
constexpr int ROW_BYTES = TILE * 256, EXPAND_MAX = 226 * 1024;
constexpr int ACCS = 4;                        // blocks' accumulators in TMEM
struct ExpandRings {
  int q, rows, smem;
};
template <typename TW, typename TY>
__host__ __device__ inline int expand_tile(int r16) { return pieces<TW>() * r16 * 2 * expand_cols<TY>(); }
template <typename TW, typename TY>
inline ExpandRings expand_rings(int r16) {
  const int h = h_pieces<TY>() * ((r16 + 63) / 64) * XT_BYTES + 1024, tile = expand_tile<TW, TY>(r16);
  ExpandRings e{QW, 4, 0};
  while (e.rows > 3 && h + e.q * tile + e.rows * ROW_BYTES > EXPAND_MAX) --e.rows;
  while (e.q > 2 && h + e.q * tile + e.rows * ROW_BYTES > EXPAND_MAX) --e.q;
  while (e.rows > 1 && h + e.q * tile + e.rows * ROW_BYTES > EXPAND_MAX) --e.rows;
  e.smem = h + e.q * tile + e.rows * ROW_BYTES;
  return e;
}

// The first `bytes` of 16, zeros behind them.
__device__ __forceinline__ void cp16(uint8_t* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint8_t* dst, const void* src, bool there) { cp16(dst, src, there ? 16 : 0); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight consecutive values in registers.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec, int left) {
    if (vec && left >= 8) {
      v = __ldg(reinterpret_cast<const uint4*>(p));
      return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < left ? __bfloat16_as_ushort(p[2 * i]) : 0u;
      const uint32_t hi = 2 * i + 1 < left ? __bfloat16_as_ushort(p[2 * i + 1]) : 0u;
      w[i] = lo | hi << 16;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(uint8_t* at, int) const { *reinterpret_cast<uint4*>(at) = v; }
};
// Eight fp32 values as NP bf16 pieces, `step` bytes apart: each piece rounds
// what the ones before it leave (as split3, two values at a time).
template <int NP>
__device__ __forceinline__ void store_pieces(uint8_t* at, int step, const float (&f)[8]) {
  uint32_t w[NP][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i], b = f[2 * i + 1];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      w[p][i] = *reinterpret_cast<const uint32_t*>(&v);
      a -= __uint_as_float(w[p][i] << 16);
      b -= __uint_as_float(w[p][i] & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(at + p * step) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p, bool vec, int left) {
    a = load4(p, vec, left);
    b = load4(p + 4, vec, left - 4);
  }
  __device__ __forceinline__ void store(uint8_t* at, int step) const {
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    store_pieces<3>(at, step, f);
  }
};

// The accumulators of a CTA's `steps` blocks, r16 TMEM columns each: `mains`
// take the large terms of the blocks in turn, `low` = 1 more, behind them, the
// small terms of operands in pieces.  8 blocks (512 columns) meet in one where
// TMEM has room, else up to 16; beyond, `round` blocks at a time (0: all at
// once) are added up in fp32 and kept in the place behind these.  Sums of
// 28672 positive fp32 terms in one CTA, rank 12, are off by 13 u on average (u
// = 2^-24; by 600 u with all blocks in three accumulators).  The rounds' waits
// cost 4096 bf16 tokens x 28672, rank 128, 83 us for 77.
struct ShrinkAccs {
  int mains, low, round;
};
template <bool SPLIT> __host__ __device__ constexpr int shrink_cols() { return SPLIT ? 512 : 256; }
template <bool SPLIT>
__host__ __device__ inline ShrinkAccs shrink_accs(int r16, int steps) {
  const int low = SPLIT ? 1 : 0, most = shrink_cols<SPLIT>() / r16 - low, usual = (r16 <= 64 ? 4 : 2) - low;
  if (steps > 16 * most) return {most - 1, low, 16 * (most - 1)};
  const int want = (steps + 7) / 8;
  return {want < usual ? usual : want < most ? want : most, low, 0};
}

// The sum of accumulators 0 .. last into the columns from `to` on, the last
// first; columns j0, j0 + step, ... by sixteen.
__device__ __noinline__ void keep_round(uint32_t lanes, int j0, int step, int r16, int last, int to) {
  for (int j = j0; j < r16; j += step) {
    float v[16];
    tmem_ld16(lanes + last * r16 + j, v);
    for (int q = last - 1; q >= 0; --q) {
      float w[16];
      tmem_ld16(lanes + q * r16 + j, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] += w[e];
    }
    tmem_st16(lanes + to + j, v);
  }
}
// acc: of the cluster's largest share of n; KEEP: with rounds.
template <typename TX, typename TW, bool CP, bool KEEP>
__global__ void __launch_bounds__(stage_threads<CP>(), CP ? 2 : 1)
    k_adapter_shrink(const __grid_constant__ ApplyArgs<TX, TW, float> a, const __grid_constant__ ShrinkAccs acc, void* plan) {
  constexpr int PX = pieces<TX>(), PW = pieces<TW>(), SW = stage_warps<CP>(), ST = stage_threads<CP>();
  constexpr bool SPLIT = PX > 1 || PW > 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int tok[TILE];
  __shared__ uint64_t full[4], empty[4], all_done, round_done, round_kept;
  __shared__ uint32_t tmem_base;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, a.T, a.count);
  const int unit = blockIdx.x / nc;
  if (!plan_ok(pv, a.T, a.count) || unit >= pv.head[H_TILES]) return;      // the whole cluster
  const int2 tile = pv.tiles[unit];
  const int l = tile.x, cnt = min(TILE, pv.start[l + 1] - tile.y), r = a.r;
  if (tid < TILE) tok[tid] = tid < cnt ? pv.order[tile.y + tid] : -1;
  if (l == a.count) {                          // no adapter: h = 0
    __syncthreads();
    for (int i = rank * ST + tid; i < cnt * r; i += nc * ST) a.h[(int64_t)tok[i / r] * r + i % r] = 0.f;
    return;
  }
  const int r16 = (r + 15) / 16 * 16, stage = shrink_stage<TX, TW>(r16), stages = shrink_stages(stage);
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int blocks = (a.n + 63) / 64, per = (blocks + nc - 1) / nc;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&full[i], SW), mbar_init(&empty[i], 1);
    mbar_init(&all_done, 1), mbar_init(&round_done, 1), mbar_init(&round_kept, 4 * SW);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&tmem_base, shrink_cols<SPLIT>());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;                  // a wait that ran out is the last: what follows it is not stored
  const TW* P = a.P + (int64_t)l * r * a.n;
  // this CTA's 64-column blocks [k0, k0 + steps)
  const int k0 = min(blocks, rank * per), steps = min(blocks, k0 + per) - k0;
  int kept = 0;                    // rounds whose sum is kept
  // the stages' warps, each once its blocks before `block` are there: keep the
  // sums of the rounds before it
  auto keep = [&](int block) {
    for (; (kept + 1) * acc.round <= block; ++kept) {
      ok = ok && mbar_wait(&round_done, (uint32_t)(kept & 1));
      tc_fence_after();
      if (32 * (warp % 4) < cnt)
        keep_round(tmem + ((uint32_t)(32 * (warp % 4)) << 16), 16 * (warp / 4), 16 * SW, r16, acc.mains + acc.low - (kept > 0 ? 0 : 1),
                   (acc.mains + acc.low) * r16);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&round_kept);
    }
  };
  if (warp < 4 * SW) {
    const int s = warp / SW;
    if (s < stages) {
      const int ch = lane % 8, row0 = lane / 8 + 4 * (warp % SW);   // the lane's 16-byte column and first row
      uint8_t* xs = sm + s * stage;
      uint8_t* ps = xs + PX * XT_BYTES;
      auto spot = [&](int row) { return row * 128 + ((ch ^ (row & 7)) << 4); };
      // the lane's rows of x are those of every block
      constexpr int ROWS = TILE / (4 * SW), BATCH = KEEP && SPLIT ? 2 : 4;
      int mine[ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) mine[k] = tok[row0 + 4 * SW * k];
      for (int i = s; i < steps; i += stages) {
        if (i >= stages) ok = ok && mbar_wait(&empty[s], (uint32_t)((i / stages - 1) & 1));
        const int c = 64 * (k0 + i) + 8 * ch, left = a.n - c;
        if constexpr (CP) {
          const __nv_bfloat16* x = a.x + (c < a.n ? c : 0);
#pragma unroll
          for (int k = 0; k < ROWS; ++k)       // rows past the tile's tokens only feed their own sums
            if (mine[k] >= 0) cp16(xs + spot(row0 + 4 * SW * k), x + (int64_t)mine[k] * a.ldx, c < a.n);
#pragma unroll 4
          for (int row = row0; row < r16; row += 4 * SW) {
            const bool there = row < r && c < a.n;
            cp16(ps + spot(row), P + (there ? (int64_t)row * a.n + c : 0), there);
          }
          cp_wait_all();
        } else {
          // batches of loads, then their stores: a load does not pass a store by itself
          Eight<TW> w[BATCH];
          auto load_p = [&](int row) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int j = row + 4 * SW * k;
              w[k].zero();
              if (j < r && left > 0) w[k].load(P + (int64_t)j * a.n + c, a.vec_p, left);
            }
          };
          load_p(row0);
#pragma unroll
          for (int k0 = 0; k0 < ROWS; k0 += BATCH) {
            Eight<TX> v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              v[k].zero();
              if (mine[k0 + k] >= 0 && left > 0) v[k].load(a.x + (int64_t)mine[k0 + k] * a.ldx + c, a.vec_x, left);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
              if (mine[k0 + k] >= 0) v[k].store(xs + spot(row0 + 4 * SW * (k0 + k)), XT_BYTES);
          }
          for (int row = row0; row < r16; row += 4 * SW * BATCH) {
            if (row > row0) load_p(row);
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int j = row + 4 * SW * k;
              if (j < r16) w[k].store(ps + spot(j), r16 * 128);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if constexpr (KEEP) keep(i);
      }
    }
    if constexpr (KEEP) keep(steps - 1);
  } else if (lane == 0) {
    // descriptors' addresses count 16 bytes: stages and steps are added to them
    const uint32_t idesc = make_idesc_bf16(TILE, r16, 0, 0);
    const uint64_t x0 = make_sw128_desc(smem_u32(sm), 16, 1024), p0 = x0 + (uint64_t)(PX * XT_BYTES >> 4);
    const int pp = r16 * 128 >> 4;
    const uint32_t low = tmem + (uint32_t)(acc.mains * r16);
    uint32_t large = tmem;                     // the block's accumulator
    bool begun = false;                        // it holds blocks of this round
    int s = 0, b = 0;                          // stage; the block's number in its round
    uint32_t phase = 0;
    for (int i = 0; i < steps && ok; ++i, ++b) {
      if (KEEP && b == acc.round) {
        b = 0, large = tmem, begun = false;
        tc_commit(&round_done);
        ok = mbar_wait(&round_kept, (uint32_t)((i / acc.round - 1) & 1));
      }
      ok = ok && mbar_wait(&full[s], phase);
      if (!ok) break;
      tc_fence_after();
      const uint64_t xd = x0 + (uint64_t)(s * stage >> 4), pd = p0 + (uint64_t)(s * stage >> 4);
#pragma unroll
      for (int px = 0; px < PX; ++px)
#pragma unroll
        for (int pw = 0; pw < PW && px + pw <= 2; ++pw)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const bool main = px + pw == 0, first = (PW > 1 ? px == 0 && pw == 1 : px == 1) && kk == 0;   // of the small terms
            tc_mma_f16(main ? large : low, xd + (uint64_t)((px * XT_BYTES >> 4) + kk * 2),
                       pd + (uint64_t)(pw * pp + kk * 2), idesc, main ? (begun || kk > 0) : (b > 0 || !first));
          }
      tc_commit(&empty[s]);
      if (++s == stages) s = 0, phase ^= 1u;
      large += (uint32_t)r16;
      if (large == low) large = tmem, begun = true;
    }
    if (steps > 0 && ok) tc_commit(&all_done);
  }
  __syncwarp();
  if (steps > 0) ok = ok && mbar_wait(&all_done, 0u);
  __syncthreads();
  tc_fence_after();
  // ---- the partial sums of the cluster's CTAs
  const int pitch = r16 + 4;
  float* hpart = reinterpret_cast<float*>(sm);
  if (warp < 4 && 32 * warp < cnt) {
    const int t = 32 * warp + lane;
    for (int j = 0; j < r16; j += 16) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
      // from the rounds before and the small terms on; of the others those that were used
      const int used = steps - kept * acc.round;
      for (int q = acc.mains + acc.low - (KEEP && kept > 0 ? 0 : 1); q >= 0; --q) {
        if (q >= acc.mains ? steps > 0 : q < used) {
          float w[16];
          tmem_ld16(tmem + ((uint32_t)(32 * warp) << 16) + q * r16 + j, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] += w[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(hpart + t * pitch + j + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
  }
  tc_fence_before();
  if (nc > 1) cluster.sync();
  else __syncthreads();
  {
    const int share = (cnt + nc - 1) / nc, t0 = min(cnt, rank * share), t1 = min(cnt, t0 + share), quads = r16 / 4;
    const float scale = a.h_scaled && a.scale ? a.scale[l] : 1.f;
    for (int i = tid; i < (t1 - t0) * quads; i += ST) {
      const int t = t0 + i / quads, j = 4 * (i % quads);
      float4 w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < nc) w[c] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(hpart, c) + t * pitch + j);
      float4 v = w[0];
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < nc) v.x += w[c].x, v.y += w[c].y, v.z += w[c].z, v.w += w[c].w;
      const float e[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
      if (ok) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < r) a.h[(int64_t)tok[t] * r + j + q] = e[q];
      }
    }
  }
  if (nc > 1) cluster.sync();                  // the others' shared memory is read until here
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, shrink_cols<SPLIT>());
  }
}

// 16 bytes of a row, or what of them is left of it
template <typename TY>
__device__ __forceinline__ uint4 load_vec(const TY* p, bool vec, int left) {
  constexpr int EV = 16 / sizeof(TY);
  if (vec && left >= EV) return *reinterpret_cast<const uint4*>(p);
  alignas(16) TY e[EV];
#pragma unroll
  for (int k = 0; k < EV; ++k) e[k] = k < left ? p[k] : TY(0.f);
  return *reinterpret_cast<const uint4*>(e);
}
template <typename TY>
__device__ __forceinline__ void store_vec(TY* p, const uint4& u, bool vec, int left) {
  constexpr int EV = 16 / sizeof(TY);
  if (vec && left >= EV) {
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    const TY* e = reinterpret_cast<const TY*>(&u);
#pragma unroll
    for (int k = 0; k < EV; ++k)
      if (k < left) p[k] = e[k];
  }
}
// base + v, rounded once
__device__ __forceinline__ uint4 add_vec(const uint4& b, const float* v, float) {
  return make_uint4(__float_as_uint(__uint_as_float(b.x) + v[0]), __float_as_uint(__uint_as_float(b.y) + v[1]),
                    __float_as_uint(__uint_as_float(b.z) + v[2]), __float_as_uint(__uint_as_float(b.w) + v[3]));
}
__device__ __forceinline__ uint4 add_vec(const uint4& b, const float* v, __nv_bfloat16) {
  const uint32_t u[4] = {b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 s = __floats2bfloat162_rn(__uint_as_float(u[i] << 16) + v[2 * i],
                                                   __uint_as_float(u[i] & 0xFFFF0000u) + v[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// a.h as the shrink step left it, times the scale already where a.h_scaled.
template <typename TW, typename TY, bool CP>
__global__ void __launch_bounds__(ET, 1)
    k_adapter_expand(const __grid_constant__ ApplyArgs<float, TW, TY> a, ExpandRings rings, void* plan) {
  constexpr int PW = pieces<TW>(), NP = h_pieces<TY>(), CB = expand_cols<TY>(), EV = 16 / (int)sizeof(TY);
  constexpr int CH = CB / 8, TCOLS = ACCS * CB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int tok[TILE];
  __shared__ uint64_t full[ACCS], read[ACCS], there[QW];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = a.r;
  // The launch before released this one after its own wait: all but h is there.
  const PlanView pv = plan_view(plan, a.T, a.count);
  const bool mine = plan_ok(pv, a.T, a.count);
  const int blocks = (a.m + CB - 1) / CB;
  const int64_t work = mine ? (int64_t)pv.head[H_TILES] * blocks : 0;
  const int64_t w0 = work * blockIdx.x / gridDim.x, w1 = work * (blockIdx.x + 1) / gridDim.x;
  const int r16 = (r + 15) / 16 * 16, kb = (r16 + 63) / 64, qtile = expand_tile<TW, TY>(r16);
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = sm + NP * kb * XT_BYTES;
  if (tid == 0) {
    for (int i = 0; i < ACCS; ++i) mbar_init(&full[i], 1), mbar_init(&read[i], 4);
    for (int i = 0; i < QW; ++i) mbar_init(&there[i], 1);
    fence_mbar_init();
  }
  uint32_t tmem = 0;
  bool ok = true, started = false;             // the wait for h, and TMEM
  int done = 0;                                // blocks multiplied so far: accumulator and phase of the next
  int ring = 0;                                // the multiplying warp's next tile of Q, and its phase
  uint32_t ring_phase = 0;
  const uint32_t idesc = make_idesc_bf16(TILE, CB, 0, 1);
  for (int64_t w = w0; w < w1;) {
    const int2 tile = pv.tiles[w / blocks];
    const int l = tile.x, cnt = min(TILE, pv.start[l + 1] - tile.y);
    const int b0 = (int)(w % blocks), steps = (int)min((int64_t)(blocks - b0), w1 - w);
    w += steps;
    __syncthreads();                           // the tile before is done with tok and h's pieces
    if (tid < TILE) tok[tid] = tid < cnt ? pv.order[tile.y + tid] : -1;
    __syncthreads();
    // Group warp / 4, 32 tokens.  To and from memory a lane moves 16 bytes, 16
    // lanes to a row, of rows 2 v + lane / 16.
    const int token0 = 32 * (warp % 4), group = warp / 4, col = lane % 16 * EV;
    const bool busy = group < rings.rows && token0 < cnt;
    uint8_t* rows = qs + rings.q * qtile + warp * 8192;    // 32 rows of 256 bytes
    auto piece = [&](int tr, int p) { return tr * 256 + ((p ^ (tr & 7)) << 4); };
    // Whole blocks of 32 tokens that are all there go by offsets kept in
    // registers, others by tok's, four rounds at once.
    const bool fast = a.fast_y && busy && token0 + 32 <= cnt && l != a.count;
    uint32_t offset[16];
#pragma unroll
    for (int v = 0; v < 16; ++v)
      offset[v] = fast ? (uint32_t)(tok[token0 + 2 * v + lane / 16] * (a.ldy / EV)) + lane % 16 : 0u;
    const int rounds = busy ? (min(32, cnt - token0) + 1) / 2 : 0;
    auto fill_rows = [&](int i) {
      if (i >= steps || !a.base || !busy) return;
      if (fast && (b0 + i + 1) * CB <= a.m) {
        const uint4* from = reinterpret_cast<const uint4*>(a.base) + (b0 + i) * (CB / EV);
        const uint32_t to = smem_u32(rows) + lane / 16 * 256;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           to + v * 512 + (((lane % 16) ^ ((2 * v + lane / 16) & 7)) << 4)),
                       "l"(from + offset[v])
                       : "memory");
      } else if (sizeof(TY) == 4 && !a.vec_y) {
        // fp32 at any alignment: a lane's columns are lane and lane + 32
        const int c = (b0 + i) * CB + lane;
        const uint32_t to = smem_u32(rows) + lane % 4 * 4;
#pragma unroll 8
        for (int tr = 0; tr < 32; ++tr) {
          const int t = tok[token0 + tr];
          if (t < 0) break;                    // the tile's tokens come first
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (c + 32 * h < a.m)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + piece(tr, 8 * h + lane / 4)),
                           "l"(a.base + t * a.ldb + c + 32 * h)
                           : "memory");
        }
      } else {
        const int c = (b0 + i) * CB + col, left = a.m - c;
        if (a.vec_y && (b0 + i + 1) * CB <= a.m) {
          for (int v0 = 0; v0 < rounds; v0 += 4) {
            int t[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) t[v] = tok[token0 + 2 * (v0 + v) + lane / 16];
#pragma unroll
            for (int v = 0; v < 4; ++v)        // zeros where there is no token
              cp16(rows + piece(2 * (v0 + v) + lane / 16, lane % 16), a.base + max(t[v], 0) * a.ldb + c, t[v] >= 0);
          }
          return;
        }
        for (int v0 = 0; v0 < 16; v0 += 4) {   // four loads, then their stores
          uint4 u[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t t = tok[token0 + 2 * (v0 + v) + lane / 16];
            u[v] = make_uint4(0u, 0u, 0u, 0u);
            if (t >= 0) u[v] = load_vec(a.base + t * a.ldb + c, a.vec_y, left);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint4*>(rows + piece(2 * (v0 + v) + lane / 16, lane % 16)) = u[v];
        }
      }
    };
    const TW* Q = a.Q + (int64_t)l * r * a.m;
    // warp EW + q fills the q-th tile of the ring, for blocks n = q modulo the ring
    auto fill_q = [&](int i) {
      const int ch = lane % CH, c = (b0 + i) * CB + 8 * ch;
      uint8_t* to = qs + (warp - EW) * qtile;
      // MN-major boxes of 64 columns, 128 bytes to a row
      auto spot = [&](int j) { return (ch / 8) * (r16 * 128) + j * 128 + (((ch % 8) ^ (j & 7)) << 4); };
      if constexpr (CP) {
        const TW* from = Q + (c < a.m ? c : 0);
#pragma unroll 8
        for (int j = lane / CH; j < r16; j += 32 / CH) {
          const bool in = j < r && c < a.m;
          cp16(to + spot(j), from + (in ? (int64_t)j * a.m : 0), in);
        }
        cp_wait_all();
      } else {
        constexpr int BATCH = 4;
        for (int j0 = lane / CH; j0 < r16; j0 += 32 / CH * BATCH) {
          Eight<TW> v[BATCH];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int j = j0 + 32 / CH * k;
            v[k].zero();
            if (j < r && c < a.m) v[k].load(Q + (int64_t)j * a.m + c, a.vec_q, a.m - c);
          }
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int j = j0 + 32 / CH * k;
            if (j < r16) v[k].store(to + spot(j), r16 * 2 * CB);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&there[warp - EW]);
    };
    // the first block of this run whose tile this warp fills
    const int q0 = warp >= EW && warp < EW + rings.q ? ((warp - EW - done) % rings.q + rings.q) % rings.q : steps;
    if (l != a.count) {
      if (warp < EW) fill_rows(group);
      else if (q0 < steps) fill_q(q0);
    }
    if (!started) {                            // TMEM only now: the launch before may still need it
      started = true;
      pdl_wait_then_release();
      if (warp == 0) tmem_alloc(&tmem_base, TCOLS);
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      tmem = tmem_base;
    }
    if (l == a.count) {                        // no adapter: y = base
      if (a.y != a.base && group < EW / 4 && token0 < cnt)
        for (int i = group; i < steps; i += EW / 4) {
          const int c = (b0 + i) * CB + col, left = a.m - c;
#pragma unroll
          for (int h = 0; h < 2; ++h) {        // eight loads in flight
            uint4 u[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const int64_t t = tok[token0 + 16 * h + 2 * v + lane / 16];
              u[v] = t >= 0 && a.base ? load_vec(a.base + t * a.ldb + c, a.vec_y, left) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const int64_t t = tok[token0 + 16 * h + 2 * v + lane / 16];
              if (t >= 0) store_vec(a.y + t * a.ldy + c, u[v], a.vec_y, left);
            }
          }
        }
      continue;
    }
    // ---- the pieces of scale h, K-major, 64 ranks to a block
    if (warp < EW) {
      const float scale = a.scale && !a.h_scaled ? a.scale[l] : 1.f;
      const int eights = r16 / 8;
      const bool vec_h = r % 4 == 0 && (reinterpret_cast<uintptr_t>(a.h) & 15) == 0;
      for (int i = tid; i < cnt * eights; i += 32 * EW) {
        const int t = i / eights, c = i % eights;
        const float* h = a.h + (int64_t)tok[t] * r + 8 * c;
        float f[8];
        if (vec_h) {
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 u = 8 * c < r ? *reinterpret_cast<const float4*>(h) : z;
          const float4 v = 8 * c + 4 < r ? *reinterpret_cast<const float4*>(h + 4) : z;
          f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 8 * c + e < r ? h[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= scale;
        store_pieces<NP>(sm + (c / 8) * XT_BYTES + t * 128 + (((c % 8) ^ (t & 7)) << 4), kb * XT_BYTES, f);
      }
      fence_proxy_async_smem();
    }
    __syncthreads();
    if (warp == EW + QW) {
      if (lane == 0) {
        // descriptors' addresses (low 14 bits) count 16 bytes: pieces and steps
        // are added to them
        const uint64_t ha = make_sw128_desc(smem_u32(sm), 16, 1024);
        const int ks = r16 / 16;
        for (int i = 0; i < steps && ok; ++i) {
          const int n = done + i, b = n % ACCS;
          ok = mbar_wait(&there[ring], ring_phase);
          if (n >= ACCS) ok = ok && mbar_wait(&read[b], (uint32_t)((n / ACCS - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qa = make_sw128_desc(smem_u32(qs + ring * qtile), r16 * 128, 1024);
          const uint32_t d = tmem + (uint32_t)(b * CB);
          // one product in the code: unrolled, 512 tokens over 32 adapters took
          // 63 us (59 now), 4096 of rank 64 the same
          bool more = false;
#pragma unroll 1
          for (int ph = NP - 1; ph >= 0; --ph)           // the small terms first
#pragma unroll 1
            for (int pw = min(PW - 1, 2 - ph); pw >= 0; --pw) {
              uint64_t hd = ha + (uint64_t)(ph * kb * XT_BYTES >> 4);
              uint64_t qd = qa + (uint64_t)(pw * r16 * 2 * CB >> 4);
#pragma unroll 1
              for (int k = 0; k < ks; ++k, qd += 2048 >> 4) {
                tc_mma_f16(d, hd, qd, idesc, more);
                hd += k % 4 == 3 ? (XT_BYTES - 96) >> 4 : 32 >> 4;
                more = true;
              }
            }
          if (++ring == rings.q) ring = 0, ring_phase ^= 1u;
          tc_commit(&full[b]);
        }
      }
      __syncwarp();
    } else if (warp >= EW) {
      for (int i = q0 + rings.q; i < steps; i += rings.q) {
        const int back = done + i - rings.q;   // the block that read this tile
        ok = ok && mbar_wait(&full[back % ACCS], (uint32_t)((back / ACCS) & 1));
        fill_q(i);
      }
    } else {
      for (int i = group; group < rings.rows && i < steps; i += rings.rows) {
        const int n = done + i, b = n % ACCS;
        cp_wait_all();
        __syncwarp();
        ok = ok && mbar_wait(&full[b], (uint32_t)((n / ACCS) & 1));
        tc_fence_after();
        if (busy) {
          const uint32_t at = tmem + ((uint32_t)token0 << 16) + (uint32_t)(b * CB);
#pragma unroll
          for (int g = 0; g < CB / 32; ++g) {
            float d[32];
            tmem_ld32(at + 32 * g, d);
#pragma unroll
            for (int p = 0; p < 32 / EV; ++p) {
              uint4* e = reinterpret_cast<uint4*>(rows + lane * 256 + (((g * (32 / EV) + p) ^ (lane & 7)) << 4));
              *e = add_vec(a.base ? *e : make_uint4(0u, 0u, 0u, 0u), d + p * EV, TY());
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&read[b]);
        if (fast && ok && (b0 + i + 1) * CB <= a.m) {
          uint4* to = reinterpret_cast<uint4*>(a.y) + (b0 + i) * (CB / EV);
#pragma unroll
          for (int v = 0; v < 16; ++v)
            to[offset[v]] = *reinterpret_cast<const uint4*>(rows + piece(2 * v + lane / 16, lane % 16));
        } else if (a.vec_y && busy && ok && (b0 + i + 1) * CB <= a.m) {
          const int c = (b0 + i) * CB + col;
          for (int v0 = 0; v0 < rounds; v0 += 4) {
            int t[4];
            uint4 u[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              t[v] = tok[token0 + 2 * (v0 + v) + lane / 16];
              u[v] = *reinterpret_cast<const uint4*>(rows + piece(2 * (v0 + v) + lane / 16, lane % 16));
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (t[v] >= 0) *reinterpret_cast<uint4*>(a.y + t[v] * a.ldy + c) = u[v];
          }
        } else if (sizeof(TY) == 4 && !a.vec_y && busy && ok) {
          const int c = (b0 + i) * CB + lane;
#pragma unroll 8
          for (int tr = 0; tr < 32; ++tr) {
            const int t = tok[token0 + tr];
            const float f0 = *reinterpret_cast<const float*>(rows + piece(tr, lane / 4) + lane % 4 * 4);
            const float f1 = *reinterpret_cast<const float*>(rows + piece(tr, 8 + lane / 4) + lane % 4 * 4);
            TY* y = a.y + t * a.ldy + c;
            if (t >= 0 && c < a.m) put(y, f0);
            if (t >= 0 && c + 32 < a.m) put(y + 32, f1);
          }
        } else if (busy && ok) {
          const int c = (b0 + i) * CB + col, left = a.m - c;
#pragma unroll 4
          for (int v = 0; v < 16; ++v) {
            const int tr = 2 * v + lane / 16, t = tok[token0 + tr];
            if (t >= 0)
              store_vec(a.y + (int64_t)t * a.ldy + c,
                        *reinterpret_cast<const uint4*>(rows + piece(tr, lane % 16)), a.vec_y, left);
          }
        }
        __syncwarp();                          // the group's next rows go there
        fill_rows(i + rings.rows);
      }
    }
    cp_wait_all();
    done += steps;
  }
  if (!started) {
    pdl_wait_then_release();
    return;
  }
  // every multiplication is over: its accumulator was waited for
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TCOLS);
  }
}

// ---------------------------------------------------------------- sums over an adapter's tokens
// out[l][j][c] (+)= k_l sum_{t of l} u[t][j] x[t][c], u: T x r fp32, k_l = 1 or
// scale[l], for the ranks above 128.  One CTA per (chunk, 512 columns, 16 rows j): fp32 sums over the
// chunk's tokens in their order; an adapter's only chunk goes straight to
// out, the others to their slot of `partial`, which k_adapter_join adds up.
template <typename TX>
struct OuterArgs {
  const TX* x;
  int64_t ldx;
  const float* u;
  const float* scale;
  float* out;                  // count x r x width
  float* partial;              // slots x r x width
  int T, width, r, count, accumulate;
  bool vec_x;
};
constexpr int OT = 128, OROWS = 16;            // threads; rows of u per CTA
template <typename TX>
__global__ void __launch_bounds__(OT) k_adapter_outer(const __grid_constant__ OuterArgs<TX> a, void* plan) {
  __shared__ float us[64][OROWS];
  __shared__ int tok[64];
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, a.T, a.count);
  if (!plan_ok(pv, a.T, a.count) || (int)blockIdx.z >= pv.head[H_CHUNKS]) return;
  const int4 chunk = pv.chunks[blockIdx.z];
  const int l = chunk.x, first = chunk.y, cnt = max(0, min(CHUNK, pv.start[l + 1] - first));
  const int c = (blockIdx.x * OT + threadIdx.x) * 4, j0 = blockIdx.y * OROWS, left = a.width - c;
  float acc[OROWS][4];
#pragma unroll
  for (int j = 0; j < OROWS; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  for (int t0 = 0; t0 < cnt; t0 += 64) {
    const int nt = min(64, cnt - t0);
    __syncthreads();
    if (threadIdx.x < nt) tok[threadIdx.x] = pv.order[first + t0 + threadIdx.x];
    __syncthreads();
    for (int i = threadIdx.x; i < nt * OROWS; i += OT) {
      const int t = i / OROWS, j = i % OROWS;
      us[t][j] = j0 + j < a.r ? a.u[(int64_t)tok[t] * a.r + j0 + j] : 0.f;
    }
    __syncthreads();
    if (left > 0) {
#pragma unroll 4
      for (int t = 0; t < nt; ++t) {
        const float4 v = load4(a.x + (int64_t)tok[t] * a.ldx + c, a.vec_x, left);
#pragma unroll
        for (int j = 0; j < OROWS; ++j) {
          const float u = us[t][j];
          acc[j][0] = fmaf(u, v.x, acc[j][0]);
          acc[j][1] = fmaf(u, v.y, acc[j][1]);
          acc[j][2] = fmaf(u, v.z, acc[j][2]);
          acc[j][3] = fmaf(u, v.w, acc[j][3]);
        }
      }
    }
  }
  if (left <= 0) return;
  const float k = a.scale && cnt > 0 ? a.scale[l] : 1.f;      // an adapter without tokens: 0, whatever its scale
  float* out = chunk.z < 0 ? a.out + (int64_t)l * a.r * a.width : a.partial + (int64_t)chunk.z * a.r * a.width;
  const bool add = chunk.z < 0 && a.accumulate;
  for (int j = 0; j < OROWS && j0 + j < a.r; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        float* o = out + (int64_t)(j0 + j) * a.width + c + i;
        *o = (add ? *o : 0.f) + k * acc[j][i];
      }
}

// The same on the tensor cores: D[column][j] = x^T u (M = 128 columns, N = r,
// K = tokens, x MN-major as its rows lie in memory), SUB tokens at a time, two
// times 128 columns (one with fp32 rows) that share u's tile.  u is cut into
// three bf16 pieces that lie one after the other, so one product takes several
// as more columns of D: its time is that of reading x from shared memory, 60
// cycles whatever N.  (OuterBlocks: which pieces go together.)  The pieces are
// made once, K-major and swizzled as the tensor core reads them
// (k_adapter_pieces), so that a stage takes them by one bulk copy.
// 8192 tokens, 4096 and 11008 columns, rank 32: 80 us for both sums, 3.1 TB/s
// (38 us at the copy rate); 100 us with a product per piece, 150 us with u cut
// into pieces by every CTA, 3700 us on the CUDA cores with all else.
__host__ __device__ inline int64_t max_subs(int64_t T, int64_t count) { return T / SUB + (count < T ? count : T) + 1; }
__host__ __device__ inline int u_bytes(int r16) { return 3 * r16 * 128; }    // of SUB tokens

// One CTA per SUB tokens of an adapter and matrix u (blockIdx.y).
struct PiecesArgs {
  const float* u[2];
  uint8_t* out[2];
  int T, r, count;
};
__global__ void __launch_bounds__(128) k_adapter_pieces(const __grid_constant__ PiecesArgs a, void* plan) {
  __shared__ int tok[SUB];
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, a.T, a.count);
  const int k = blockIdx.x / (CHUNK / SUB), sub = blockIdx.x % (CHUNK / SUB);
  if (!plan_ok(pv, a.T, a.count) || k >= pv.head[H_CHUNKS]) return;
  const int4 chunk = pv.chunks[k];
  const int first = chunk.y + sub * SUB, cnt = min(SUB, pv.start[chunk.x + 1] - first), r16 = (a.r + 15) / 16 * 16;
  if (cnt <= 0) return;
  if (threadIdx.x < SUB) tok[threadIdx.x] = threadIdx.x < cnt ? pv.order[first + threadIdx.x] : -1;
  __syncthreads();
  const float* u = a.u[blockIdx.y];
  uint8_t* out = a.out[blockIdx.y] + (int64_t)(chunk.w + sub) * u_bytes(r16);
  for (int e = threadIdx.x; e < r16 * (SUB / 8); e += 128) {
    const int j = e % r16, o = e / r16;
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int t = tok[8 * o + q];
      f[q] = t >= 0 && j < a.r ? u[(int64_t)t * a.r + j] : 0.f;
    }
    store_pieces<3>(out + j * 128 + ((o ^ (j & 7)) << 4), r16 * 128, f);
  }
}

// Halves of 128 columns per CTA.
template <typename TX> __host__ __device__ constexpr int outer_halves() { return sizeof(TX) == 2 ? 2 : 1; }
template <typename TX>
__host__ __device__ inline int outer_stage(int r16) {
  return SUB * 256 * pieces<TX>() * outer_halves<TX>() + u_bytes(r16);
}
__host__ __device__ inline int outer_stages(int stage) {
  const int s = 216 * 1024 / stage;
  return s > 4 ? 4 : s;
}
// Accumulators of a half, in blocks of r16 columns whose sum is the result:
// MAINS sets of `width` blocks that take x's first piece times u's first
// `width` pieces, a step in turn (few steps meet in each), then `low` blocks
// for the other terms.  Up to rank 32 all of u in one product; up to 64 u's
// second and third piece in one; beyond, each by itself.
struct OuterBlocks {
  int width, low, total;
};
constexpr int MAINS = 2;
__host__ __device__ inline OuterBlocks outer_blocks(int r16, int px) {
  OuterBlocks b;
  b.width = r16 <= 32 ? 3 : 1;
  b.low = r16 <= 32 ? (px > 1 ? 2 : 0) : r16 <= 64 ? 2 : 1;
  const int mains = r16 <= 64 ? MAINS : 1;
  b.total = mains * b.width + b.low;
  return b;
}
template <typename TX>
struct OuterPair {             // column blocks [0, split) are the first's, the rest the second's
  OuterArgs<TX> a[2];
  const uint8_t* u[2];
  int split;
};
// Resident CTAs take the (chunk, column block) pairs in turn, so that all get
// long and short chunks alike.  Warps: the stages', one to
// multiply, others that write a pair's sums while the next is multiplied into
// the other half of TMEM (where two sets of accumulators fit); each goes
// through the pairs by itself.
template <typename TX, bool CP>
__host__ __device__ constexpr int outer_threads() { return stage_threads<CP>() + 128 * outer_halves<TX>(); }
template <typename TX, bool CP>
__global__ void __launch_bounds__(outer_threads<TX, CP>(), 1)
    k_adapter_outer_tc(const __grid_constant__ OuterPair<TX> both, int blocks, void* plan) {
  constexpr int PX = pieces<TX>(), XB = SUB * 256;       // bytes of one piece of SUB tokens x 128 columns
  constexpr int SW = stage_warps<CP>(), MW = 4 * SW, H = outer_halves<TX>();
  constexpr int CHS = 16 * H, ROWS = SUB / SW, AT_ONCE = 32 / CHS, TCOLS = 512;   // 16-byte columns; a warp's rows
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[4], empty[4], ready[2], drained[2];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  const int T = both.a[0].T, count = both.a[0].count, r = both.a[0].r;
  const PlanView pv = plan_view(plan, T, count);
  if (!plan_ok(pv, T, count)) return;
  const int chunks = pv.head[H_CHUNKS];
  const int64_t work = (int64_t)chunks * blocks;
  if (blockIdx.x >= work) return;
  const int r16 = (r + 15) / 16 * 16;
  const OuterBlocks blk = outer_blocks(r16, PX);
  const int mains = (blk.total - blk.low) / blk.width, sets = 2 * H * blk.total * r16 <= TCOLS ? 2 : 1;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage = outer_stage<TX>(r16), stages = outer_stages(stage);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&full[i], 1 + SW), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ready[i], 1), mbar_init(&drained[i], 4 * H);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&tmem_base, TCOLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;
  // pair w's chunk and its number of tokens, looked up one pair ahead
  auto look = [&](int64_t w, int4& chunk, int& cnt) {
    if (w < work) {
      chunk = pv.chunks[w / blocks];
      cnt = max(0, min(CHUNK, pv.start[chunk.x + 1] - chunk.y));
    }
  };
  int4 chunk, next;
  int cnt, next_cnt;
  look(blockIdx.x, chunk, cnt);
  int fills = 0, items = 0;                    // stages filled and pairs with tokens before this one
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x, chunk = next, cnt = next_cnt) {
    look(w + gridDim.x, next, next_cnt);
    const int l = chunk.x, steps = (cnt + SUB - 1) / SUB, block = (int)(w % blocks), which = block >= both.split;
    const OuterArgs<TX>& a = both.a[which];
    const int c0 = (block - (which ? both.split : 0)) * 128 * H;
    if (warp < MW) {
      const int s = warp / SW;
      if (s < stages) {
        // stage s takes fills f = s modulo the stages
        const int ch = lane % CHS, row0 = ROWS * (warp % SW), c = c0 + 8 * ch, left = a.width - c;
        uint8_t* xs = sm + s * stage;
        auto spot = [&](int row) { return (ch / 8) * 8192 + row * 128 + (((ch % 8) ^ (row & 7)) << 4); };
        for (int i = ((s - fills) % stages + stages) % stages; i < steps; i += stages) {
          const int f = fills + i, rows = min(ROWS, cnt - SUB * i - row0);       // of this warp's that are there
          const int mine = lane < rows ? pv.order[chunk.y + SUB * i + row0 + lane] : -1;
          if (f >= stages) ok = ok && mbar_wait(&empty[s], (uint32_t)((f / stages - 1) & 1));
          __syncwarp();
          if (warp % SW == 0 && lane == 0) {
            mbar_arrive_expect_tx(&full[s], (uint32_t)u_bytes(r16));
            bulk_load_1d(xs + PX * H * XB, both.u[which] + (int64_t)(chunk.w + i) * u_bytes(r16), (uint32_t)u_bytes(r16),
                         &full[s]);
          }
          // rows past the adapter's tokens are 0: they would meet u's zeros as anything
          if constexpr (CP) {
            const int bytes = min(16, 2 * left);         // the row may end inside the 16
#pragma unroll 8
            for (int k = 0; k < ROWS; k += AT_ONCE) {
              const int row = k + lane / CHS, t = __shfl_sync(0xffffffffu, mine, row);
              const bool there = t >= 0 && left > 0;
              cp16(xs + spot(row0 + row), a.x + (there ? (int64_t)t * a.ldx + c : 0), there ? bytes : 0);
            }
            cp_wait_all();
          } else {
            constexpr int BATCH = ROWS / AT_ONCE < 4 ? ROWS / AT_ONCE : 4;
#pragma unroll
            for (int k0 = 0; k0 < ROWS; k0 += AT_ONCE * BATCH) {
              Eight<TX> v[BATCH];
#pragma unroll
              for (int k = 0; k < BATCH; ++k) {
                const int t = __shfl_sync(0xffffffffu, mine, k0 + AT_ONCE * k + lane / CHS);
                v[k].zero();
                if (t >= 0 && left > 0) v[k].load(a.x + (int64_t)t * a.ldx + c, a.vec_x, left);
              }
#pragma unroll
              for (int k = 0; k < BATCH; ++k) v[k].store(xs + spot(row0 + k0 + AT_ONCE * k + lane / CHS), H * XB);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
      }
    } else if (warp == MW) {
      if (lane == 0) {
        // descriptors' addresses count 16 bytes: stages and steps are added to them
        const uint64_t x0 = make_sw128_desc(smem_u32(sm), 8192, 1024);
        const uint64_t u0 = make_sw128_desc(smem_u32(sm) + PX * H * XB, 16, 1024);
        const int up = r16 * 128 >> 4;
        for (int i = 0; i < steps && ok; ++i) {
          const int f = fills + i, s = f % stages, n = items;
          if (i == 0 && n >= sets) ok = mbar_wait(&drained[n % sets], (uint32_t)((n / sets - 1) & 1));
          ok = ok && mbar_wait(&full[s], (uint32_t)((f / stages) & 1));
          if (!ok) break;
          tc_fence_after();
          uint64_t xd = x0 + (uint64_t)(s * stage >> 4);
          const uint64_t ud = u0 + (uint64_t)(s * stage >> 4);
          const uint32_t set = tmem + (uint32_t)(n % sets * (TCOLS / 2));
          // x's piece px times `n` pieces of u from pu on, into D's blocks from `to` on
          auto product = [&](int px, int pu, int n, uint32_t to, bool add) {
            const uint32_t idesc = make_idesc_bf16(128, n * r16, 1, 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16(to, xd + (uint64_t)((px * H * XB + kk * 2048) >> 4), ud + (uint64_t)(pu * up + kk * 2), idesc,
                         add || kk > 0);
          };
#pragma unroll
          for (int hh = 0; hh < H; ++hh, xd += XB >> 4) {
            const uint32_t half = set + (uint32_t)(hh * blk.total * r16), low = half + (uint32_t)(mains * blk.width * r16);
            product(0, 0, blk.width, half + (uint32_t)(i % mains * blk.width * r16), i >= mains);
            bool add = i > 0;
            if (blk.width == 1) {
              if (blk.low == 2) {
                product(0, 1, 2, low, add);
              } else {
                product(0, 1, 1, low, add);
                product(0, 2, 1, low, true);
              }
              add = true;
            }
            if constexpr (PX > 1) {
              if (blk.low == 2) {
                product(1, 0, 2, low, add);
              } else {
                product(1, 0, 1, low, add);
                product(1, 1, 1, low, true);
              }
              product(2, 0, 1, low, true);
            }
          }
          tc_commit(&empty[s]);
          if (i == steps - 1) tc_commit(&ready[n % sets]);
        }
      }
      __syncwarp();
    } else {
      // TMEM lanes 32 (warp % 4) ..: columns of the warp's half of the block
      const int half = (warp - MW - 1) / 4, n = items, c = c0 + 128 * half + 32 * (warp % 4) + lane;
      if (steps > 0) ok = ok && mbar_wait(&ready[n % sets], (uint32_t)((n / sets) & 1));
      tc_fence_after();
      const float k = a.scale && steps > 0 ? a.scale[l] : 1.f;      // an adapter without tokens: 0, whatever its scale
      float* out = chunk.z < 0 ? a.out + (int64_t)l * r * a.width : a.partial + (int64_t)chunk.z * r * a.width;
      const bool add = chunk.z < 0 && a.accumulate;
      const uint32_t at = tmem + ((uint32_t)(32 * (warp % 4)) << 16) + (uint32_t)(n % sets * (TCOLS / 2) + half * blk.total * r16);
      for (int j = 0; j < r16; j += 16) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        for (int q = blk.total - 1; q >= 0; --q) {       // from the small terms on
          if (q >= mains * blk.width ? steps > 0 : q / blk.width < steps) {
            float t[16];
            tmem_ld16(at + q * r16 + j, t);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] += t[e];
          }
        }
        if (c < a.width && ok) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (j + e < r) {
              float* o = out + (int64_t)(j + e) * a.width + c;
              *o = (add ? *o : 0.f) + k * v[e];
            }
        }
        __syncwarp();
      }
      if (steps > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&drained[n % sets]);
      }
    }
    if (steps > 0) ++items;
    fills += steps;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TCOLS);
  }
}

// out[l] (+)= the sum of adapter l's slots, in their order; two outputs.
__global__ void __launch_bounds__(256)
    k_adapter_join(float* out0, const float* part0, int64_t size0, float* out1, const float* part1, int64_t size1, int T,
                   int count, int accumulate, void* plan) {
  pdl_wait_then_release();
  const PlanView pv = plan_view(plan, T, count);
  if (!plan_ok(pv, T, count)) return;
  const int l = blockIdx.y;
  const int2 slots = pv.parts[l];
  if (slots.y == 0) return;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < size0 + size1; i += gridDim.x * 256ll) {
    const bool one = i >= size0;
    const int64_t e = one ? i - size0 : i, size = one ? size1 : size0;
    const float* p = (one ? part1 : part0) + slots.x * size + e;
    float* o = (one ? out1 : out0) + l * size + e;
    float v = accumulate ? *o : 0.f;
    for (int s = 0; s < slots.y; ++s) v += p[s * size];
    *o = v;
  }
}

}  // namespace adapter
}  // namespace quip
