// How attention's work is cut: the visible keys of a unit, equal shares of
// all units' steps for the workers, and the records from which partial
// results are joined. Shared by the attention kernels.
//
// A unit is one tile of a sequence's rows for one KV head (or group of
// heads); a row is a (token, query head of the group) pair, f = token * G +
// head. Its steps are blocks of keys that some row of the tile sees. All steps
// of all units form one line; worker w takes [w * share, (w + 1) * share) of
// it, so every worker has the same work whatever the lengths, and only a unit
// that straddles a border is cut. A worker's first segment may continue a unit
// (partial slot 0) and its last may leave one unfinished (slot 1).
#pragma once

#include <type_traits>

#include "kv_attend.cuh"
#include "kv_attend_launch.h"

namespace gtkv {

// Rows at positions i0 to i1: blocks [0, n_first) and [b0, b1) of STEP keys.
struct KeySpan {
  int32_t n_first;  // blocks that hold the first tokens, before the window's
  int32_t b0, b1;
  __device__ __forceinline__ int32_t steps() const { return n_first + b1 - b0; }
  __device__ __forceinline__ int32_t block(int32_t i) const { return i < n_first ? i : b0 + (i - n_first); }
};

template <int STEP>
__device__ __forceinline__ KeySpan key_span(const AttendArgs& a, int32_t i0, int32_t i1) {
  KeySpan k;
  k.b1 = i1 / STEP + 1;
  const int32_t lo = a.window && i0 + 1 > a.window ? i0 + 1 - a.window : 0;
  k.b0 = lo / STEP;
  const int32_t first = a.window ? (a.sinks < lo ? a.sinks : lo) : 0;
  const int32_t nf = (first + STEP - 1) / STEP;
  k.n_first = nf < k.b0 ? nf : k.b0;
  return k;
}

// Where the workers' shares begin. Called by all THREADS threads of a block
// for its KW workers; loc[k] = {sequence, offset in its steps} or s = -1.
struct ShareStart {
  int32_t s;
  int64_t off;
};

template <int THREADS, int KW, class F>
__device__ __forceinline__ int64_t find_shares(int32_t n_seqs, int64_t first_worker, int64_t n_workers,
                                               int32_t min_share, ShareStart* loc, int64_t* tmp, F&& steps_of) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = THREADS / 32;
  int64_t sum = 0, mine = 0;
  for (int32_t s = tid; s < n_seqs; s += THREADS) {
    mine = steps_of(s);
    sum += mine;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) tmp[warp] = sum;
  if (tid < KW) loc[tid].s = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) total += tmp[w];
  __syncthreads();
  int64_t share = (total + n_workers - 1) / n_workers;
  if (share < min_share) share = min_share;
  int64_t base = 0;
  const int64_t last = (first_worker + KW - 1) * share;  // start of the block's last worker
  for (int32_t s0 = 0; s0 < n_seqs && base <= last; s0 += THREADS) {
    const int32_t s = s0 + tid;
    const int64_t n = s >= n_seqs ? 0 : n_seqs <= THREADS ? mine : steps_of(s);
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    int64_t before = base, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += tmp[w];
      all += tmp[w];
    }
    const int64_t begin = before + inc - n;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int64_t at = (first_worker + k) * share;
      if (at >= begin && at < begin + n) {
        loc[k].s = s;
        loc[k].off = at - begin;
      }
    }
    base += all;
    __syncthreads();
  }
  __syncthreads();
  return share;
}

namespace {

constexpr float kNoRef = -1e30f;  // reference before the first key; finite, so that -inf - m stays -inf

constexpr int kJoinBlock = 256;

__device__ __forceinline__ uint32_t shared_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? N : 0;  // 0: the bytes become zero
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// All ones in the elements of a word of cached values that are not finite.
template <class C>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (std::is_same_v<C, CodeE4M3>)
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  else if constexpr (std::is_same_v<C, __half>)
    return __vcmpeq2(w & 0x7c007c00u, 0x7c007c00u);
  else
    return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Over the whole range, subnormal results included (a quick division is 0 for
// divisors past 2^126, which denominators under the smallest scales of 8-bit values reach).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return BF16 ? pack_b(lo, hi) : pack_h(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  return BF16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : halves(w);
}

// Where the segments of a cut unit meet when no join follows (shared prefixes): a binary tree over them in the workers'
// order. Of the two halves of a node the one that is done first leaves its sums and goes on to its other work; the
// second adds them to its own and goes up. The sums do not depend on who was first.
struct TreePlace {
  int32_t worker0;   // of the unit's first segment
  int32_t n;         // segments
  int32_t a;         // first segment of what the warp holds
  int32_t s;         // it holds [a, a + s) of them
  int32_t node;      // worker whose node it meets the other half at
  bool left;         // it holds the left half

  // The first of n segments.
  __device__ __forceinline__ void begin(int32_t worker, int32_t segments) {
    worker0 = worker;
    n = segments;
    a = 0;
    s = 1;
  }
  // A later one, at the start of the worker's share: `in` of the unit's part of the line lies before it.
  __device__ __forceinline__ void go_on(int64_t worker, int64_t share, int64_t in, int32_t steps, int32_t unit_cost) {
    const int64_t first = worker * share - in + unit_cost;  // the first step in the line of all
    worker0 = static_cast<int32_t>(first / share);
    n = static_cast<int32_t>((first + steps - 1) / share) - worker0 + 1;
    a = static_cast<int32_t>(worker) - worker0;
    s = 1;
  }
  // The next node; false when the warp holds all segments.
  __device__ __forceinline__ bool up() {
    while (s < n) {
      if (a / s & 1) {
        left = false;
        node = worker0 + a;
        return true;
      }
      if (a + s < n) {
        left = true;
        node = worker0 + a + s;
        return true;
      }
      s *= 2;  // nobody to meet
    }
    return false;
  }
  __device__ __forceinline__ void joined() {
    if (!left) a -= s;
    s *= 2;
  }
};

// A warp's step at a node: true when the other half is there, left by worker *other. `leave` writes
// the warp's sums where the other half will look for them.
template <class F>
__device__ __forceinline__ bool meet(int32_t* node, int32_t worker, int32_t* other, F&& leave) {
  const int lane = threadIdx.x & 31;
  int32_t x = 0;
  if (lane == 0) asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(node) : "memory");
  x = __shfl_sync(kFull, x, 0);
  if (x == 0) {
    leave();
    __threadfence();
    __syncwarp();
    if (lane == 0) x = atomicExch(node, worker + 1);
    x = __shfl_sync(kFull, x, 0);
    if (x == 0) return false;
  }
  __syncwarp();  // what lane 0 has seen comes before the other lanes' loads
  __threadfence();
  *other = x - 1;
  return true;
}

// Joins the partial sums of units that were cut, adding a unit's segments in
// the workers' order under a running reference. An item is a row of a cut unit; a warp takes one, or,
// when there are few items (a long context of few rows, cut many times), the
// eight warps of a block share its segments. It reads what the cut units left, a few MB at most
// (2 * workers * rows * (D + 2) floats), and overlaps the attention kernel's
// tail.
template <class C, int D>
__device__ __forceinline__ void join_split(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w,
                                           int32_t* owners, float* tmp, int& bits) {
  constexpr int E = D / 32, NW = kJoinBlock / 32, U = 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the workers that left a unit unfinished, and their rows (at most 256)
  int32_t count = 0;
  int32_t* warp_count = reinterpret_cast<int32_t*>(tmp);
  for (int32_t w0 = 0; w0 < w.n_workers; w0 += kJoinBlock) {
    int32_t nf = 0;
    if (w0 + tid < w.n_workers && w.rec[w0 + tid].s >= 0) nf = w.rec[w0 + tid].nf;
    const uint32_t vote = __ballot_sync(kFull, nf > 0);
    if (lane == 0) warp_count[warp] = __popc(vote);
    __syncthreads();
    int32_t at = count;
    for (int k = 0; k < NW; ++k) {
      if (k < warp) at += warp_count[k];
      count += warp_count[k];
    }
    if (nf > 0) owners[at + __popc(vote & ((1u << lane) - 1))] = (w0 + tid) << 9 | nf;
    __syncthreads();
  }
  const int32_t rows = w.hw * w.nq;
  const int32_t items = count * rows;
  const bool shared = items <= 2 * static_cast<int32_t>(gridDim.x);  // a block an item
  const int32_t stride = shared ? gridDim.x : gridDim.x * NW;
  const int64_t part_floats = static_cast<int64_t>(w.nq) * (D + 2);
  auto add = [&](float& m, float& sum, float (&acc)[E], float m2, float s2, const float (&x)[E]) {
    const float top = fmaxf(m, m2);
    const float k1 = ex2(m - top), k2 = ex2(m2 - top);
    m = top;
    sum = sum * k1 + s2 * k2;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * k1 + x[e] * k2;
  };
  for (int32_t i = shared ? blockIdx.x : blockIdx.x * NW + warp; i < items; i += stride) {
    const int32_t owner = owners[i / rows], worker = owner >> 9;
    const int32_t hw = i % rows / w.nq, col = i % w.nq;
    if (col >= (owner & 511)) continue;
    const SplitRecord rec = w.rec[worker];
    float m = kNoRef, sum = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    const int32_t kd = shared ? NW : 1;
    for (int32_t k0 = worker + (shared ? warp : 0); k0 <= rec.last; k0 += U * kd) {
      float mk[U], sk[U], x[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t k = k0 + u * kd;
        mk[u] = kNoRef;
        sk[u] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = 0.0f;
        if (k <= rec.last) {
          const float* at = w.part + ((static_cast<int64_t>(k) * w.hw + hw) * 2 + (k == worker ? 1 : 0)) * part_floats;
          mk[u] = at[w.nq * D + col];
          sk[u] = at[w.nq * (D + 1) + col];
#pragma unroll
          for (int e = 0; e < E; ++e) x[u][e] = at[col * D + lane * E + e];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add(m, sum, acc, mk[u], sk[u], x[u]);
    }
    if (shared) {
      float* at = tmp + warp * (D + 2);
#pragma unroll
      for (int e = 0; e < E; ++e) at[lane * E + e] = acc[e];
      if (lane == 0) at[D] = m, at[D + 1] = sum;
      __syncthreads();
      if (warp == 0) {
        for (int k = 1; k < NW; ++k) {
          float x[E];
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = tmp[k * (D + 2) + lane * E + e];
          add(m, sum, acc, tmp[k * (D + 2) + D], tmp[k * (D + 2) + D + 1], x);
        }
      }
    }
    if (!shared || warp == 0) {
      const float inv = sum == 0.0f ? 0.0f : rcp(sum);
      bool bad = !(sum <= 3.402823466e38f);
      const int32_t f = rec.f0 + col;
      const int64_t r = rec.row0 + f / a.G;
      const int32_t qh = (rec.head * w.hw + hw) * a.G + f % a.G;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = acc[e] * inv;
        bad = bad || !(fabsf(y) <= 3.402823466e38f);
        store_out(a, (r * a.Q + qh) * D + lane * E + e, y);
      }
      if (a.lse && lane == 0) a.lse[r * a.Q + qh] = sum == 0.0f ? -INFINITY : (m - w.lift + log2f(sum)) * kLn2;
      if (__any_sync(kFull, bad)) {
        __syncwarp();
        attend_row<C>(p, b, a, rec.s, rec.a + f / a.G, r, qh, &bits);
      }
    }
    if (shared) __syncthreads();
  }
}

// Looks at groups on the way, where there are any.
template <class C, int D>
__global__ void __launch_bounds__(kJoinBlock) k_attend_join(DevPool p, Batch b, AttendArgs a, Split few, Split tile,
                                                               Groups g) {
  __shared__ int32_t owners[kMaxWorkers];
  __shared__ float tmp[kJoinBlock / 32 * (D + 2)];
  int bits = 0;
  // while the kernels before it run
  if (g.first && blockIdx.x == 0 && groups_bad(b, g, threadIdx.x, kJoinBlock)) bits |= KV_DEV_ERR_TABLE;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (few.n_workers) join_split<C, D>(p, b, a, few, owners, tmp, bits);
  __syncthreads();
  if (tile.n_workers) join_split<C, D>(p, b, a, tile, owners, tmp, bits);
  store_bits(p, bits);
}

}  // namespace

}  // namespace gtkv
