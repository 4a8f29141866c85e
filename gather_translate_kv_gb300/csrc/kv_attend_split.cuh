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

#include "kv_attend.cuh"

namespace gtkv {

// Rows [f0, f1) of sequence q: blocks [0, n_first) and [b0, b1) of `step` keys.
struct KeySpan {
  int32_t n_first;  // blocks that hold the first tokens, before the window's
  int32_t b0, b1;
  __device__ __forceinline__ int32_t steps() const { return n_first + b1 - b0; }
  __device__ __forceinline__ int32_t block(int32_t i) const { return i < n_first ? i : b0 + (i - n_first); }
};

template <int STEP>
__device__ __forceinline__ KeySpan key_span(const AttendArgs& a, const Seq& q, int32_t f0, int32_t f1) {
  const int32_t i0 = q.a + f0 / a.G, i1 = q.a + (f1 - 1) / a.G;  // first and last position
  KeySpan k;
  k.b1 = i1 / STEP + 1;
  const int32_t lo = a.window && i0 + 1 > a.window ? i0 + 1 - a.window : 0;
  k.b0 = lo / STEP;
  const int32_t first = a.window ? (a.sinks < lo ? a.sinks : lo) : 0;
  const int32_t nf = (first + STEP - 1) / STEP;
  k.n_first = nf < k.b0 ? nf : k.b0;
  return k;
}

// What a worker leaves behind for the join.
struct SplitRecord {
  int32_t s, tile, head;  // unit of the unfinished last segment (slot 1), s < 0: none
  int32_t cont;           // bit 0: slot 0 holds a continuing segment; bit 1: the unit ends with it
};

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

}  // namespace gtkv
