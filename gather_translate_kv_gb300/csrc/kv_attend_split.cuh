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

// Where a call's partial results are, and how its units are shaped.
struct Split {
  SplitRecord* rec;   // one per worker
  float* part;        // [worker][head of the worker][slot][nq * (D + 2)]: sums, references, denominators
  int64_t n_workers;
  int32_t hw;         // KV heads of a worker
  int32_t nq;         // rows of a unit
  int32_t min_share;  // steps
  int32_t min_new, max_new;  // new tokens of the sequences that the kernel takes
  int32_t blocks;
  int32_t q_wide;     // query rows start on 16 bytes
  int32_t out_wide;   // out starts on 16 bytes
  float lift;         // log2 of the weights' lift
};

inline int64_t split_record_bytes(int64_t workers) {
  return (workers * static_cast<int64_t>(sizeof(SplitRecord)) + 255) / 256 * 256;
}

namespace {

constexpr float kNoRef = -1e30f;  // reference before the first key; finite, so that -inf - m stays -inf

constexpr int kJoinBlock = 128;

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
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two e4m3 codes (bytes 0 and 1 of a half word) as two fp16.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t y;
  asm("{.reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t y;
  asm("{.reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(y) : "r"(w));
  return y;
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

__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Joins the partial sums of units that were cut: block x looks at worker x's
// unfinished unit and adds the continuing segments of the workers after it, one
// warp a row, in the workers' order.
template <class C, int D>
__global__ void __launch_bounds__(kJoinBlock) k_attend_join(DevPool p, Batch b, AttendArgs a, Split w) {
  constexpr int E = D / 32;
  const int NQ = w.nq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t worker = blockIdx.x;
  const SplitRecord rec = w.rec[worker];
  if (rec.s < 0) return;
  int64_t last = worker + 1;
  while (last + 1 < w.n_workers && !(w.rec[last].cont & 2)) ++last;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.y * (kJoinBlock / 32) + (threadIdx.x >> 5);  // (head of the group, column)
  const int hw = item / NQ, col = item - hw * NQ;
  int bits = 0;
  const Seq q = seq_of(p, b, rec.s, bits);
  const int32_t f = rec.tile * NQ + col;
  if (hw >= w.hw || f >= q.n * a.G) return;
  auto part = [&](int64_t k) {
    return w.part + ((k * w.hw + hw) * 2 + (k == worker ? 1 : 0)) * (static_cast<int64_t>(NQ) * (D + 2));
  };
  float m = kNoRef;
  for (int64_t k = worker + lane; k <= last; k += 32) m = fmaxf(m, part(k)[NQ * D + col]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  float acc[E], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int64_t k = worker; k <= last; ++k) {
    const float* x = part(k);
    const float f_ = ex2(x[NQ * D + col] - m);
    sum += x[NQ * (D + 1) + col] * f_;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += x[col * D + lane * E + e] * f_;
  }
  const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
  bool bad = !(sum <= 3.402823466e38f);
  const int64_t r = q.row0 + f / a.G;
  const int32_t qh = (rec.head * w.hw + hw) * a.G + f % a.G;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float y = acc[e] * inv;
    bad = bad || !(fabsf(y) <= 3.402823466e38f);
    store_out(a, (r * a.Q + qh) * D + lane * E + e, y);
  }
  if (a.lse && lane == 0)
    a.lse[r * a.Q + qh] = sum == 0.0f ? -INFINITY : (m - w.lift + log2f(sum)) * kLn2;
  if (__any_sync(kFull, bad)) {
    __syncwarp();
    attend_row<C>(p, b, a, rec.s, q.a + f / a.G, r, qh, &bits);
  }
  store_bits(p, bits);
}


// The join may start while the kernel before it drains; it waits for that kernel's end itself.
template <class C, int D>
cudaError_t launch_join(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(w.n_workers),
                     static_cast<unsigned>((w.hw * w.nq + kJoinBlock / 32 - 1) / (kJoinBlock / 32)));
  cfg.blockDim = dim3(kJoinBlock);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend_join<C, D>, p, b, a, w);
}

}  // namespace

}  // namespace gtkv
