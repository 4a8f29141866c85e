// Device side of a kv_batch (kv_attention.h): sequence metadata, page lookup,
// the enumeration of page runs, and element types. Shared by the append, the
// attention and the scaled gather.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_attention.h"
#include "kv_common.cuh"

namespace gtkv {

struct Batch {
  const int32_t* table;
  const int32_t* start;
  const int32_t* len;
  const int64_t* cu;
  int64_t n_rows;
  int32_t n_seqs;
  int32_t max_pages;
  int32_t kernel_facing;
};

// A sequence's part of the step: tokens [a, a + n) are rows row0 + (0 .. n).
// n = 0 for a sequence without tokens or with inconsistent metadata.
struct Seq {
  int64_t row0;
  int32_t a;
  int32_t n;
};

__device__ __forceinline__ Seq seq_of(const DevPool& p, const Batch& b, int32_t s, int& bits) {
  const int64_t a = b.start ? __ldg(b.start + s) : 0;
  const int64_t e = __ldg(b.len + s);
  const int64_t c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1);
  Seq q{c0, 0, 0};
  if (a < 0 || e > static_cast<int64_t>(b.max_pages) * p.ps || c0 < 0 || c1 < c0 || c1 > b.n_rows || c1 - c0 < e - a) {
    bits |= KV_DEV_ERR_TABLE;
    return q;
  }
  if (e > a) {
    q.a = static_cast<int32_t>(a);
    q.n = static_cast<int32_t>(e - a);
  }
  return q;
}

// Raises KV_DEV_ERR_TABLE for every inconsistent sequence. Kernels that find
// sequences through rows or runs never meet one that owns none of them, so
// they have spare threads (number `first` of `step` in the grid) look at all.
__device__ __forceinline__ void check_seqs(const DevPool& p, const Batch& b, int64_t first, int64_t step, int& bits) {
  for (int64_t s = first; s < b.n_seqs; s += step) seq_of(p, b, static_cast<int32_t>(s), bits);
}

// Table entry -> physical page, 0 (the sink) for tombstones and bad entries.
__device__ __forceinline__ int64_t page_of_entry(const DevPool& p, const Batch& b, int32_t e, int& bits) {
  if (e <= 0) return 0;
  if (b.kernel_facing) {
    const uint32_t q = static_cast<uint32_t>(e) / static_cast<uint32_t>(p.blocks);
    if (q * static_cast<uint32_t>(p.blocks) != static_cast<uint32_t>(e)) {
      bits |= KV_DEV_ERR_FORM;
      return 0;
    }
    e = static_cast<int32_t>(q);
  }
  if (e >= p.num_pages) {
    bits |= KV_DEV_ERR_ROW;
    return 0;
  }
  return e;
}

// Largest s with key(s) <= x, for key non-decreasing on [0, n) with key(0) <= x
// (0 when not); the whole warp searches, 32 probes a round.
template <class F>
__device__ __forceinline__ int32_t warp_search(int32_t n, int64_t x, F&& key) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step;
    const bool le = i < hi && key(static_cast<int32_t>(i)) <= x;
    const int32_t k = __popc(__ballot_sync(kFull, le));
    lo += k * step;
    if (hi - lo > step) hi = lo + step;
  }
  return lo;
}

// Page runs: the step's tokens cut at page ends. Sequence s gets run numbers
// from base(s) = cu[s] / ps + 2 s on, room for every page that its tokens can
// touch, so all runs lie in [0, n_rows / ps + 2 n_seqs) and numbers past a
// sequence's last page are empty. By rows (decode steps, where that is the
// smaller range) a run's number is the row of its first token instead.
struct PageRun {
  int64_t row;   // row of the first token
  int64_t j;     // its index in the sequence
  int64_t page;  // physical page, 0: tombstone
  int32_t s;
  int32_t off;   // offset of the first token in the page
  int32_t m;     // tokens, 0: empty
};

// That is at about two tokens a sequence, and so is the crossing of the two forms of the 8-bit append that go with it
// (k_append_e4m3), by row and by page: 512 sequences, 8 heads of 64, pages of 32, 1 / 2 / 3 / 4 / 7 tokens 24 / 27 / 32 /
// 44 / 64 and 33 / 33 / 36 / 35 / 61 us; 64 sequences, 8 heads of 128, pages of 16, 20 / 23 / 26 / 28 / 36 and
// 19 / 21 / 20 / 19 / 25 us.
inline __host__ __device__ int64_t run_numbers(const Batch& b, int64_t ps, bool by_row) {
  return by_row ? b.n_rows : b.n_rows / ps + 2 * static_cast<int64_t>(b.n_seqs);
}
inline bool runs_by_row(const Batch& b, int64_t ps) { return run_numbers(b, ps, true) <= run_numbers(b, ps, false); }

// Called by whole warps.
__device__ __forceinline__ PageRun page_run(const DevPool& p, const Batch& b, int64_t c, bool by_row, int& bits) {
  PageRun r{0, 0, 0, 0, 0, 0};
  const int64_t ps = p.ps;
  r.s = by_row ? warp_search(b.n_seqs, c, [&](int32_t s) { return __ldg(b.cu + s); })
               : warp_search(b.n_seqs, c, [&](int32_t s) { return div_ps(p, __ldg(b.cu + s)) + 2 * static_cast<int64_t>(s); });
  const Seq q = seq_of(p, b, r.s, bits);
  if (q.n == 0) return r;
  int64_t j;  // first token
  if (by_row) {
    j = q.a + (c - q.row0);
    if (c < q.row0 || j >= static_cast<int64_t>(q.a) + q.n) return r;
    if (j != q.a && j - div_ps(p, j) * ps != 0) return r;  // not the first of its page in this step
  } else {
    const int64_t i = c - (div_ps(p, q.row0) + 2 * static_cast<int64_t>(r.s));
    if (i < 0) return r;
    j = (div_ps(p, q.a) + i) * ps;
    if (j < q.a) j = q.a;
    if (j >= static_cast<int64_t>(q.a) + q.n) return r;
  }
  const int64_t k = div_ps(p, j);
  r.off = static_cast<int32_t>(j - k * ps);
  const int64_t left = static_cast<int64_t>(q.a) + q.n - j;
  r.m = static_cast<int32_t>(left < ps - r.off ? left : ps - r.off);
  r.row = q.row0 + (j - q.a);
  r.j = j;
  r.page = page_of_entry(p, b, __ldg(b.table + static_cast<int64_t>(r.s) * b.max_pages + k), bits);
  return r;
}

// ---- element types -----------------------------------------------------------

template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};

// e4m3 code <-> float. to_e4m3 rounds to nearest even and saturates; NaN and
// infinities give the NaN code.
__device__ __forceinline__ float from_e4m3(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ uint8_t to_e4m3(float x) {
  return isfinite(x) ? __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3) : 0x7f;
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

__device__ __forceinline__ float2 halves(uint32_t h2) { return __half22float2(*reinterpret_cast<const __half2*>(&h2)); }

// Four floats as four codes; what is not finite becomes the NaN code.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  auto fin = [](float x) { return fabsf(x) <= 3.402823466e38f ? x : NAN; };
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(fin(b)), "f"(fin(a)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(fin(d)), "f"(fin(c)));
  return lo | static_cast<uint32_t>(hi) << 16;
}

// Four codes times f, as codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = halves(codes_lo(w)), b = halves(codes_hi(w));
  return encode4(a.x * f, a.y * f, b.x * f, b.y * f);
}

__device__ __forceinline__ void store_bits(const DevPool& p, int bits) {
  if (bits) atomicOr(p.err, bits);
}

}  // namespace gtkv
