// Attention, one row at a time: the formula itself, key by key, in 32 bits.
// Used where no tensor-core kernel applies (head sizes other than 64 and 128)
// and for the rows that those kernels hand back.
#pragma once

#include "kv_attn_launch.h"
#include "kv_e2m1.cuh"

namespace gtkv {

constexpr int kAttendMaxDim = 256;
constexpr float kLn2 = 0.6931471805599453f;

// Cache element types. Head: the elements of one KV head in a row of the cache.
struct CodeE4M3 {};
struct CodeE2M1 {};

template <class C>
struct Head {
  const C* x;
  __device__ __forceinline__ Head(const void* row, const AttendArgs& a, int32_t h)
      : x(static_cast<const C*>(row) + static_cast<int64_t>(h) * a.D) {}
  __device__ __forceinline__ float operator[](int e) const { return Elem<C>::get(x[e]); }
};
template <>
struct Head<CodeE4M3> {
  const uint8_t* x;
  __device__ __forceinline__ Head(const void* row, const AttendArgs& a, int32_t h)
      : x(static_cast<const uint8_t*>(row) + static_cast<int64_t>(h) * a.D) {}
  __device__ __forceinline__ float operator[](int e) const { return from_e4m3(x[e]); }
};
template <>
struct Head<CodeE2M1> {
  const uint8_t* codes;
  const uint8_t* scales;
  __device__ __forceinline__ Head(const void* row, const AttendArgs& a, int32_t h)
      : codes(static_cast<const uint8_t*>(row) + h * (a.D / 2)),
        scales(static_cast<const uint8_t*>(row) + code_bytes(a.H, a.D) + h * (a.D / 16)) {}
  __device__ __forceinline__ float operator[](int e) const {
    return code_value(codes[e >> 1] >> 4 * (e & 1) & 15, scales[e >> 4]);
  }
};

// Does the token at position i see token j <= i? (tombstones apart)
__device__ __forceinline__ bool in_sight(const AttendArgs& a, int64_t i, int64_t j) {
  return j <= i && (a.window == 0 || i - j < a.window || j < a.sinks);
}

// Does some row at positions from i0 on, past token `j`, see one of tokens [j, last]? (tombstones apart)
// Entries of other tokens are not looked up: a window that has moved on leaves them stale.
__device__ __forceinline__ bool some_row_sees(const AttendArgs& a, int64_t i0, int64_t j, int64_t last) {
  return a.window == 0 || i0 - last < a.window || j < a.sinks;
}

__device__ __forceinline__ float load_q(const AttendArgs& a, const void* q, int64_t i) {
  return a.type == KV_TYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i])
                                : __half2float(static_cast<const __half*>(q)[i]);
}
__device__ __forceinline__ void store_out(const AttendArgs& a, int64_t i, float x) {
  if (a.type == KV_TYPE_BF16)
    static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(a.out)[i] = __float2half_rn(x);
}

// Row r (position i of sequence s), query head h, by one warp. Lane k takes key
// j0 + k of 32 for the scores, elements lane, lane + 32, ... of the head for
// the sum over values. A key out of sight is skipped, not multiplied by zero.
template <class C>
__device__ __noinline__ void attend_row(const DevPool& p, const Batch& b, const AttendArgs& a, int32_t s, int64_t i,
                                        int64_t r, int32_t h, int* bits) {
  const int lane = threadIdx.x & 31;
  const int32_t kvh = h / a.G;
  const int64_t q0 = r * a.q_stride + static_cast<int64_t>(h) * a.D;
  float acc[kAttendMaxDim / 32];
#pragma unroll
  for (int e = 0; e < kAttendMaxDim / 32; ++e) acc[e] = 0.0f;
  float top = -INFINITY, total = 0.0f;
  const int64_t lo = a.window == 0 || i + 1 <= a.window ? 0 : i + 1 - a.window;
  const int64_t sink_end = a.sinks < lo ? a.sinks : lo;
  for (int64_t j0 = 0; j0 <= i; j0 += 32) {
    if (j0 >= sink_end && j0 + 32 <= lo) {  // between the first tokens and the window
      j0 = lo / 32 * 32 - 32;
      continue;
    }
    const int64_t j = j0 + lane;
    int64_t page = 0, off = 0;
    if (j <= i && in_sight(a, i, j)) {
      const int64_t k = div_ps(p, j);
      off = j - k * p.ps;
      page = page_of_entry(p, b, __ldg(b.table + static_cast<int64_t>(s) * b.max_pages + k), *bits);
    }
    const int64_t row = page * p.stride + 2 * static_cast<int64_t>(a.layer) * p.ps + off;
    float x = -INFINITY, sv = 1.0f;
    if (page != 0) {
      float sk = 1.0f;
      if (a.scales) {
        const int64_t at = (page * p.blocks + 2 * a.layer) * a.H + kvh;
        sk = __ldg(a.scales + at);
        sv = __ldg(a.scales + at + a.H);
      }
      const Head<C> k(p.base + row * p.vpr, a, kvh);
      float d = 0.0f;
      for (int e = 0; e < a.D; ++e) d = fmaf(load_q(a, a.q, q0 + e), k[e], d);
      x = d * sk * a.scale_log2;
    }
    const uint32_t seen = __ballot_sync(kFull, page != 0);
    if (seen == 0) continue;
    float m = page != 0 ? x : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    m = fmaxf(top, m);
    const float ref = m == -INFINITY ? 0.0f : m;  // only scores of -infinity so far
    const float keep = exp2f(top - ref);
    const float w = page != 0 ? exp2f(x - ref) : 0.0f;
    top = m;
    total = total * keep + w;
#pragma unroll
    for (int e = 0; e < kAttendMaxDim / 32; ++e) acc[e] *= keep;
    for (uint32_t left = seen; left; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const int64_t rk = __shfl_sync(kFull, row, k);
      const float wk = __shfl_sync(kFull, w, k) * __shfl_sync(kFull, sv, k);
      const Head<C> v(p.base + (rk + p.ps) * p.vpr, a, kvh);
#pragma unroll
      for (int e = 0; e < kAttendMaxDim / 32; ++e)
        if (lane + 32 * e < a.D) acc[e] = fmaf(wk, v[lane + 32 * e], acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  const bool none = total == 0.0f;
#pragma unroll
  for (int e = 0; e < kAttendMaxDim / 32; ++e)
    if (lane + 32 * e < a.D) store_out(a, (r * a.Q + h) * a.D + lane + 32 * e, none ? 0.0f : acc[e] / total);
  if (a.lse && lane == 0) a.lse[r * a.Q + h] = none ? -INFINITY : (top + log2f(total)) * kLn2;
}

}  // namespace gtkv
