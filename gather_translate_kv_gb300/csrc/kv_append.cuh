// Pieces of the append kernels: the rotation, a lane's 16 elements of a head, where rows lie
// in the pool. Shared by kv_append.cu and kv_append4.cu.
#pragma once

#include "kv_attn_launch.h"
#include "kv_batch.cuh"

namespace gtkv {

constexpr int kAppendBlock = 256;

struct Rot {
  const float* cs;
  const int32_t* pos;
  int64_t n_pos;
  int32_t rd;  // rotary_dim, 0: no rotation
  int32_t interleaved;
  int32_t n_axes;
  int32_t end[4];  // first pair past each axis
};

// Axis of pair f.
__device__ __forceinline__ int axis_of(const Rot& t, int f) {
  return (t.n_axes > 1 && f >= t.end[0]) + (t.n_axes > 2 && f >= t.end[1]) + (t.n_axes > 3 && f >= t.end[2]);
}

// Position of token j (row r) on the axis of pair f; -1 when outside the table.
__device__ __forceinline__ int64_t position(const Rot& t, const Batch& b, int64_t r, int64_t j, int f) {
  const int64_t q = t.pos ? __ldg(t.pos + axis_of(t, f) * b.n_rows + r) : j;
  return q >= 0 && q < t.n_pos ? q : -1;
}

// Whether every axis' position of the row lies in the table.
__device__ __forceinline__ bool positions_ok(const Rot& t, const Batch& b, int64_t r, int64_t j) {
  if (t.rd == 0) return true;
  if (!t.pos) return j < t.n_pos;
  for (int a = 0; a < t.n_axes; ++a) {
    const int64_t q = __ldg(t.pos + a * b.n_rows + r);
    if (q < 0 || q >= t.n_pos) return false;
  }
  return true;
}

__device__ __forceinline__ void turn(float& x1, float& x2, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  const float b = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = a;
  x2 = b;
}

// ---- a lane's task -----------------------------------------------------------

struct Task {
  int a, b;    // element offsets of its two chunks in a head
  int f0, f1;  // first of the first and of the last four of its 8 pairs, -1: not rotated
};

__device__ __forceinline__ Task task_of(const Rot& t, int D, int c) {
  const int n = t.rd / 16;
  if (c >= n) return {t.rd + (c - n) * 8, t.rd + (D - t.rd) / 2 + (c - n) * 8, -1, -1};
  if (t.interleaved) return {c * 8, t.rd / 2 + c * 8, c * 4, t.rd / 4 + c * 4};
  return {c * 8, t.rd / 2 + c * 8, c * 8, c * 8 + 4};
}

template <class T>
struct Raw {
  uint4 v[sizeof(T)];  // 16 elements: sizeof(T) vectors of 16 bytes
};

template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* x, const Task& k) {
  Raw<T> r;
  constexpr int N = sizeof(T) / 2;  // vectors a chunk
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r.v[i] = *reinterpret_cast<const uint4*>(x + k.a + i * (16 / sizeof(T)));
    r.v[N + i] = *reinterpret_cast<const uint4*>(x + k.b + i * (16 / sizeof(T)));
  }
  return r;
}

template <class T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&x)[16]) {
  const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = Elem<T>::get(e[i]);
}

template <class T>
__device__ __forceinline__ void store16(T* y, const Task& k, const float (&x)[16]) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
  for (int i = 0; i < 16; ++i) e[i] = Elem<T>::put(x[i]);
  constexpr int N = sizeof(T) / 2;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    *reinterpret_cast<uint4*>(y + k.a + i * (16 / sizeof(T))) = r.v[i];
    *reinterpret_cast<uint4*>(y + k.b + i * (16 / sizeof(T))) = r.v[N + i];
  }
}

template <class T>
__device__ __forceinline__ void store_raw(T* y, const Task& k, const Raw<T>& r) {
  constexpr int N = sizeof(T) / 2;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    *reinterpret_cast<uint4*>(y + k.a + i * (16 / sizeof(T))) = r.v[i];
    *reinterpret_cast<uint4*>(y + k.b + i * (16 / sizeof(T))) = r.v[N + i];
  }
}

// Cosines and sines of the task's 8 pairs; pos(f): position on the axis of
// pair f (positions checked before).
template <class F>
__device__ __forceinline__ void load_cs(const Rot& t, const Task& k, F&& pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int f = h ? k.f1 : k.f0;
    if (axis_of(t, f) == axis_of(t, f + 3)) {
      const float* row = t.cs + pos(f) * t.rd + f;
      const float4 x = __ldg(reinterpret_cast<const float4*>(row)), y = __ldg(reinterpret_cast<const float4*>(row + t.rd / 2));
      c[4 * h] = x.x, c[4 * h + 1] = x.y, c[4 * h + 2] = x.z, c[4 * h + 3] = x.w;
      s[4 * h] = y.x, s[4 * h + 1] = y.y, s[4 * h + 2] = y.z, s[4 * h + 3] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* row = t.cs + pos(f + i) * t.rd + f + i;
        c[4 * h + i] = __ldg(row);
        s[4 * h + i] = __ldg(row + t.rd / 2);
      }
    }
  }
}

// Two products an instruction, each rounded as on its own. (Sums stay apart: a packed product and a packed sum are
// fused into one rounding, whatever their rounding says.)
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// turn16 two pairs at a time (half pairing), for the kernel that has more to do than to move rows.
__device__ __forceinline__ void turn16_wide(const Rot& t, float (&x)[16], const float (&c)[8], const float (&s)[8]) {
  if (t.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x1 = make_float2(x[i], x[i + 1]), x2 = make_float2(x[8 + i], x[9 + i]);
    const float2 cc = make_float2(c[i], c[i + 1]), ss = make_float2(s[i], s[i + 1]);
    const float2 c1 = mul2(x1, cc), s2 = mul2(x2, ss), c2 = mul2(x2, cc), s1 = mul2(x1, ss);
    x[i] = __fsub_rn(c1.x, s2.x), x[i + 1] = __fsub_rn(c1.y, s2.y);
    x[8 + i] = __fadd_rn(c2.x, s1.x), x[9 + i] = __fadd_rn(c2.y, s1.y);
  }
}

__device__ __forceinline__ void turn16(const Rot& t, float (&x)[16], const float (&c)[8], const float (&s)[8]) {
  if (t.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], c[i], s[i]);
  }
}

// The token of row r, if it is one of sequence s (ok): its index j in the sequence and its page row.
struct Token {
  int64_t j;
  int64_t page;
  int32_t off;
  bool ok;
  int32_t pos[4];  // on each axis
};

__device__ __forceinline__ Token token_of_row(const DevPool& p, const Batch& b, int32_t s, int64_t r, int& bits) {
  Token t{};
  const Seq q = seq_of(p, b, s, bits);
  if (r < q.row0 || r - q.row0 >= q.n) return t;
  t.j = q.a + (r - q.row0);
  const int64_t k = div_ps(p, t.j);
  t.off = static_cast<int32_t>(t.j - k * p.ps);
  t.page = page_of_entry(p, b, __ldg(b.table + static_cast<int64_t>(s) * b.max_pages + k), bits);
  t.ok = true;
  return t;
}

struct AppendArgs {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  float* scales;
  int64_t k_stride, v_stride, q_stride;  // elements
  int32_t H, Q, D;
  int32_t layer;
};

// First element of (page, offset, K or V, head 0) of the layer in the pool.
template <class T>
__device__ __forceinline__ T* pool_row(const DevPool& p, int32_t layer, int kv, int64_t page, int64_t off) {
  const int64_t row = page * p.stride + (2 * static_cast<int64_t>(layer) + kv) * p.ps + off;
  return reinterpret_cast<T*>(p.base + row * p.vpr);
}

__device__ __forceinline__ int64_t scale_at(const DevPool& p, int32_t H, int64_t page, int32_t layer, int kv, int h) {
  return (page * p.blocks + 2 * layer + kv) * H + h;  // blocks = 2L: [page][layer][K or V][head]
}

// 4-bit pools, any head size, rotary_dim, alignment or stride (kv_append4.cu).
template <class T>
cudaError_t launch_append4_any(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t, bool by_row,
                               int64_t n_runs, cudaStream_t s);

}  // namespace gtkv
