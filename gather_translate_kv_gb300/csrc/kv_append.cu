// Append with position rotation, and the gather of an 8-bit pool's values.
//
// Rotation of pair (x1, x2) by the angle of its axis' position:
// (x1 c - x2 s, x2 c + x1 s), products and sums rounded one by one in 32
// bits, so the result does not depend on how a compiler fuses them and codes
// come out the same wherever the formula is evaluated.
//
// All of it is memory traffic: rows in, rows out, a few operations per
// element, so the kernels are built around 16-byte loads. A lane takes the 16
// elements of a "task": two 8-element chunks that hold the 8 pairs
// 8c .. 8c + 7 under either pairing (chunks c and c + rotary_dim / 16 for
// half pairing, 2c and 2c + 1 for adjacent pairs), so it needs 8 cosines and
// 8 sines and no other lane's data. D / 16 lanes cover a head's row.
#include "kv_attn_launch.h"
#include "kv_batch.cuh"

namespace gtkv {

namespace {

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

// Position of token j (row r) on the axis of pair f; -1 when outside the table.
__device__ __forceinline__ int64_t position(const Rot& t, const Batch& b, int64_t r, int64_t j, int f) {
  int64_t q = j;
  if (t.pos) {
    int a = 0;
    while (a + 1 < t.n_axes && f >= t.end[a]) ++a;
    q = __ldg(t.pos + a * b.n_rows + r);
  }
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
  int a, b;  // element offsets of its two chunks in a head
  int c8;    // first of its 8 pairs, -1: not rotated
};

__device__ __forceinline__ Task task_of(const Rot& t, int c) {
  const int n = t.rd / 16;
  if (c < n && !t.interleaved) return {c * 8, t.rd / 2 + c * 8, c * 8};
  return {c * 16, c * 16 + 8, c < n ? c * 8 : -1};
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

// Cosines and sines of the task's 8 pairs for one row (positions checked before).
__device__ __forceinline__ void load_cs(const Rot& t, const Batch& b, int64_t r, int64_t j, const Task& k,
                                        float (&c)[8], float (&s)[8]) {
  const int64_t p0 = position(t, b, r, j, k.c8), p1 = position(t, b, r, j, k.c8 + 7);
  if (p0 == p1) {  // 8 pairs of one axis (or of axes at the same position)
    bool one = true;
    for (int a = 0; a + 1 < t.n_axes; ++a) one = one && (t.end[a] <= k.c8 || t.end[a] > k.c8 + 7);
    if (one) {
      const float4* row = reinterpret_cast<const float4*>(t.cs + p0 * t.rd + k.c8);
      const float4* rsn = reinterpret_cast<const float4*>(t.cs + p0 * t.rd + t.rd / 2 + k.c8);
      const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(rsn), s1 = __ldg(rsn + 1);
      c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
      s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t q = position(t, b, r, j, k.c8 + i);
    c[i] = __ldg(t.cs + q * t.rd + k.c8 + i);
    s[i] = __ldg(t.cs + q * t.rd + t.rd / 2 + k.c8 + i);
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

// The step's token of a row: its index j in the sequence and page row, or ok = false.
struct Token {
  int64_t j;
  int64_t page;
  int32_t off;
  bool ok;
};

__device__ __forceinline__ Token token_of_row(const DevPool& p, const Batch& b, int64_t r, int& bits) {
  Token t{0, 0, 0, false};
  const int32_t s = warp_search(b.n_seqs, r, [&](int32_t i) { return __ldg(b.cu + i); });
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

constexpr int kRowThreads = 64;                       // threads a row
constexpr int kRowsAtOnce = kAppendBlock / kRowThreads;
constexpr int kMaxRows = 16;                          // rows a block

// Heads [0, heads) of the list (queries, keys, values) of rows [r0, r0 + rows),
// 64 threads a row, four rows at a time. Where the rows belong is a chain of four or
// five dependent loads; the block's warps follow it for all its rows at once,
// while the first rows' data is already on its way. A lane keeps its task and
// so its cosines and sines for all heads of a row, U of them in flight.
template <class T>
__device__ __forceinline__ void append_rows(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t,
                                            int64_t r0, int rows, int heads, Token* tokens, int& bits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / kRowThreads, lt = threadIdx.x % kRowThreads;
  const int nt = g.D / 16;
  const int groups = kRowThreads / nt;
  const int grp = lt / nt;
  const Task task = task_of(t, lt - grp * nt);
  constexpr int U = sizeof(T) == 2 ? 6 : 3;
  Raw<T> raw[U];
  const int h_lo = grp < groups ? grp : heads;  // lanes left over by the tasks have no head
  auto load = [&](int64_t r, int h0) {
    const T* q = static_cast<const T*>(g.q) + r * g.q_stride;
    const T* kk = static_cast<const T*>(g.k) + r * g.k_stride;
    const T* vv = static_cast<const T*>(g.v) + r * g.v_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * groups;
      if (h < heads)
        raw[u] = load_raw<T>(h < g.Q ? q + h * g.D : h < g.Q + g.H ? kk + (h - g.Q) * g.D : vv + (h - g.Q - g.H) * g.D,
                             task);
    }
  };
  if (sub < rows && r0 + sub < b.n_rows) load(r0 + sub, h_lo);
  for (int i = warp; i < rows; i += kAppendBlock / 32) {
    Token k{0, 0, 0, false};
    if (r0 + i < b.n_rows) {
      k = token_of_row(p, b, r0 + i, bits);
      if (k.ok && !positions_ok(t, b, r0 + i, k.j)) {
        bits |= KV_DEV_ERR_POSITION;
        k.ok = false;
      }
    }
    if (lane == 0) tokens[i] = k;
  }
  __syncthreads();
  for (int i = sub; i < rows; i += kRowsAtOnce) {
    const int64_t r = r0 + i;
    const Token k = tokens[i];
    if (!k.ok) continue;
    float c[8], s[8];
    if (i != sub) load(r, h_lo);
    if (task.c8 >= 0) load_cs(t, b, r, k.j, task, c, s);
    for (int h0 = h_lo; h0 < heads; h0 += groups * U) {
      if (h0 != h_lo) load(r, h0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * groups;
        if (h >= heads) break;
        T* y;
        if (h < g.Q) {
          y = static_cast<T*>(g.q_out) + (r * g.Q + h) * g.D;
        } else {
          if (k.page == 0) break;  // tombstone: not stored (keys and values come after all queries)
          const int kv = h >= g.Q + g.H;
          y = pool_row<T>(p, g.layer, kv, k.page, k.off) + (h - g.Q - kv * g.H) * g.D;
        }
        if (task.c8 >= 0 && h < g.Q + g.H) {
          float x[16];
          unpack(raw[u], x);
          turn16(t, x, c, s);
          store16(y, task, x);
        } else {
          store_raw(y, task, raw[u]);
        }
      }
    }
  }
}

// Rows a block: sixteen share one chain of lookups where there are blocks enough.
inline int rows_per_block(int64_t n_rows) { return n_rows >= 4096 ? kMaxRows : kRowsAtOnce; }

// Pools that hold the inputs' own type.
template <class T>
__global__ void __launch_bounds__(kAppendBlock, 2) k_append(DevPool p, Batch b, AppendArgs g, Rot t, int rows) {
  __shared__ Token tokens[kMaxRows];
  int bits = 0;
  append_rows<T>(p, b, g, t, static_cast<int64_t>(blockIdx.x) * rows, rows, g.Q + 2 * g.H, tokens, bits);
  store_bits(p, bits);
}

// The least 2^e, e >= -60, with amax <= 448 * 2^e (448 = 1.75 * 2^8), amax finite and >= 0.
__device__ __forceinline__ float power_of_two(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  e = e < -60 ? -60 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // infinities and NaN do not count
}

// The scale after the append, from the page's earlier scale (0: none) and the largest new magnitude.
__device__ __forceinline__ float new_scale(float amax, float old, float* base) {
  if (!(old > 0.0f && old <= 3.402823466e38f)) old = 0.0f;
  *base = old;
  return fmaxf(old, power_of_two(amax));
}

// 8-bit pools, few tokens a run (decode steps): a warp takes K or V of a run,
// D / 16 lanes a head, so one token of eight 64-element heads fills it. Four
// tokens and the codes of eight earlier ones are in flight per lane.
template <class T>
__device__ __forceinline__ void append_run_few(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t,
                                               const PageRun& run, int kv, int& bits) {
  const int lane = threadIdx.x & 31;
  const int nt = g.D / 16, heads_at_once = 32 / nt;
  const int grp = lane / nt, part = lane - grp * nt;
  const Task task = task_of(t, part);
  const int64_t row_bytes = p.vpr * 16;
  const int64_t stride = kv ? g.v_stride : g.k_stride;
  constexpr int M = sizeof(T) == 2 ? 4 : 2, O = 8;
  for (int h0 = 0; h0 < g.H; h0 += heads_at_once) {
    const int h = h0 + grp;
    const bool in = grp < heads_at_once && h < g.H;
    const T* src = (kv ? static_cast<const T*>(g.v) : static_cast<const T*>(g.k)) + h * g.D;
    uint8_t* page = pool_row<uint8_t>(p, g.layer, kv, run.page, 0) + h * g.D;
    float* at = g.scales + scale_at(p, g.H, run.page, g.layer, kv, in ? h : 0);
    Raw<T> raw[M];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < M; ++i)
        if (in && i0 + i < run.m) raw[i] = load_raw<T>(src + (run.row + i0 + i) * stride, task);
    };
    auto values = [&](int i0, int i, float (&x)[16]) -> bool {
      if (!in || i0 + i >= run.m) return false;
      const int64_t r = run.row + i0 + i, j = run.j + i0 + i;
      if (!positions_ok(t, b, r, j)) {
        bits |= KV_DEV_ERR_POSITION;
        return false;
      }
      unpack(raw[i], x);
      if (kv == 0 && task.c8 >= 0) {
        float c[8], s[8];
        load_cs(t, b, r, j, task, c, s);
        turn16(t, x, c, s);
      }
      return true;
    };
    uint2 old[O][2];
    auto load_old = [&](int i0) {
#pragma unroll
      for (int i = 0; i < O; ++i)
        if (in && i0 + i < run.off) {
          const uint8_t* y = page + (i0 + i) * row_bytes;
          old[i][0] = *reinterpret_cast<const uint2*>(y + task.a);
          old[i][1] = *reinterpret_cast<const uint2*>(y + task.b);
        }
    };
    load(0);
    const float before = in && run.off > 0 ? *at : 0.0f;
    load_old(0);
    float amax = 0.0f;
    for (int i0 = 0; i0 < run.m; i0 += M) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float x[16];
        if (values(i0, i, x)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(x[e]));
        }
      }
    }
    float top = amax;  // over the head's lanes
    for (int o = 1; o < nt; ++o) {
      const int other = grp * nt + (part + o) % nt;
      top = fmaxf(top, __shfl_sync(kFull, amax, other & 31));
    }
    float base;
    const float S = new_scale(top, before, &base);
    if (run.off > 0 && base != S) {  // the earlier tokens' codes under the new scale
      const float f = base / S;
      for (int i0 = 0; i0 < run.off; i0 += O) {
        if (i0 > 0) load_old(i0);
#pragma unroll
        for (int i = 0; i < O; ++i)
          if (in && i0 + i < run.off) {
            uint8_t* y = page + (i0 + i) * row_bytes;
            *reinterpret_cast<uint2*>(y + task.a) = make_uint2(rescale4(old[i][0].x, f), rescale4(old[i][0].y, f));
            *reinterpret_cast<uint2*>(y + task.b) = make_uint2(rescale4(old[i][1].x, f), rescale4(old[i][1].y, f));
          }
      }
    }
    const float inv = 1.0f / S;
    for (int i0 = 0; i0 < run.m; i0 += M) {
      if (run.m > M) load(i0);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float x[16];
        if (!values(i0, i, x)) continue;
        uint8_t* y = page + (run.off + i0 + i) * row_bytes;
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = encode4(x[4 * e] * inv, x[4 * e + 1] * inv, x[4 * e + 2] * inv, x[4 * e + 3] * inv);
        *reinterpret_cast<uint2*>(y + task.a) = make_uint2(v[0], v[1]);
        *reinterpret_cast<uint2*>(y + task.b) = make_uint2(v[2], v[3]);
      }
    }
    __syncwarp();
    if (in && part == 0) *at = S;
  }
}

// 8-bit pools, page by page: a warp takes one head of K or V of a run, 32 /
// (D / 16) tokens a wave, four waves held in registers as they were loaded, so
// a run of up to 16 tokens of 128 elements (32 of 64) is read once; longer
// runs are read again, from L1 or L2, once the scale is known. The rotation is
// done twice, for the maximum and for the codes: it is cheaper than the
// registers that would keep its result.
template <class T>
__device__ __forceinline__ void append_run(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t,
                                           const PageRun& run, int kvh, int& bits) {
  const int lane = threadIdx.x & 31;
  const int nt = g.D / 16;
  const int tpw = 32 / nt;  // tokens a wave
  const int tok = lane / nt;
  const bool in = tok < tpw;
  const Task task = task_of(t, lane - tok * nt);
  constexpr int W = 4;
  const bool one = run.m <= W * tpw;  // the run fits the registers
  const bool held = run.off > 0;
  const int kv = kvh >= g.H, h = kvh - kv * g.H;
  const T* src = (kv ? static_cast<const T*>(g.v) : static_cast<const T*>(g.k)) + h * g.D;
  const int64_t stride = kv ? g.v_stride : g.k_stride;
  Raw<T> raw[W];
  auto load = [&](int i0) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int i = i0 + w * tpw + tok;
      if (in && i < run.m) raw[w] = load_raw<T>(src + (run.row + i) * stride, task);
    }
  };
  // wave w of the tokens from i0 on: its 16 values, false where there is no such token
  auto values = [&](int i0, int w, float (&x)[16]) -> bool {
    const int i = i0 + w * tpw + tok;
    if (!in || i >= run.m) return false;
    if (!positions_ok(t, b, run.row + i, run.j + i)) {
      bits |= KV_DEV_ERR_POSITION;
      return false;
    }
    unpack(raw[w], x);
    if (kv == 0 && task.c8 >= 0) {
      float c[8], s[8];
      load_cs(t, b, run.row + i, run.j + i, task, c, s);
      turn16(t, x, c, s);
    }
    return true;
  };
  load(0);
  float* at = g.scales + scale_at(p, g.H, run.page, g.layer, kv, h);
  const float before = held ? *at : 0.0f;
  float amax = 0.0f;
  for (int i0 = 0; i0 < run.m; i0 += W * tpw) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float x[16];
      if (values(i0, w, x)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(x[e]));
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  float base;
  const float S = new_scale(amax, before, &base);
  uint8_t* page = pool_row<uint8_t>(p, g.layer, kv, run.page, 0) + h * g.D;
  const int64_t row_bytes = p.vpr * 16;
  if (held && base != S) {  // the earlier tokens' codes under the new scale
    const float f = base / S;
#pragma unroll 4
    for (int i = tok; i < run.off; i += tpw) {
      if (!in) break;
      uint8_t* y = page + i * row_bytes;
      const uint2 v0 = *reinterpret_cast<const uint2*>(y + task.a), v1 = *reinterpret_cast<const uint2*>(y + task.b);
      *reinterpret_cast<uint2*>(y + task.a) = make_uint2(rescale4(v0.x, f), rescale4(v0.y, f));
      *reinterpret_cast<uint2*>(y + task.b) = make_uint2(rescale4(v1.x, f), rescale4(v1.y, f));
    }
  }
  const float inv = 1.0f / S;
  for (int i0 = 0; i0 < run.m; i0 += W * tpw) {
    if (!one) load(i0);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float x[16];
      if (!values(i0, w, x)) continue;
      uint8_t* y = page + (run.off + i0 + w * tpw + tok) * row_bytes;
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = encode4(x[4 * e] * inv, x[4 * e + 1] * inv, x[4 * e + 2] * inv, x[4 * e + 3] * inv);
      *reinterpret_cast<uint2*>(y + task.a) = make_uint2(v[0], v[1]);
      *reinterpret_cast<uint2*>(y + task.b) = make_uint2(v[2], v[3]);
    }
  }
  __syncwarp();
  if (lane == 0) *at = S;
}

constexpr int kRunsPerBlock = 4;

// Four runs a block, looked up by a warp each, then shared out by head (or,
// where runs are a few tokens, by K and V); blocks after the runs' rotate the queries.
template <class T, bool FEW>
__global__ void __launch_bounds__(kAppendBlock, 2) k_append_e4m3(DevPool p, Batch b, AppendArgs g, Rot t, int64_t n_runs,
                                                                 int rows) {
  __shared__ Token tokens[kMaxRows];
  __shared__ PageRun runs[kRunsPerBlock];
  int bits = 0;
  const int64_t run_blocks = (n_runs + kRunsPerBlock - 1) / kRunsPerBlock;
  if (blockIdx.x >= run_blocks) {
    append_rows<T>(p, b, g, t, (blockIdx.x - run_blocks) * rows, rows, g.Q, tokens, bits);
    store_bits(p, bits);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int NW = kAppendBlock / 32;
  if (warp < kRunsPerBlock) {
    const int64_t c = blockIdx.x * static_cast<int64_t>(kRunsPerBlock) + warp;
    PageRun run{0, 0, 0, 0, 0, 0};
    if (c < n_runs) run = page_run(p, b, c, FEW, bits);
    if (lane == 0) runs[warp] = run;
  }
  __syncthreads();
  if constexpr (FEW) {
    const PageRun run = runs[warp >> 1];
    static_assert(NW == 2 * kRunsPerBlock);
    if (run.m != 0 && run.page != 0) append_run_few<T>(p, b, g, t, run, warp & 1, bits);
  } else {
    for (int i = warp; i < kRunsPerBlock * 2 * g.H; i += NW) {
      const PageRun run = runs[i / (2 * g.H)];
      if (run.m != 0 && run.page != 0) append_run<T>(p, b, g, t, run, i % (2 * g.H), bits);
    }
  }
  store_bits(p, bits);
}

// Any head size, rotary_dim, alignment or stride: a warp per (page run, head),
// a lane per pair or single element, two passes over the run's tokens for a
// head that is coded in 8 bits.
template <class T, bool E4M3>
__global__ void __launch_bounds__(kAppendBlock) k_append_any(DevPool p, Batch b, AppendArgs g, Rot t, bool by_row,
                                                             int64_t n_runs) {
  int bits = 0;
  const int lane = threadIdx.x & 31;
  const int heads = g.Q + 2 * g.H;
  const int half = t.rd / 2;
  const int units = half + (g.D - t.rd);  // pairs, then single elements
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAppendBlock / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kAppendBlock / 32) + (threadIdx.x >> 5); w < n_runs * heads;
       w += warps) {
    const int64_t c = w / heads;
    const int head = static_cast<int>(w - c * heads);
    const PageRun run = page_run(p, b, c, by_row, bits);
    const bool is_q = head < g.Q;
    if (run.m == 0 || (run.page == 0 && !is_q)) continue;
    const int kv = head >= g.Q + g.H, h = is_q ? head : head - g.Q - kv * g.H;
    const int64_t jseq = run.j;
    const T* src = static_cast<const T*>(is_q ? g.q : kv ? g.v : g.k) + static_cast<int64_t>(h) * g.D;
    const int64_t stride = is_q ? g.q_stride : kv ? g.v_stride : g.k_stride;
    // element offsets and values of unit u of token i
    auto value = [&](int i, int u, int& e1, int& e2, float& x1, float& x2) {
      const T* row = src + (run.row + i) * stride;
      if (u < half) {
        e1 = t.interleaved ? 2 * u : u;
        e2 = t.interleaved ? 2 * u + 1 : u + half;
        x1 = Elem<T>::get(row[e1]);
        x2 = Elem<T>::get(row[e2]);
        if (is_q || kv == 0) {
          const int64_t ps = position(t, b, run.row + i, jseq + i, u);
          turn(x1, x2, __ldg(t.cs + ps * t.rd + u), __ldg(t.cs + ps * t.rd + half + u));
        }
      } else {
        e1 = t.rd + (u - half);
        e2 = -1;
        x1 = Elem<T>::get(row[e1]);
        x2 = 0.0f;
      }
    };
    const bool coded = E4M3 && !is_q;
    float inv = 1.0f;
    float S = 0.0f;
    float* at = nullptr;
    if (coded) {
      float amax = 0.0f;
      for (int i = 0; i < run.m; ++i) {
        if (!positions_ok(t, b, run.row + i, jseq + i)) continue;
        for (int u = lane; u < units; u += 32) {
          int e1, e2;
          float x1, x2;
          value(i, u, e1, e2, x1, x2);
          amax = fmaxf(amax, fmaxf(finite_abs(x1), finite_abs(x2)));
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      at = g.scales + scale_at(p, g.H, run.page, g.layer, kv, h);
      const bool held = run.off > 0;
      float base;
      S = new_scale(amax, held ? *at : 0.0f, &base);
      if (held && base != S) {
        const float f = base / S;
        for (int i = 0; i < run.off; ++i) {
          uint8_t* y = pool_row<uint8_t>(p, g.layer, kv, run.page, i) + h * g.D;
          for (int e = lane; e < g.D; e += 32) y[e] = to_e4m3(from_e4m3(y[e]) * f);
        }
      }
      inv = 1.0f / S;
    }
    for (int i = 0; i < run.m; ++i) {
      if (!positions_ok(t, b, run.row + i, jseq + i)) {
        bits |= KV_DEV_ERR_POSITION;
        continue;
      }
      for (int u = lane; u < units; u += 32) {
        int e1, e2;
        float x1, x2;
        value(i, u, e1, e2, x1, x2);
        if (coded) {
          uint8_t* y = pool_row<uint8_t>(p, g.layer, kv, run.page, run.off + i) + h * g.D;
          y[e1] = to_e4m3(x1 * inv);
          if (e2 >= 0) y[e2] = to_e4m3(x2 * inv);
        } else {
          T* y = is_q ? static_cast<T*>(g.q_out) + ((run.row + i) * g.Q + h) * g.D
                      : pool_row<T>(p, g.layer, kv, run.page, run.off + i) + h * g.D;
          y[e1] = Elem<T>::put(x1);
          if (e2 >= 0) y[e2] = Elem<T>::put(x2);
        }
      }
    }
    __syncwarp();
    if (coded && lane == 0) *at = S;
  }
  store_bits(p, bits);
}

bool vec16(const void* x, int64_t stride, size_t size) {
  return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (stride * static_cast<int64_t>(size)) % 16 == 0;
}

template <class T>
cudaError_t launch(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t, bool e4m3, cudaStream_t s) {
  const bool by_row = runs_by_row(b, p.ps);
  const int64_t n_runs = run_numbers(b, p.ps, by_row);
  const bool wide = g.D % 16 == 0 && g.D <= 512 && t.rd % 16 == 0 && vec16(g.k, g.k_stride, sizeof(T)) &&
                    vec16(g.v, g.v_stride, sizeof(T)) && vec16(t.cs, 0, 4) &&
                    (g.Q == 0 || (vec16(g.q, g.q_stride, sizeof(T)) && vec16(g.q_out, 0, 2)));
  auto grid = [](int64_t n) { return static_cast<unsigned>(n < 1 ? 1 : n > 0x7fffffff ? 0x7fffffff : n); };
  if (!wide) {
    const unsigned n = grid((n_runs * (g.Q + 2 * g.H) + kAppendBlock / 32 - 1) / (kAppendBlock / 32));
    if (e4m3)
      k_append_any<T, true><<<n, kAppendBlock, 0, s>>>(p, b, g, t, by_row, n_runs);
    else
      k_append_any<T, false><<<n, kAppendBlock, 0, s>>>(p, b, g, t, by_row, n_runs);
  } else {
    const int rows = rows_per_block(b.n_rows);
    const int64_t row_blocks = (b.n_rows + rows - 1) / rows;
    const int64_t run_blocks = (n_runs + kRunsPerBlock - 1) / kRunsPerBlock;
    if (row_blocks + run_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned blocks = grid(run_blocks + (g.Q ? row_blocks : 0));
    if (!e4m3)
      k_append<T><<<grid(row_blocks), kAppendBlock, 0, s>>>(p, b, g, t, rows);
    else if (by_row)
      k_append_e4m3<T, true><<<blocks, kAppendBlock, 0, s>>>(p, b, g, t, n_runs, rows);
    else
      k_append_e4m3<T, false><<<blocks, kAppendBlock, 0, s>>>(p, b, g, t, n_runs, rows);
  }
  return cudaGetLastError();
}

// Scaled gather: a block per page run, K and then V, 16 codes a thread and
// step. A run's rows are consecutive in the pool and in the output, so both sides are whole
// streams; four loads are in flight before any store.
template <class T>
__global__ void __launch_bounds__(kAppendBlock) k_gather_scaled(DevPool p, Batch b, const float* __restrict__ scales,
                                                                int32_t layer, int32_t H, int32_t D, T* out_k,
                                                                T* out_v, bool by_row) {
  int bits = 0;
  const PageRun run = page_run(p, b, blockIdx.x, by_row, bits);
  store_bits(p, bits);
  if (run.m == 0) return;
  const int32_t vpr = static_cast<int32_t>(p.vpr);
  const int64_t n = static_cast<int64_t>(run.m) * vpr;
  const bool whole = D % 16 == 0;  // a piece of 16 codes lies in one head
  constexpr int U = 4;
  const int32_t step = kAppendBlock % vpr;
  for (int kv = 0; kv < 2; ++kv) {
    const uint4* src = reinterpret_cast<const uint4*>(pool_row<uint8_t>(p, layer, kv, run.page, run.off));
    T* dst = (kv ? out_v : out_k) + run.row * H * D;
    const float* sc = scales + scale_at(p, H, run.page, layer, kv, 0);
    int32_t col = threadIdx.x % vpr;  // piece of the row
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += kAppendBlock * U) {
      uint4 v[U];
      float f[U];
      int32_t cols[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * kAppendBlock;
        cols[u] = col;
        v[u] = make_uint4(0, 0, 0, 0);
        f[u] = 0.0f;
        if (i < n && run.page != 0) {
          v[u] = __ldg(src + i);
          if (whole) f[u] = __ldg(sc + col * 16 / D);
        }
        col += step;
        if (col >= vpr) col -= vpr;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * kAppendBlock;
        if (i >= n) break;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        float x[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = halves(codes_lo(w[k])), hi = halves(codes_hi(w[k]));
          x[4 * k] = lo.x, x[4 * k + 1] = lo.y, x[4 * k + 2] = hi.x, x[4 * k + 3] = hi.y;
        }
        if (whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = run.page != 0 ? x[k] * f[u] : 0.0f;
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = run.page != 0 ? x[k] * __ldg(sc + (cols[u] * 16 + k) / D) : 0.0f;
        }
        uint4 o[sizeof(T)];
        T* y = reinterpret_cast<T*>(o);
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = Elem<T>::put(x[k]);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(T)); ++k) {
          uint4* to = reinterpret_cast<uint4*>(dst + i * 16) + k;
          asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(to), "r"(o[k].x), "r"(o[k].y), "r"(o[k].z),
                       "r"(o[k].w)
                       : "memory");
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(const DevPool& p, const Batch& b, int32_t layer, int32_t type, bool e4m3, int32_t H,
                          int32_t D, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const kv_rotary* rot, const void* q, int64_t q_stride, int32_t Q, void* q_out, float* scales,
                          cudaStream_t s) {
  Rot t{};
  t.n_axes = 1;
  if (rot != nullptr && rot->rotary_dim > 0) {
    t.cs = rot->cos_sin_dev;
    t.pos = rot->positions_dev;
    t.n_pos = rot->n_positions;
    t.rd = rot->rotary_dim;
    t.interleaved = rot->interleaved;
    t.n_axes = rot->n_axes;
    int end = 0;
    for (int a = 0; a < rot->n_axes; ++a) t.end[a] = end += rot->axis_pairs[a];
  }
  const AppendArgs g{k, v, q, q_out, scales, k_stride, v_stride, q_stride, H, Q, D, layer};
  switch (type) {
    case KV_TYPE_BF16: return launch<__nv_bfloat16>(p, b, g, t, e4m3, s);
    case KV_TYPE_F16: return launch<__half>(p, b, g, t, e4m3, s);
    default: return launch<float>(p, b, g, t, e4m3, s);
  }
}

cudaError_t launch_gather_scaled(const DevPool& p, const Batch& b, int32_t layer, int32_t H, int32_t D,
                                 const float* scales, int32_t type, void* out_k, void* out_v, cudaStream_t s) {
  const bool by_row = runs_by_row(b, p.ps);
  const int64_t n_runs = run_numbers(b, p.ps, by_row);
  if (n_runs > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&]<class T>(T* k, T* v) {
    k_gather_scaled<T><<<static_cast<unsigned>(n_runs), kAppendBlock, 0, s>>>(p, b, scales, layer, H, D, k, v, by_row);
  };
  if (type == KV_TYPE_BF16)
    go(static_cast<__nv_bfloat16*>(out_k), static_cast<__nv_bfloat16*>(out_v));
  else if (type == KV_TYPE_F16)
    go(static_cast<__half*>(out_k), static_cast<__half*>(out_v));
  else
    go(static_cast<float*>(out_k), static_cast<float*>(out_v));
  return cudaGetLastError();
}

}  // namespace gtkv
