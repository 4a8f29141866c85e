// Append with position rotation, and the gather of an 8-bit pool's values.
//
// Rotation of pair (x1, x2) by the angle of its axis' position:
// (x1 c - x2 s, x2 c + x1 s), products and sums rounded one by one in 32
// bits, so the result does not depend on how a compiler fuses them and codes
// come out the same wherever the formula is evaluated.
//
// All of it is memory traffic: rows in, rows out, a few operations per
// element, so the kernels are built around 16-byte loads. A lane takes the 16
// elements of a "task": chunks c and c + rotary_dim / 16 of 8 elements, which
// hold 8 whole pairs under either pairing (pairs 8c .. 8c + 7 for half
// pairing, 4c .. and rotary_dim / 4 + 4c .. for adjacent pairs), so it needs 8
// cosines and 8 sines and no other lane's data, and the lanes' chunks follow
// one another. D / 16 lanes cover a head's row.
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

constexpr int kRowThreads = 64;                       // threads a row
constexpr int kRowsAtOnce = kAppendBlock / kRowThreads;
constexpr int kMaxRows = 16;                          // rows a block

constexpr int kStagePieces = 8;                        // pieces of 16 bytes a thread
constexpr int kStageBytes = kStagePieces * 16 * kAppendBlock;
constexpr int kAppendStages = 3;
constexpr int kAppendSmem = kAppendStages * kStageBytes;

// Heads [0, heads) of the list (queries, keys, values) of rows [r0, r0 + rows),
// 64 threads a row, four rows at a time. A thread copies the pieces that it
// will turn into shared memory of its own (cp.async), two batches of heads or groups of
// rows ahead, so that loads never stop; no barrier is needed for them. Where the rows belong is a
// chain of four or five dependent loads; one warp follows it, a row a lane,
// under the first copies.
template <class T>
__device__ __forceinline__ void append_rows(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t,
                                            int64_t r0, int rows, int heads, Token* tokens, uint8_t* stage, int& bits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / kRowThreads, lt = threadIdx.x % kRowThreads;
  const int nt = g.D / 16;
  const int groups = kRowThreads / nt;
  const int grp = lt / nt;
  const Task task = task_of(t, g.D, lt - grp * nt);
  constexpr int V = sizeof(T);  // pieces of a task
  constexpr int U = kStagePieces / V;  // heads a batch
  const int h_lo = grp < groups ? grp : heads;  // lanes left over by the tasks have no head
  const int batches = (heads + groups * U - 1) / (groups * U);
  const int items = (rows + kRowsAtOnce - 1) / kRowsAtOnce * batches;
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(stage)) + threadIdx.x * 16;
  auto slot = [&](int item, int u, int v) { return mine + item % kAppendStages * kStageBytes + (u * V + v) * (kAppendBlock * 16); };
  auto copy = [&](int item) {
    const int64_t r = r0 + sub + item / batches * kRowsAtOnce;
    if (item < items && r < b.n_rows && r - r0 < rows) {
      const T* q = static_cast<const T*>(g.q) + r * g.q_stride;
      const T* kk = static_cast<const T*>(g.k) + r * g.k_stride;
      const T* vv = static_cast<const T*>(g.v) + r * g.v_stride;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h_lo + (item % batches * U + u) * groups;
        if (h < heads) {
          const T* x = h < g.Q ? q + h * g.D : h < g.Q + g.H ? kk + (h - g.Q) * g.D : vv + (h - g.Q - g.H) * g.D;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const T* from = x + (v < V / 2 ? task.a : task.b) + v % (V / 2) * (16 / V);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot(item, u, v)), "l"(from) : "memory");
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  copy(0);
  copy(1);
  if (warp == 0) {  // a row a lane; the first one's sequence is searched for, the others go on from there
    int32_t q = warp_search(b.n_seqs, r0, [&](int32_t i) { return __ldg(b.cu + i); });
    const int64_t r = r0 + lane;
    if (lane < rows) {
      Token k{};
      if (r < b.n_rows) {
        while (q + 1 < b.n_seqs && r >= __ldg(b.cu + q + 1)) ++q;
        k = token_of_row(p, b, q, r, bits);
        if (k.ok && t.rd > 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int64_t at = x < t.n_axes && t.pos ? __ldg(t.pos + x * b.n_rows + r) : k.j;
            if (x < t.n_axes && (at < 0 || at >= t.n_pos)) k.ok = false;
            k.pos[x] = static_cast<int32_t>(at);
          }
          if (!k.ok) bits |= KV_DEV_ERR_POSITION;
        }
      }
      tokens[lane] = k;
    }
  } else {
    constexpr int kSpare = kAppendBlock - 32;
    check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kSpare + threadIdx.x - 32,
               static_cast<int64_t>(gridDim.x) * kSpare, bits);
  }
  __syncthreads();
  // cosines and sines of this group of rows and of the next
  float c[8], s[8], c_next[8], s_next[8];
  auto ask_cs = [&](int i) {
    if (task.f0 >= 0 && i < rows && tokens[i].ok)
      load_cs(t, task, [&](int f) -> int64_t { return tokens[i].pos[axis_of(t, f)]; }, c_next, s_next);
  };
  ask_cs(sub);
  for (int item = 0; item < items; ++item) {
    copy(item + 2);
    const int i = sub + item / batches * kRowsAtOnce;
    const bool live = i < rows && tokens[i].ok;
    if (item % batches == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = c_next[e];
        s[e] = s_next[e];
      }
      ask_cs(i + kRowsAtOnce);
    }
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    if (!live) continue;
    const int64_t r = r0 + i, page = tokens[i].page;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h_lo + (item % batches * U + u) * groups;
      if (h >= heads) break;
      T* y;
      if (h < g.Q) {
        y = static_cast<T*>(g.q_out) + (r * g.Q + h) * g.D;
      } else {
        if (page == 0) break;  // tombstone: not stored (keys and values come after all queries)
        const int kv = h >= g.Q + g.H;
        y = pool_row<T>(p, g.layer, kv, page, tokens[i].off) + (h - g.Q - kv * g.H) * g.D;
      }
      Raw<T> raw;
#pragma unroll
      for (int v = 0; v < V; ++v)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(raw.v[v].x), "=r"(raw.v[v].y), "=r"(raw.v[v].z), "=r"(raw.v[v].w)
                     : "r"(slot(item, u, v))
                     : "memory");
      if (task.f0 >= 0 && h < g.Q + g.H) {
        float x[16];
        unpack(raw, x);
        turn16(t, x, c, s);
        store16(y, task, x);
      } else {
        store_raw(y, task, raw);
      }
    }
  }
}

// Rows a block: as few as let all blocks be resident at once, two on each
// SM, and at most sixteen, which then share one chain of lookups. 8 KV
// and 32 query heads of 128 in bf16, 4 / 8 / 16 rows: 9.5 / 11.5 / 17.1 us at
// 400 rows, 15.1 / 13.5 / 17.3 at 1600, 42.0 / 35.7 / 39.9 at 6400, 171 / 144 / 135 at 32768.
inline int rows_per_block(int64_t n_rows, int sm_count) {
  const int64_t resident = 2 * static_cast<int64_t>(sm_count);
  return n_rows <= resident * kRowsAtOnce ? kRowsAtOnce : n_rows <= resident * 2 * kRowsAtOnce ? 2 * kRowsAtOnce : kMaxRows;
}

// Measured (16 sequences of 2048 tokens, three axes, 806 MB): 131 us, 90 % of the copy rate; 256
// decode tokens 5.7 us in a CUDA graph, launch and lookups (7.5 us called one by one, at the host's rate).
// Pools that hold the inputs' own type; for 8-bit pools the queries alone
// (heads = Q), launched over the tail of k_append_e4m3, which it therefore outlasts.
template <class T>
__global__ void __launch_bounds__(kAppendBlock, 2) k_append(DevPool p, Batch b, AppendArgs g, Rot t, int rows, int heads) {
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ Token tokens[kMaxRows];
  int bits = 0;
  append_rows<T>(p, b, g, t, static_cast<int64_t>(blockIdx.x) * rows, rows, heads, tokens, stage, bits);
  store_bits(p, bits);
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  const Task task = task_of(t, g.D, part);
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
      if (kv == 0 && task.f0 >= 0) {
        float c[8], s[8];
        load_cs(t, task, [&](int f) { return position(t, b, r, j, f); }, c, s);
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
// The first tokens' cosines and sines and whether their positions are good lie
// in shared memory, for all heads of the run.
constexpr int kRunTokens = 32;
struct alignas(16) RunTable {
  float cs[kRunTokens * 256];  // [token][rotary_dim], rotary_dim <= 256
  uint8_t ok[kRunTokens];
};

__device__ __forceinline__ void fill_run_table(const Batch& b, const Rot& t, const PageRun& run, RunTable* table) {
  const int m = run.m < kRunTokens ? run.m : kRunTokens;
  for (int i = threadIdx.x; i < m; i += kAppendBlock) table->ok[i] = positions_ok(t, b, run.row + i, run.j + i);
  if (t.rd == 0 || t.rd > 256) return;
  const int quads = t.rd / 4;
  for (int x = threadIdx.x; x < m * quads; x += kAppendBlock) {
    const int i = x / quads, e = x % quads * 4;
    const int f = e % (t.rd / 2);  // rotary_dim is a multiple of 16 here, so the four are one half's
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t q = position(t, b, run.row + i, run.j + i, f + k);
      v[k] = q < 0 ? 0.0f : __ldg(t.cs + q * t.rd + e + k);
    }
    *reinterpret_cast<float4*>(table->cs + i * t.rd + e) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

template <class T>
__device__ __forceinline__ void append_run(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t,
                                           const PageRun& run, int kvh, const RunTable* table, int& bits) {
  const int lane = threadIdx.x & 31;
  const int nt = g.D / 16;
  const int tpw = 32 / nt;  // tokens a wave
  const int tok = lane / nt;
  const bool in = tok < tpw;
  const Task task = task_of(t, g.D, lane - tok * nt);
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
    const bool kept = i < kRunTokens;
    if (!(kept ? table->ok[i] != 0 : positions_ok(t, b, run.row + i, run.j + i))) {
      bits |= KV_DEV_ERR_POSITION;
      return false;
    }
    unpack(raw[w], x);
    if (kv == 0 && task.f0 >= 0) {
      float c[8], s[8];
      if (kept && t.rd <= 256) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float* at = table->cs + i * t.rd + (z ? task.f1 : task.f0);
          const float4 u = *reinterpret_cast<const float4*>(at), v = *reinterpret_cast<const float4*>(at + t.rd / 2);
          c[4 * z] = u.x, c[4 * z + 1] = u.y, c[4 * z + 2] = u.z, c[4 * z + 3] = u.w;
          s[4 * z] = v.x, s[4 * z + 1] = v.y, s[4 * z + 2] = v.z, s[4 * z + 3] = v.w;
        }
      } else {
        load_cs(t, task, [&](int f) { return position(t, b, run.row + i, run.j + i, f); }, c, s);
      }
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

// Runs of a few tokens: four a block; longer ones: one, so that there are blocks enough. 512 decode
// tokens of eight 64-element heads: 22 us with four and the few-token form, 31 us page by page.
constexpr __host__ __device__ int runs_per_block(bool few) { return few ? 4 : 1; }

// A block's runs, looked up by a warp each, then shared out by head (or, where
// runs are a few tokens, by K and V).
// Measured: chunks of ~1100 fp16 tokens of 12 sequences, pages of 16: 48 us, with
// the queries' 42 and the read-out's 22 112 us together (56 at the copy rate);
// what bounds it is the second rotation and the conversions, with two blocks an SM and nothing of a warp's next head
// in flight while it codes one.
template <class T, bool FEW>
__global__ void __launch_bounds__(kAppendBlock, 2) k_append_e4m3(DevPool p, Batch b, AppendArgs g, Rot t, int64_t n_runs) {
  constexpr int kRunsPerBlock = runs_per_block(FEW);
  __shared__ PageRun runs[kRunsPerBlock];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int bits = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int NW = kAppendBlock / 32;
  if (warp < kRunsPerBlock) {
    const int64_t c = blockIdx.x * static_cast<int64_t>(kRunsPerBlock) + warp;
    PageRun run{0, 0, 0, 0, 0, 0};
    if (c < n_runs) run = page_run(p, b, c, FEW, bits);
    if (lane == 0) runs[warp] = run;
  } else {
    constexpr int kSpare = kAppendBlock - 32 * kRunsPerBlock;
    check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kSpare + threadIdx.x - 32 * kRunsPerBlock,
               static_cast<int64_t>(gridDim.x) * kSpare, bits);
  }
  __syncthreads();
  if constexpr (FEW) {
    const PageRun run = runs[warp >> 1];
    static_assert(NW == 2 * kRunsPerBlock);
    if (run.m != 0 && run.page != 0) append_run_few<T>(p, b, g, t, run, warp & 1, bits);
  } else {
    __shared__ RunTable table;
    const PageRun run = runs[0];
    if (run.m != 0 && run.page != 0) {  // (the whole block)
      fill_run_table(b, t, run, &table);
      __syncthreads();
      for (int i = warp; i < 2 * g.H; i += NW) append_run<T>(p, b, g, t, run, i, &table, bits);
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
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kAppendBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kAppendBlock, bits);
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
cudaError_t launch(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t, bool e4m3, int sm_count,
                   cudaStream_t s) {
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
    const int rows = rows_per_block(b.n_rows, sm_count);
    const int64_t row_blocks = (b.n_rows + rows - 1) / rows;
    const int64_t run_blocks = (n_runs + runs_per_block(by_row) - 1) / runs_per_block(by_row);
    if (row_blocks > 0x7fffffff || run_blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (!e4m3) {
      k_append<T><<<grid(row_blocks), kAppendBlock, kAppendSmem, s>>>(p, b, g, t, rows, g.Q + 2 * g.H);
    } else {
      auto runs = by_row ? k_append_e4m3<T, true> : k_append_e4m3<T, false>;
      runs<<<grid(run_blocks), kAppendBlock, 0, s>>>(p, b, g, t, n_runs);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess || g.Q == 0) return e;
      return launch_overlapped(k_append<T>, dim3(grid(row_blocks)), kAppendBlock, kAppendSmem, s, p, b, g, t, rows, g.Q);
    }
  }
  return cudaGetLastError();
}

// Scaled gather: a block per page run, K and then V, 16 codes a thread and
// step. A run's rows are consecutive in the pool and in the output, so both sides are whole
// streams; four loads are in flight before any store. Measured: 283 us for 1.81 GB of whole sequences (94 % of the copy
// rate), 44 us for 201 MB of 128-token windows, whose blocks wait longer on their lookups than on their rows.
template <class T>
__global__ void __launch_bounds__(kAppendBlock) k_gather_scaled(DevPool p, Batch b, const float* __restrict__ scales,
                                                                int32_t layer, int32_t H, int32_t D, T* out_k,
                                                                T* out_v, bool by_row) {
  int bits = 0;
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kAppendBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kAppendBlock, bits);
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

template <class T>
cudaError_t prepare_type() {
  return cudaFuncSetAttribute(k_append<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAppendSmem);
}

}  // namespace

cudaError_t prepare_append(const kv_pool_desc& d) {
  cudaError_t e = cudaSuccess;
  if (d.latent_only || d.head_dim % 16 != 0) return e;  // refused, or k_append_any's
  if (d.itemsize != 4) e = prepare_type<__nv_bfloat16>();
  if (d.itemsize != 4 && e == cudaSuccess) e = prepare_type<__half>();
  if (d.itemsize != 2 && e == cudaSuccess) e = prepare_type<float>();
  return e;
}

cudaError_t launch_append(const DevPool& p, const Batch& b, int32_t layer, int32_t type, bool e4m3, int32_t H,
                          int32_t D, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const kv_rotary* rot, const void* q, int64_t q_stride, int32_t Q, void* q_out, float* scales,
                          int sm_count, cudaStream_t s) {
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
    case KV_TYPE_BF16: return launch<__nv_bfloat16>(p, b, g, t, e4m3, sm_count, s);
    case KV_TYPE_F16: return launch<__half>(p, b, g, t, e4m3, sm_count, s);
    default: return launch<float>(p, b, g, t, e4m3, sm_count, s);
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
