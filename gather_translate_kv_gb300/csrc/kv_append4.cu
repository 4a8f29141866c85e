// 4-bit pools (KV_FORMAT_E2M1): append for any head size, rotary_dim, alignment
// or stride, and the gather of the values. The append of ordinary shapes is
// k_append's (kv_append.cu).
#include "kv_append.cuh"
#include "kv_e2m1.cuh"

namespace gtkv {

namespace {

// A warp per (page run, head). Keys and values: a lane per block of 16
// elements; the two elements of a pair may lie in two blocks, so a lane turns
// every pair that it meets and keeps its own half. Queries: a lane per pair, which alone reads and writes
// it, since they may be turned in place.
template <class T>
__global__ void __launch_bounds__(kAppendBlock) k_append4_any(DevPool p, Batch b, AppendArgs g, Rot t, bool by_row,
                                                              int64_t n_runs) {
  int bits = 0;
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kAppendBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kAppendBlock, bits);
  const int lane = threadIdx.x & 31;
  const int heads = g.Q + 2 * g.H;
  const int half = t.rd / 2, blocks = g.D / 16;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAppendBlock / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kAppendBlock / 32) + (threadIdx.x >> 5); w < n_runs * heads;
       w += warps) {
    const int64_t c = w / heads;
    const int head = static_cast<int>(w - c * heads);
    const PageRun run = page_run(p, b, c, by_row, bits);
    const bool is_q = head < g.Q;
    if (run.m == 0 || (run.page == 0 && !is_q)) continue;
    const int kv = head >= g.Q + g.H, h = is_q ? head : head - g.Q - kv * g.H;
    const T* src = static_cast<const T*>(is_q ? g.q : kv ? g.v : g.k) + static_cast<int64_t>(h) * g.D;
    const int64_t stride = is_q ? g.q_stride : kv ? g.v_stride : g.k_stride;
    if (is_q) {
      const int units = half + (g.D - t.rd);  // pairs, then single elements
      for (int i = 0; i < run.m; ++i) {
        const int64_t r = run.row + i, j = run.j + i;
        if (!positions_ok(t, b, r, j)) {
          bits |= KV_DEV_ERR_POSITION;
          continue;
        }
        const T* row = src + r * stride;
        T* out = static_cast<T*>(g.q_out) + (r * g.Q + h) * g.D;
        for (int u = lane; u < units; u += 32) {
          if (u >= half) {
            out[half + u] = row[half + u];
            continue;
          }
          const int e1 = t.interleaved ? 2 * u : u, e2 = t.interleaved ? 2 * u + 1 : u + half;
          float x1 = Elem<T>::get(row[e1]), x2 = Elem<T>::get(row[e2]);
          const int64_t at = position(t, b, r, j, u) * t.rd + u;
          turn(x1, x2, __ldg(t.cs + at), __ldg(t.cs + at + half));
          out[e1] = Elem<T>::put(x1);
          out[e2] = Elem<T>::put(x2);
        }
      }
      continue;
    }
    const int64_t tasks = static_cast<int64_t>(run.m) * blocks;
    for (int64_t k = lane; k < tasks; k += 32) {
      const int i = static_cast<int>(k / blocks), blk = static_cast<int>(k - static_cast<int64_t>(i) * blocks);
      const int64_t r = run.row + i, j = run.j + i;
      if (!positions_ok(t, b, r, j)) {
        bits |= KV_DEV_ERR_POSITION;
        continue;
      }
      const T* row = src + r * stride;
      float x[16];
      uint32_t top = 0;
      for (int z = 0; z < 16; ++z) {
        const int e = blk * 16 + z;
        float y;
        if (e < t.rd && kv == 0) {
          const int f = t.interleaved ? e >> 1 : e % half;
          const bool second = t.interleaved ? e & 1 : e >= half;
          float x1 = Elem<T>::get(row[t.interleaved ? 2 * f : f]);
          float x2 = Elem<T>::get(row[t.interleaved ? 2 * f + 1 : f + half]);
          const int64_t at = position(t, b, r, j, f) * t.rd + f;
          turn(x1, x2, __ldg(t.cs + at), __ldg(t.cs + at + half));
          y = second ? x2 : x1;
        } else {
          y = Elem<T>::get(row[e]);
        }
        x[z] = y;
        top = max(top, abs_bits(y));
      }
      const uint32_t byte = scale_byte(top);
      const float inv = scale_inverse(byte);
      uint8_t* to = pool_row<uint8_t>(p, g.layer, kv, run.page, run.off + i);
      *reinterpret_cast<uint2*>(to + h * (g.D / 2) + blk * 8) = make_uint2(encode8(x, inv), encode8(x + 8, inv));
      to[code_bytes(g.H, g.D) + h * blocks + blk] = static_cast<uint8_t>(byte);
    }
  }
  store_bits(p, bits);
}

// Gather: a block per page run, K and then V, a block of 16 elements a thread
// and step, whose values are 32 (or 64) consecutive bytes of the output: 8 bytes of codes and a
// scale in, whole sectors out.
template <class T>
__global__ void __launch_bounds__(kAppendBlock) k_gather4(DevPool p, Batch b, int32_t layer, int32_t H, int32_t D,
                                                          T* out_k, T* out_v, bool by_row) {
  int bits = 0;
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kAppendBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kAppendBlock, bits);
  const PageRun run = page_run(p, b, blockIdx.x, by_row, bits);
  store_bits(p, bits);
  if (run.m == 0) return;
  const int32_t nb = H * (D / 16);  // blocks of a row
  const int64_t row_bytes = p.vpr * 16;
  const int64_t n = static_cast<int64_t>(run.m) * nb;
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* src = pool_row<uint8_t>(p, layer, kv, run.page, run.off);
    T* dst = (kv ? out_v : out_k) + run.row * H * D;
    for (int64_t i = threadIdx.x; i < n; i += kAppendBlock) {
      uint2 w = make_uint2(0, 0);
      uint32_t s = 0;
      if (run.page != 0) {
        const int64_t row = i / nb, blk = i - row * nb;
        const uint8_t* at = src + row * row_bytes;
        w = __ldg(reinterpret_cast<const uint2*>(at + blk * 8));
        s = scale_pair(__ldg(at + nb * 8 + blk));
      }
      uint32_t y[8];
      codes8(w.x, reinterpret_cast<uint32_t(&)[4]>(y[0]));
      codes8(w.y, reinterpret_cast<uint32_t(&)[4]>(y[4]));
      T o[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 v = halves(mul_h2(y[k], s));
        o[2 * k] = Elem<T>::put(v.x);
        o[2 * k + 1] = Elem<T>::put(v.y);
      }
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(T)); ++k)
        reinterpret_cast<uint4*>(dst + i * 16)[k] = reinterpret_cast<const uint4*>(o)[k];
    }
  }
}

}  // namespace

template <class T>
cudaError_t launch_append4_any(const DevPool& p, const Batch& b, const AppendArgs& g, const Rot& t, bool by_row,
                               int64_t n_runs, cudaStream_t s) {
  int64_t n = (n_runs * (g.Q + 2 * g.H) + kAppendBlock / 32 - 1) / (kAppendBlock / 32);
  n = n < 1 ? 1 : n > 0x7fffffff ? 0x7fffffff : n;
  k_append4_any<T><<<static_cast<unsigned>(n), kAppendBlock, 0, s>>>(p, b, g, t, by_row, n_runs);
  return cudaGetLastError();
}

template cudaError_t launch_append4_any<__nv_bfloat16>(const DevPool&, const Batch&, const AppendArgs&, const Rot&, bool,
                                                       int64_t, cudaStream_t);
template cudaError_t launch_append4_any<__half>(const DevPool&, const Batch&, const AppendArgs&, const Rot&, bool, int64_t,
                                                cudaStream_t);
template cudaError_t launch_append4_any<float>(const DevPool&, const Batch&, const AppendArgs&, const Rot&, bool, int64_t,
                                               cudaStream_t);

cudaError_t launch_gather4(const DevPool& p, const Batch& b, int32_t layer, int32_t H, int32_t D, int32_t type,
                           void* out_k, void* out_v, cudaStream_t s) {
  const bool by_row = runs_by_row(b, p.ps);
  const int64_t n_runs = run_numbers(b, p.ps, by_row);
  if (n_runs > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&]<class T>(T* k, T* v) {
    k_gather4<T><<<static_cast<unsigned>(n_runs), kAppendBlock, 0, s>>>(p, b, layer, H, D, k, v, by_row);
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
