// 4-bit pools (KV_FORMAT_E2M1): append for any head size, rotary_dim, alignment
// or stride, and the gather of the values. The append of ordinary shapes is
// k_append's (kv_append.cu).
#include <type_traits>

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

__device__ __forceinline__ void store32(void* to, const uint32_t* y, bool wide) {
  if (!wide) {  // the output starts on 16 bytes alone
    __stcs(static_cast<uint4*>(to), make_uint4(y[0], y[1], y[2], y[3]));
    __stcs(static_cast<uint4*>(to) + 1, make_uint4(y[4], y[5], y[6], y[7]));
    return;
  }
  asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
               "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}

// Gather: a block per page run, K and V as one list, N blocks of 16 elements a thread and item: 8 N bytes of codes and
// N scales in, whole sectors of 32 bytes out, kGatherItems items of a thread in flight. N is 2 where rows hold an even
// number of blocks. Measured: 232 us for 1.54 GB of whole sequences (98 % of the copy rate; items of 8 bytes of codes
// and 16-byte stores 276), 33 us for 172 MB of 128-token windows, whose blocks wait for their lookups. Items and
// resident blocks: 2 / 5 as good, 4 / 5 247 us, 8 / 3 236.
constexpr int kGatherItems = 4;
constexpr int kGatherBlocks = 4;
template <class T, int N>
__global__ void __launch_bounds__(kAppendBlock, kGatherBlocks) k_gather4(DevPool p, Batch b, int32_t layer, int32_t H, int32_t D,
                                                             T* out_k, T* out_v, bool by_row, bool wide) {
  int bits = 0;
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kAppendBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kAppendBlock, bits);
  const PageRun run = page_run(p, b, blockIdx.x, by_row, bits);
  store_bits(p, bits);
  if (run.m == 0) return;
  const int32_t ni = H * (D / 16) / N;  // items of a row
  const int64_t row_bytes = p.vpr * 16;
  const uint8_t* src = pool_row<uint8_t>(p, layer, 0, run.page, run.off);
  const int64_t v_bytes = p.ps * row_bytes;
  const int64_t out0 = run.row * H * D;
  // the thread's items: item `col` of row `row`, rows of K and then of V
  const int32_t rows = 2 * run.m, step_row = kAppendBlock / ni, step_col = kAppendBlock - step_row * ni;
  int32_t row = threadIdx.x / ni, col = threadIdx.x - row * ni;
  while (row < rows) {
    uint32_t w[kGatherItems][2 * N], s[kGatherItems];
    int32_t rows_of[kGatherItems], cols[kGatherItems];
#pragma unroll
    for (int u = 0; u < kGatherItems; ++u) {
      rows_of[u] = row;
      cols[u] = col;
#pragma unroll
      for (int k = 0; k < 2 * N; ++k) w[u][k] = 0;
      s[u] = 0;
      if (row < rows && run.page != 0) {
        const uint8_t* from = src + (row < run.m ? row * row_bytes : v_bytes + (row - run.m) * row_bytes);
        if constexpr (N == 2) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(from) + col);
          w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
          s[u] = __ldg(reinterpret_cast<const uint16_t*>(from + ni * 16) + col);
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(from) + col);
          w[u][0] = v.x, w[u][1] = v.y;
          s[u] = __ldg(from + ni * 8 + col);
        }
      }
      row += step_row;
      col += step_col;
      if (col >= ni) {
        col -= ni;
        ++row;
      }
    }
#pragma unroll
    for (int u = 0; u < kGatherItems; ++u) {
      if (rows_of[u] >= rows) break;
      const bool v = rows_of[u] >= run.m;
      T* dst = (v ? out_v : out_k) + out0 + (static_cast<int64_t>(v ? rows_of[u] - run.m : rows_of[u]) * ni + cols[u]) * (16 * N);
#pragma unroll
      for (int blk = 0; blk < N; ++blk) {
        const uint32_t sc = scale_pair(s[u] >> 8 * blk & 255);
        uint32_t y[8];
        codes8(w[u][2 * blk], reinterpret_cast<uint32_t(&)[4]>(y[0]));
        codes8(w[u][2 * blk + 1], reinterpret_cast<uint32_t(&)[4]>(y[4]));
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = mul_h2(y[k], sc);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t z[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 a = halves(y[4 * half + k]);
              z[2 * k] = __float_as_uint(a.x), z[2 * k + 1] = __float_as_uint(a.y);
            }
            store32(dst + 16 * blk + 8 * half, z, wide);
          }
        } else {
          if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 a = halves(y[k]);
              const __nv_bfloat162 z = __floats2bfloat162_rn(a.x, a.y);
              y[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          store32(dst + 16 * blk, y, wide);
        }
      }
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
  const bool wide = ((reinterpret_cast<uintptr_t>(out_k) | reinterpret_cast<uintptr_t>(out_v)) & 31u) == 0;
  auto go = [&]<class T>(T* k, T* v) {
    auto kernel = H * D % 32 == 0 ? k_gather4<T, 2> : k_gather4<T, 1>;
    kernel<<<static_cast<unsigned>(n_runs), kAppendBlock, 0, s>>>(p, b, layer, H, D, k, v, by_row, wide);
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
