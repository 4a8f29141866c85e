// Attention over the pages: which kernel takes a call, and the row-by-row form.
#include "kv_attend.cuh"
#include "kv_attend_launch.h"

namespace gtkv {

namespace {

constexpr int kRowBlock = 128;

// A warp per (row, query head).
template <class C>
__global__ void __launch_bounds__(kRowBlock) k_attend_rows(DevPool p, Batch b, AttendArgs a) {
  int bits = 0;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowBlock / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowBlock / 32) + (threadIdx.x >> 5); w < b.n_rows * a.Q;
       w += warps) {
    const int64_t r = w / a.Q;
    const int32_t s = warp_search(b.n_seqs, r, [&](int32_t i) { return __ldg(b.cu + i); });
    const Seq q = seq_of(p, b, s, bits);
    if (r < q.row0 || r - q.row0 >= q.n) continue;
    attend_row<C>(p, b, a, s, q.a + static_cast<int32_t>(r - q.row0), r, static_cast<int32_t>(w - r * a.Q), &bits);
  }
  store_bits(p, bits);
}

cudaError_t launch_rows(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, cudaStream_t s) {
  const int64_t n = (b.n_rows * a.Q + kRowBlock / 32 - 1) / (kRowBlock / 32);
  const unsigned grid = static_cast<unsigned>(n > 0x7fffffff ? 0x7fffffff : n);
  if (e4m3)
    k_attend_rows<CodeE4M3><<<grid, kRowBlock, 0, s>>>(p, b, a);
  else if (a.type == KV_TYPE_BF16)
    k_attend_rows<__nv_bfloat16><<<grid, kRowBlock, 0, s>>>(p, b, a);
  else
    k_attend_rows<__half><<<grid, kRowBlock, 0, s>>>(p, b, a);
  return cudaGetLastError();
}

bool has_tiles(int32_t D) { return D == 64 || D == 128; }

}  // namespace

cudaError_t prepare_attend() {
  const cudaError_t e = prepare_attend_few();
  return e == cudaSuccess ? prepare_attend_tile() : e;
}

int64_t attend_workspace_bytes(int32_t H, int32_t, int32_t D, int32_t, int64_t, int sm_count) {
  if (!has_tiles(D)) return 16;
  const int64_t few = attend_few_workspace(H, D, sm_count), tile = attend_tile_workspace(D, sm_count);
  return few > tile ? few : tile;  // the two run one after the other
}

cudaError_t launch_attend(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, void* workspace,
                          int sm_count, cudaStream_t s) {
  if (!has_tiles(a.D)) return launch_rows(p, b, a, e4m3, s);
  const int32_t few = 16 / a.G;  // new tokens up to which a sequence's rows of a KV head are few
  if (few > 0) {
    const cudaError_t e = launch_attend_few(p, b, a, e4m3, few, workspace, sm_count, s);
    if (e != cudaSuccess || b.n_rows <= few) return e;
  }
  return launch_attend_tile(p, b, a, e4m3, few + 1, workspace, sm_count, s);
}

}  // namespace gtkv
