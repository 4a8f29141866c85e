// Attention over the pages: which kernels take a call, the join of cut units,
// and the row-by-row form.
#include "kv_attend_split.cuh"

namespace gtkv {

namespace {

constexpr int kRowBlock = 128;

// A warp per (row, query head).
template <class C>
__global__ void __launch_bounds__(kRowBlock) k_attend_rows(DevPool p, Batch b, AttendArgs a) {
  int bits = 0;
  check_seqs(p, b, static_cast<int64_t>(blockIdx.x) * kRowBlock + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kRowBlock, bits);
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

cudaError_t launch_rows(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, cudaStream_t s) {
  const int64_t n = (b.n_rows * a.Q + kRowBlock / 32 - 1) / (kRowBlock / 32);
  const unsigned grid = static_cast<unsigned>(n > 0x7fffffff ? 0x7fffffff : n);
  if (kind == Kind::kE4M3)
    k_attend_rows<CodeE4M3><<<grid, kRowBlock, 0, s>>>(p, b, a);
  else if (kind == Kind::kE2M1)
    k_attend_rows<CodeE2M1><<<grid, kRowBlock, 0, s>>>(p, b, a);
  else if (a.type == KV_TYPE_BF16)
    k_attend_rows<__nv_bfloat16><<<grid, kRowBlock, 0, s>>>(p, b, a);
  else
    k_attend_rows<__half><<<grid, kRowBlock, 0, s>>>(p, b, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_attend(const kv_pool_desc& d, bool shared) {
  if (d.latent_only || d.itemsize > 2 || !has_tiles(d.head_dim)) return cudaSuccess;
  const Kind kind = kind_of(d);
  const bool p16 = d.page_size % 16 == 0;
  const cudaError_t e = prepare_attend_few(d.head_dim, kind, p16, shared);
  return e == cudaSuccess ? prepare_attend_tile(d.head_dim, kind, p16, shared) : e;
}

namespace {

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

template <class C>
cudaError_t launch_join(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& few, const Split& tile,
                        const Groups& g, int sm_count, cudaStream_t s) {
  const int workers = few.n_workers > tile.n_workers ? few.n_workers : tile.n_workers;
  const int rows = workers * (few.n_workers ? few.hw * few.nq : tile.nq);
  const dim3 grid(rows / (kJoinBlock / 32) < 4 * sm_count ? (rows + kJoinBlock / 32 - 1) / (kJoinBlock / 32) : 4 * sm_count);
  return launch_overlapped(a.D == 64 ? k_attend_join<C, 64> : k_attend_join<C, 128>, grid, kJoinBlock, 0, s, p, b, a,
                           few, tile, g);
}

// Groups of a call that has nothing to join. It outlasts the kernel before it, over whose tail it runs.
__global__ void __launch_bounds__(kJoinBlock) k_check_groups(DevPool p, Batch b, Groups g) {
  store_bits(p, groups_bad(b, g, threadIdx.x, kJoinBlock) ? KV_DEV_ERR_TABLE : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

cudaError_t launch_check(const DevPool& p, const Batch& b, const Groups& g, cudaStream_t s) {
  return g.first ? launch_overlapped(k_check_groups, dim3(1), kJoinBlock, 0, s, p, b, g) : cudaSuccess;
}

}  // namespace

cudaError_t launch_attend_join(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Split& few,
                               const Split& tile, const Groups& g, int sm_count, cudaStream_t s) {
  if (kind == Kind::kE2M1) return launch_join<CodeE2M1>(p, b, a, few, tile, g, sm_count, s);
  if (kind == Kind::kE4M3) return launch_join<CodeE4M3>(p, b, a, few, tile, g, sm_count, s);
  return a.type == KV_TYPE_BF16 ? launch_join<__nv_bfloat16>(p, b, a, few, tile, g, sm_count, s)
                                : launch_join<__half>(p, b, a, few, tile, g, sm_count, s);
}

int64_t attend_workspace_bytes(int32_t, int32_t, int32_t D, int32_t, int64_t, int sm_count) {
  if (!has_tiles(D)) return 16;
  return align256(attend_few_workspace(D, sm_count)) + attend_tile_workspace(D, sm_count);
}

// Which kernels: the few-rows kernel alone when the sequences' rows of a KV head number at most 16 (8-bit and 4-bit
// caches: 32) on average (decode steps and drafts; a longer sequence among them takes several row tiles there), else
// both, each taking the sequences on its side of that. Lengths are known on the device alone, so the rule goes by
// averages. 32 sequences of 4000 tokens, 4 query heads a KV head, D = 128, few-rows against tile kernel, us: 16-bit 110
// / 147 at 8 rows, 137 / 150 at 16, 195 / 151 at 20; 8-bit 83 / 154 at 16, 126 / 159 at 32, 182 / 160 at 40 (fp16
// output 91 / 189, 143 / 195, 205 / 195); 4-bit 75 / 158, 121 / 162, 169 / 162 (fp16 output 82 / 187, 138 / 189, 195 /
// 189).
cudaError_t launch_tiles(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& g,
                         void* workspace, int sm_count, cudaStream_t s) {
  const int32_t few_rows = few_rows_of(kind);
  const bool only_few = b.n_rows * a.G <= few_rows * static_cast<int64_t>(b.n_seqs);
  const int32_t limit = only_few ? 0x7fffffff : few_rows / a.G;
  Split few{}, tile{};
  cudaError_t e = cudaSuccess;
  if (limit > 0) e = launch_attend_few(p, b, a, kind, limit, workspace, sm_count, Launch::kPlain, nullptr, &few, s);
  if (e == cudaSuccess && !only_few)
    e = launch_attend_tile(p, b, a, kind, limit + 1,
                           static_cast<uint8_t*>(workspace) + align256(attend_few_workspace(a.D, sm_count)), sm_count,
                           limit > 0 ? Launch::kAfter : Launch::kPlain, nullptr, &tile, s);
  if (e != cudaSuccess) return e;
  if (few.whole) few.n_workers = 0;
  if (few.n_workers == 0 && tile.n_workers == 0) return launch_check(p, b, g, s);
  return launch_attend_join(p, b, a, kind, few, tile, g, sm_count, s);
}

cudaError_t launch_attend(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& g,
                          void* workspace, int sm_count, cudaStream_t s) {
  if (has_tiles(a.D)) return launch_tiles(p, b, a, kind, g, workspace, sm_count, s);
  const cudaError_t e = launch_rows(p, b, a, kind, s);
  return e == cudaSuccess ? launch_check(p, b, g, s) : e;
}

}  // namespace gtkv
