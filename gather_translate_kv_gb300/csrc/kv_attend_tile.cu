// Attention of many rows a sequence: the launch, and the kernel (kv_attend_tile.cuh) for caches of 16 and 8 bits.
#include "kv_attend_tile.cuh"

namespace gtkv {

namespace {

constexpr int kMinShare = 2;  // steps of 128 keys below which a block's share is not cut

}  // namespace

cudaError_t prepare_attend_tile(int32_t D, Kind kind, bool p16) {
  cudaError_t e;
  if (kind == Kind::kE2M1) return prepare_tile4(D);
  if (kind == Kind::kElements) {
    e = prepare_one<__half, false, true>(D);
    return e == cudaSuccess ? prepare_one<__nv_bfloat16, false, true>(D) : e;
  }
  e = p16 ? prepare_one<CodeE4M3, true, false>(D) : prepare_one<CodeE4M3, false, false>(D);
  if (e != cudaSuccess) return e;
  return p16 ? prepare_one<CodeE4M3, true, true>(D) : prepare_one<CodeE4M3, false, true>(D);
}

int64_t attend_tile_workspace(int32_t D, int sm_count) {
  return split_record_bytes(sm_count) + static_cast<int64_t>(sm_count) * 2 * kRows * (D + 2) * 4;
}

cudaError_t launch_attend_tile(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, int32_t min_new,
                               void* workspace, int sm_count, Launch how, Split* out, cudaStream_t s) {
  Split w{};
  w.hw = 1;
  w.nq = kRows;
  w.min_new = min_new;
  w.min_share = kMinShare;
  const int64_t steps = static_cast<int64_t>(b.max_pages) * p.ps / kKeys + 1 + kUnitCost;
  const int64_t tiles = b.n_rows * a.G / kRows + (b.n_rows < b.n_seqs ? b.n_rows : b.n_seqs);
  const int64_t blocks = (steps * tiles * a.H + kMinShare - 1) / kMinShare;
  w.blocks = static_cast<int>(blocks < sm_count ? blocks : sm_count);
  w.n_workers = w.blocks;
  w.rec = static_cast<SplitRecord*>(workspace);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + split_record_bytes(sm_count));
  w.q_wide = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_stride % 8 == 0;
  w.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
  w.lift = kind == Kind::kElements && a.type == KV_TYPE_BF16 ? 0.0f : 6.0f;
  w.first = how == Launch::kFirst;
  *out = w;
  const bool after = how != Launch::kPlain;
  auto go = [&]<class C, bool P16, bool TWO>() { return launch_one<C, P16, TWO>(p, b, a, w, after, s); };
  const bool bf16 = a.type == KV_TYPE_BF16;
  if (kind == Kind::kE2M1) return launch_tile4(p, b, a, w, after, s);
  if (kind == Kind::kElements)
    return bf16 ? go.template operator()<__nv_bfloat16, false, true>() : go.template operator()<__half, false, true>();
  if (p.ps % 16 == 0)
    return bf16 ? go.template operator()<CodeE4M3, true, false>() : go.template operator()<CodeE4M3, true, true>();
  return bf16 ? go.template operator()<CodeE4M3, false, false>() : go.template operator()<CodeE4M3, false, true>();
}

}  // namespace gtkv
