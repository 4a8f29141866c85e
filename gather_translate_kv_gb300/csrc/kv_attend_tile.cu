// Attention of many rows a sequence: the launch. The kernel is kv_attend_tile.cuh's, its instances are
// kv_attend_tile_*.cu's.
#include "kv_attend_launch.h"

namespace gtkv {

namespace {

constexpr int kMinShare = 2;  // steps of 128 keys below which a block's share is not cut

}  // namespace

cudaError_t prepare_attend_tile(int32_t D, Kind kind, bool p16, bool shared) {
  auto set = [&]<class C>() { return shared ? prepare_tile<C, true>(D, p16) : prepare_tile<C, false>(D, p16); };
  if (kind == Kind::kE2M1) return set.template operator()<CodeE2M1>();
  if (kind == Kind::kE4M3) return set.template operator()<CodeE4M3>();
  const cudaError_t e = set.template operator()<__half>();
  return e == cudaSuccess ? set.template operator()<__nv_bfloat16>() : e;
}

int64_t attend_tile_workspace(int32_t D, int sm_count) {
  return split_record_bytes(sm_count) + static_cast<int64_t>(sm_count) * 2 * kTileRows * (D + 2) * 4;
}

cudaError_t launch_attend_tile(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, int32_t min_new,
                               void* workspace, int sm_count, Launch how, int32_t* nodes, Split* out, cudaStream_t s) {
  Split w{};
  w.hw = 1;
  w.nq = kTileRows;
  w.min_new = min_new;
  w.min_share = kMinShare;
  const int64_t steps = static_cast<int64_t>(b.max_pages) * p.ps / kTileKeys + 1 + kTileUnitCost;
  const int64_t tiles = b.n_rows * a.G / kTileRows + (b.n_rows < b.n_seqs ? b.n_rows : b.n_seqs);
  const int64_t blocks = (steps * tiles * a.H + kMinShare - 1) / kMinShare;
  w.blocks = static_cast<int>(blocks < sm_count ? blocks : sm_count);
  w.n_workers = w.blocks;
  w.rec = static_cast<SplitRecord*>(workspace);
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + split_record_bytes(sm_count));
  w.q_wide = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_stride % 8 == 0;
  w.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
  w.lift = kind == Kind::kElements && a.type == KV_TYPE_BF16 ? 0.0f : 6.0f;
  w.first = how == Launch::kFirst;
  w.nodes = nodes;
  *out = w;
  const bool after = how != Launch::kPlain;
  auto go = [&]<class C>() {
    return b.seqs ? launch_tile<C, true>(p, b, a, w, after, s) : launch_tile<C, false>(p, b, a, w, after, s);
  };
  if (kind == Kind::kE2M1) return go.template operator()<CodeE2M1>();
  if (kind == Kind::kE4M3) return go.template operator()<CodeE4M3>();
  return a.type == KV_TYPE_BF16 ? go.template operator()<__nv_bfloat16>() : go.template operator()<__half>();
}

}  // namespace gtkv
