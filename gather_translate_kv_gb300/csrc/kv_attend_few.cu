// Attention of few rows a sequence: the launch. The kernel is kv_attend_few.cuh's, its instances are
// kv_attend_few_*.cu's.
#include "kv_attend_launch.h"

namespace gtkv {

namespace {

constexpr int kWhole = 24;    // steps up to which units are not cut where they fill the GPU; a third of it where they do not
constexpr int kMinShare = 4;  // steps of 16 keys below which a worker's share is not cut

int heads_of_worker(int32_t H) { return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1; }

}  // namespace

cudaError_t prepare_attend_few(int32_t D, Kind kind, bool p16, bool shared) {
  auto set = [&]<class C>() { return shared ? prepare_few<C, true>(D, p16) : prepare_few<C, false>(D, p16); };
  if (kind == Kind::kE2M1) return set.template operator()<CodeE2M1>();
  if (kind == Kind::kE4M3) return set.template operator()<CodeE4M3>();
  const cudaError_t e = set.template operator()<__half>();
  return e == cudaSuccess ? set.template operator()<__nv_bfloat16>() : e;
}

int64_t attend_few_workspace(int32_t D, int sm_count) {
  const int64_t warps = static_cast<int64_t>(sm_count) * kFewBlocksPerSM * kFewWarps;
  return split_record_bytes(warps) + warps * 2 * 16 * (D + 2) * 4;
}

cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, int32_t max_new,
                              void* workspace, int sm_count, Launch how, int32_t* nodes, Split* out, cudaStream_t s) {
  Split w{};
  w.hw = heads_of_worker(a.H);
  w.max_new = max_new;
  const int kw = kFewWarps / w.hw;
  // one tile of 8 columns when the sequences' rows of a KV head fit on average, else 16 (4 rows, 256 x 4096 tokens, on
  // one GPU: 686 us with 8 columns, 803 with 16)
  const int nt = b.n_rows * a.G <= 8 * spans_of(b) ? 1 : 2;
  // steps of one unit at most, and of all units
  int64_t most = static_cast<int64_t>(b.max_pages) * p.ps / 16 + 1;
  if (a.window) {
    const int64_t seen = (static_cast<int64_t>(a.window) + 16) / 16 + 2 + (a.sinks + 15) / 16;
    most = seen < most ? seen : most;
  }
  const int64_t tiles = (b.n_rows * a.G) / (8 * nt) + b.n_seqs;  // row tiles of all sequences
  const int row_bytes = kind == Kind::kE2M1 ? a.D / 2 : kind == Kind::kE4M3 ? a.D : 2 * a.D;
  int64_t cap = static_cast<int64_t>(sm_count) * few_blocks(row_bytes, nt, kind == Kind::kE2M1) * kw;
  // units that are short anyway are never cut, and then there is nothing to join: 512 sequences of 300 tokens (8-bit,
  // D = 64) 52 us against 63 cut, 4 of 128 tokens 15.0 against 15.2
  w.whole = most <= (tiles * (a.H / w.hw) >= cap ? kWhole : kWhole / 3);
  const int64_t all = (w.whole ? 1 : most + kFewUnitCost) * tiles * (a.H / w.hw);
  cap = cap < kMaxWorkers ? cap : kMaxWorkers;
  // a prefix of few rows is cut into many segments, which then meet level by level: 4 sequences in 2 groups behind 8192
  // tokens (in wide tables) 43 us with 4 steps a segment and with 8, 8-bit 51 / 45, 4-bit 49 / 45; with more groups the
  // same
  w.min_share = w.whole ? 1 : a.state ? 2 * kMinShare : kMinShare;
  int64_t workers = (all + w.min_share - 1) / w.min_share;
  workers = workers > cap ? cap : workers;
  w.blocks = static_cast<int>((workers + kw - 1) / kw);
  if (w.blocks * kw > kMaxWorkers) w.blocks = kMaxWorkers / kw;
  w.n_workers = w.blocks * kw;
  // a block with an SM to itself may have the longer ring (one sequence of 203 tokens: 15.1 us against 15.5); where
  // blocks share an SM it costs residency (8 sequences of 2000 tokens: 39 us against 28)
  w.deep = w.blocks <= sm_count;
  w.rec = static_cast<SplitRecord*>(workspace);
  const int64_t warps = static_cast<int64_t>(sm_count) * kFewBlocksPerSM * kFewWarps;
  w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + split_record_bytes(warps));
  w.nq = 8 * nt;
  w.lift = 0.0f;  // the partial results' references are below it already
  w.q_wide = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_stride % 8 == 0;
  w.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  w.first = how == Launch::kFirst;
  w.nodes = nodes;
  *out = w;
  const bool after = how != Launch::kPlain;
  auto go = [&]<class C>() {
    return b.seqs ? launch_few<C, true>(p, b, a, w, nt, after, s) : launch_few<C, false>(p, b, a, w, nt, after, s);
  };
  if (kind == Kind::kE2M1) return go.template operator()<CodeE2M1>();
  if (kind == Kind::kE4M3) return go.template operator()<CodeE4M3>();
  return a.type == KV_TYPE_BF16 ? go.template operator()<__nv_bfloat16>() : go.template operator()<__half>();
}

}  // namespace gtkv
