// The attention kernels behind launch_attend: few rows a sequence
// (kv_attend_few.cuh), tiles of rows (kv_attend_tile.cuh) and the join of units
// that they cut (kv_attend.cu), head sizes 64 and 128.
#pragma once

#include "kv_attn_launch.h"

namespace gtkv {

constexpr int kMaxWorkers = 2048;

struct CodeE4M3;
struct CodeE2M1;

// Few rows a sequence.
constexpr int kFewWarps = 4;
constexpr int kFewBlock = 32 * kFewWarps;
constexpr int kFewBlocksPerSM = 4;  // at most
constexpr int kFewUnitCost = 2;     // steps' worth of a unit's queries and output
// Resident blocks: shared memory for 256-byte rows, registers for 16 columns allow three, or two without spills
// where codes of 4 bits are turned.
constexpr int few_blocks(int row, int nt, bool e2m1) { return e2m1 && nt > 1 ? 2 : row >= 256 || nt > 1 ? 3 : kFewBlocksPerSM; }

// Tiles of rows.
constexpr int kTileRows = 256;    // rows of a unit
constexpr int kTileKeys = 128;    // keys of a step
constexpr int kTileUnitCost = 3;  // steps' worth of a unit's queries and output

// What a worker leaves behind for the join: the unit that its last segment
// left unfinished, s < 0 for none, and the last worker that continues it.
struct SplitRecord {
  int32_t s;       // sequence
  int32_t a;       // position of its first new token
  int32_t f0, nf;  // rows [f0, f0 + nf) of the sequence
  int32_t head;    // KV head, or group of heads
  int32_t last;    // worker
  int64_t row0;    // row of the tensors that f = 0 belongs to
};

// Where a call's partial results are, and how its units are shaped.
struct Split {
  SplitRecord* rec;   // one per worker
  float* part;        // [worker][head of the worker][slot][nq * (D + 2)]: sums, references, denominators
  int32_t n_workers;  // 0: the kernel takes no part in the call
  int32_t hw;         // KV heads of a worker
  int32_t nq;         // rows of a unit
  int32_t min_share;  // steps
  int32_t min_new, max_new;  // new tokens of the sequences that the kernel takes
  int32_t blocks;
  int32_t q_wide;     // query rows start on 16 bytes
  int32_t out_wide;   // out is aligned for the kernel's widest stores
  int32_t deep;       // the longer ring
  int32_t whole;      // units are not cut: nothing to join
  int32_t first;      // the sequences come from the kernel before this one
  int32_t* nodes;     // shared prefixes: where the segments of a unit meet (TreePlace), [worker][warps], zeros
  float lift;         // log2 of the weights' lift
};

inline int64_t split_record_bytes(int64_t workers) {
  return (workers * static_cast<int64_t>(sizeof(SplitRecord)) + 255) / 256 * 256;
}

// Shared-memory limits, on the current device, of the kernels for one kind of pool (p16: its page size is a multiple
// of 16), the plain ones or those for shared prefixes.
cudaError_t prepare_attend_few(int32_t D, Kind kind, bool p16, bool shared);
cudaError_t prepare_attend_tile(int32_t D, Kind kind, bool p16, bool shared);
// Joining nodes of a kernel, for shared prefixes.
inline int64_t few_nodes(int sm_count) { return static_cast<int64_t>(sm_count) * kFewBlocksPerSM * kFewWarps; }
inline int64_t tile_nodes(int sm_count) { return static_cast<int64_t>(sm_count) * 8; }
int64_t attend_few_workspace(int32_t D, int sm_count);
int64_t attend_tile_workspace(int32_t D, int sm_count);
// How a kernel follows the one before it: at its end, over its tail, or over its tail but reading its result first.
enum class Launch { kPlain, kAfter, kFirst };
// Sequences of at most max_new, and of at least min_new, new tokens; *w says
// what is left to join.
cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, int32_t max_new,
                              void* workspace, int sm_count, Launch how, int32_t* nodes, Split* w, cudaStream_t s);
cudaError_t launch_attend_tile(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, int32_t min_new,
                               void* workspace, int sm_count, Launch how, int32_t* nodes, Split* w, cudaStream_t s);
// The instances for a cache's element type (kv_attend_few_*.cu, kv_attend_tile_*.cu).
template <class C, bool SHARED>
cudaError_t launch_few(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, int nt, bool after,
                       cudaStream_t s);
template <class C, bool SHARED>
cudaError_t prepare_few(int32_t D, bool p16);
template <class C, bool SHARED>
cudaError_t launch_tile(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, bool after, cudaStream_t s);
template <class C, bool SHARED>
cudaError_t prepare_tile(int32_t D, bool p16);
// Both, each for the sequences on its side of few_rows_of, and the join (kv_attend.cu).
cudaError_t launch_tiles(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& g,
                         void* workspace, int sm_count, cudaStream_t s);
// Rows a KV head up to which a sequence is the few-rows kernel's.
inline int32_t few_rows_of(Kind kind) { return kind == Kind::kElements ? 16 : 32; }
inline bool has_tiles(int32_t D) { return D == 64 || D == 128; }
cudaError_t launch_attend_join(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Split& few,
                               const Split& tile, const Groups& g, int sm_count, cudaStream_t s);

}  // namespace gtkv
