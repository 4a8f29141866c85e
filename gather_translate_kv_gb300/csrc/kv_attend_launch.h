// The attention kernels behind launch_attend: few rows a sequence
// (kv_attend_few.cu), tiles of rows (kv_attend_tile.cu) and the join of units
// that they cut (kv_attend.cu), head sizes 64 and 128.
#pragma once

#include "kv_attn_launch.h"

namespace gtkv {

constexpr int kMaxWorkers = 2048;

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
  float lift;         // log2 of the weights' lift
};

inline int64_t split_record_bytes(int64_t workers) {
  return (workers * static_cast<int64_t>(sizeof(SplitRecord)) + 255) / 256 * 256;
}

// Shared-memory limits, on the current device, of the kernels for one kind of pool (p16: its page size is a multiple
// of 16).
cudaError_t prepare_attend_few(int32_t D, bool e4m3, bool p16);
cudaError_t prepare_attend_tile(int32_t D, bool e4m3, bool p16);
int64_t attend_few_workspace(int32_t D, int sm_count);
int64_t attend_tile_workspace(int32_t D, int sm_count);
// Sequences of at most max_new, and of at least min_new, new tokens; *w says
// what is left to join. `after` marks a launch that may overlap the one before it.
cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t max_new,
                              void* workspace, int sm_count, Split* w, cudaStream_t s);
cudaError_t launch_attend_tile(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t min_new,
                               void* workspace, int sm_count, bool after, Split* w, cudaStream_t s);

}  // namespace gtkv
