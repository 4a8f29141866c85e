// Attention of groups of sequences that share their first tokens.
//
// The rows of a group see its prefix alike, so the prefix is attended to
// by all of them as if they were rows of one sequence: its keys and values are
// read once for a tile of the group's rows, and where it has many rows they fill the tiles of the
// tensor cores (k_attend_tile) instead of 4 of their 128 rows. What a row has
// summed up - sum of weighted values, reference, denominator - goes to the workspace
// in 32 bits. Then every sequence attends to its own tokens (k_attend_few), takes what its rows have
// from the prefix under a common reference,
//   out = (o 2^(m - M) + o' 2^(m' - M)) / (l 2^(m - M) + l' 2^(m' - M)),   M = max(m, m'),
// and writes the result. Each launch starts over the tail of the one before it.
#include "kv_attend_launch.h"

namespace gtkv {

namespace {

constexpr int kGroupBlock = 256;
constexpr int kZeroBlocks = 24;  // at least, so that the nodes are zeros at once
// Rows a KV head and sequence, on average, past which a sequence fills tiles by itself (kv_attend_layer / shared, us,
// 32 sequences in 4 groups behind 8192 tokens, with 100 own tokens before the new ones, bf16: 276 / 132 at 64 rows, 284
// / 205 at 128, 325 / 291 at 192, 336 / 373 at 256; 8-bit 282 / 139, 289 / 209, 312 / 292, 318 / 377; 4-bit 257 / 126,
// 267 / 201, 302 / 282, 313 / 363). Own tokens are read again for every 16 rows, so with more of them the crossing
// comes sooner: 1024 of them, bf16, 299 / 202 at 64 rows, 303 / 338 at 128; 4096 behind 4096 shared ones 270 / 452 and
// 275 / 809. Lengths are known on the device alone.
constexpr int kOwnTiles = 128;

// Looks at all metadata once. own: the sequences, checked; shared: at the index of a group's first sequence with
// rows the group as one sequence, whose rows all stand at its prefix' last token, else no rows; from: where the
// sequences' own tokens begin. A prefix is cut to whole steps of 16 keys and ends before any
// member's new tokens; it is shared by two sequences at least. The runs of rows that stand for groups are disjoint,
// whatever cu holds: each lies in its group's part of the rows, and those parts follow one another.
__global__ void __launch_bounds__(kGroupBlock) k_share_groups(DevPool p, Batch b, Groups gr,
                                                              const int32_t* __restrict__ prefix_len, int32_t G, Seq* own,
                                                              Seq* shared, int32_t* from, int32_t* nodes, int32_t n_nodes) {
  __shared__ int64_t row0[kGroupBlock / 32], row1[kGroupBlock / 32];
  __shared__ int32_t start[kGroupBlock / 32], first[kGroupBlock / 32], count[kGroupBlock / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bits = 0;
  for (int32_t i = blockIdx.x * kGroupBlock + tid; i < n_nodes; i += gridDim.x * kGroupBlock) nodes[i] = 0;
  if (__syncthreads_or(groups_bad(b, gr, tid, kGroupBlock))) {  // nothing is shared
    for (int64_t s = blockIdx.x * static_cast<int64_t>(kGroupBlock) + tid; s < b.n_seqs;
         s += static_cast<int64_t>(gridDim.x) * kGroupBlock) {
      own[s] = seq_of(p, b, static_cast<int32_t>(s), bits);
      shared[s] = Seq{0, 0, 0};
      from[s] = 0;
    }
    store_bits(p, bits | KV_DEV_ERR_TABLE);
    return;
  }
  // Do some group's rows begin before those of the group before it? (A sequence is inconsistent then.)
  bool back = false;
  for (int32_t i = tid; i < gr.n; i += kGroupBlock)
    back = back || __ldg(b.cu + __ldg(gr.first + i + 1)) < __ldg(b.cu + __ldg(gr.first + i));
  for (int32_t g = blockIdx.x; g < gr.n; g += gridDim.x) {
    const int32_t s0 = __ldg(gr.first + g), s1 = __ldg(gr.first + g + 1);
    const int64_t c0 = __ldg(b.cu + s0), c1 = __ldg(b.cu + s1);
    int64_t r0 = INT64_MAX, r1 = 0;
    int32_t a = INT32_MAX, s_first = INT32_MAX, n = 0;
    for (int32_t s = s0 + tid; s < s1; s += kGroupBlock) {
      const Seq q = seq_of(p, b, s, bits);
      own[s] = q;
      if (q.n == 0) continue;
      r0 = q.row0 < r0 ? q.row0 : r0;
      r1 = q.row0 + q.n > r1 ? q.row0 + q.n : r1;
      a = min(a, q.a);
      s_first = min(s_first, s);
      ++n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const int64_t x0 = __shfl_xor_sync(kFull, r0, o), x1 = __shfl_xor_sync(kFull, r1, o);
      r0 = x0 < r0 ? x0 : r0;
      r1 = x1 > r1 ? x1 : r1;
    }
    a = __reduce_min_sync(kFull, a);
    s_first = __reduce_min_sync(kFull, s_first);
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) row0[warp] = r0, row1[warp] = r1, start[warp] = a, first[warp] = s_first, count[warp] = n;
    const bool apart = !__syncthreads_or(back);
    r0 = INT64_MAX, r1 = 0, a = INT32_MAX, s_first = INT32_MAX, n = 0;
#pragma unroll
    for (int w = 0; w < kGroupBlock / 32; ++w) {
      r0 = row0[w] < r0 ? row0[w] : r0;
      r1 = row1[w] > r1 ? row1[w] : r1;
      a = min(a, start[w]);
      s_first = min(s_first, first[w]);
      n += count[w];
    }
    __syncthreads();
    int32_t prefix = min(__ldg(prefix_len + g), a) & ~15;
    if (n < 2 || prefix < 16 || (r1 - r0) * G > INT32_MAX - 1024) prefix = 0;
    // the run of the group's rows has to lie in its part of the rows (it does where cu does not decrease)
    if (!apart || r0 < c0 || r1 > c1) prefix = 0;
    for (int32_t s = s0 + tid; s < s1; s += kGroupBlock) {
      from[s] = prefix;
      shared[s] = prefix != 0 && s == s_first ? Seq{r0, prefix - 1, static_cast<int32_t>(r1 - r0)} : Seq{0, 0, 0};
    }
  }
  store_bits(p, bits);
}

constexpr int64_t kAlign = 256;
int64_t aligned(int64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

struct Workspace {
  int64_t own, shared, from, nodes, tiles, few, state, bytes;
};

Workspace workspace_of(int32_t Q, int32_t D, int32_t n_seqs, int64_t n_rows, int sm_count) {
  Workspace w{};
  auto take = [&](int64_t n) {
    const int64_t at = w.bytes;
    w.bytes += aligned(n);
    return at;
  };
  w.tiles = take(attend_workspace_bytes(0, Q, D, n_seqs, n_rows, sm_count));
  if (!has_tiles(D)) return w;
  w.own = take(n_seqs * static_cast<int64_t>(sizeof(Seq)));
  w.shared = take(n_seqs * static_cast<int64_t>(sizeof(Seq)));
  w.from = take(n_seqs * static_cast<int64_t>(sizeof(int32_t)));
  w.nodes = take((2 * few_nodes(sm_count) + tile_nodes(sm_count)) * 4);
  w.few = take(attend_few_workspace(D, sm_count));
  w.state = take(n_rows * Q * (D + 2) * 4);
  w.bytes += kAlign;  // the caller's buffer starts on 16 bytes, sums are written 32 at a time
  return w;
}

// Whether to share at all, by what the host knows: the tables' width as a bound on the lengths. The shared form is
// three launches in a row, and until the batch's cache outgrows L2 and what it delivers kv_attend_layer is as fast:
// elements that it would read more than once, in millions, and us (kv_attend_layer / shared), 8 KV and 32 query heads
// of 128, one token a sequence: 64 sequences of one prefix, bf16, 134 41 / 43, 266 62 / 48, 531 105 / 53; 64 of 16
// prefixes 203 64 / 67, 404 133 / 95, 807 335 / 154; 16 of one prefix 126 43 / 47, 252 64 / 51; 8 bits, 64 of one 134
// 39 / 49, 266 57 / 54, 64 of 16 203 59 / 60, 404 102 / 77; 4 bits 46 / 51, 63 / 56, 63 / 52, 99 / 67. In tables that
// are wider than the batch is long it shares too early: four answers behind 608 tokens 17 us, in a table for 131072
// tokens 29 (8 bits 17 and 35, 4 bits 19 and 33).
bool worth_sharing(const DevPool& p, const Batch& b, const AttendArgs& a, int32_t n_groups) {
  if (n_groups >= b.n_seqs || b.n_rows * a.G > kOwnTiles * static_cast<int64_t>(b.n_seqs)) return false;
  const double again = static_cast<double>(b.n_seqs - n_groups) * b.max_pages * p.ps * a.H * a.D * 2;
  return again >= (b.n_seqs / 32 >= n_groups ? 0x1p27 : 0x1p28);
}

// Which kernel attends to the prefixes, by a group's rows of a KV head on average: k_attend_few up to 8 (8-bit and
// 4-bit caches 32), else k_attend_tile. us, few / tile: 16-bit, 8 rows (64 sequences in 32 groups behind 4096 tokens)
// 117 / 153, 16 rows (16 groups, 2048 tokens) 69 / 67, 32 rows (8 groups, 4096) 83 / 68; 8-bit 16 rows (8192) 102 /
// 158, 32 rows (4096) 71 / 74, 48 rows 80 / 79, 64 rows 92 / 84; 4-bit 91 / 157, 63 / 68, 74 / 72, 87 / 79. One kernel
// takes all prefixes: a group far larger than the average is gone over once for every 8 or 16 of its rows in the first,
// one far smaller leaves tiles empty in the second.
int64_t prefix_few_rows(Kind kind) { return kind == Kind::kElements ? 8 : 32; }

}  // namespace

int64_t attend_shared_workspace_bytes(int32_t Q, int32_t D, int32_t n_seqs, int64_t n_rows, int sm_count) {
  return workspace_of(Q, D, n_seqs, n_rows, sm_count).bytes;
}

cudaError_t launch_attend_shared(const DevPool& p, const Batch& b, const AttendArgs& a, Kind kind, const Groups& gr,
                                 const int32_t* prefix_len, void* workspace, int sm_count, cudaStream_t s) {
  const int32_t n_groups = gr.n;
  if (!has_tiles(a.D) || !worth_sharing(p, b, a, gr.n)) return launch_attend(p, b, a, kind, gr, workspace, sm_count, s);
  const Workspace w = workspace_of(a.Q, a.D, b.n_seqs, b.n_rows, sm_count);
  uint8_t* ws = reinterpret_cast<uint8_t*>(aligned(static_cast<int64_t>(reinterpret_cast<uintptr_t>(workspace))));
  Seq* own = reinterpret_cast<Seq*>(ws + w.own);
  Seq* shared = reinterpret_cast<Seq*>(ws + w.shared);
  int32_t* from = reinterpret_cast<int32_t*>(ws + w.from);
  int32_t* nodes = reinterpret_cast<int32_t*>(ws + w.nodes);
  const int32_t n_nodes = static_cast<int32_t>(2 * few_nodes(sm_count) + tile_nodes(sm_count));
  k_share_groups<<<n_groups < kZeroBlocks ? kZeroBlocks : n_groups < 2 * sm_count ? n_groups : 2 * sm_count, kGroupBlock, 0, s>>>(
      p, b, gr, prefix_len, a.G, own, shared, from, nodes, n_nodes);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  Split split{};
  Batch bb = b;
  AttendArgs aa = a;
  aa.state_rows = b.n_rows * a.Q;
  bb.seqs = shared;
  bb.n_spans = n_groups;
  aa.state = reinterpret_cast<float*>(ws + w.state);
  aa.Gp = INT32_MAX;
  if (b.n_rows * a.G <= prefix_few_rows(kind) * static_cast<int64_t>(n_groups))
    e = launch_attend_few(p, bb, aa, kind, INT32_MAX, ws + w.tiles, sm_count, Launch::kFirst, nodes, &split, s);
  else
    e = launch_attend_tile(p, bb, aa, kind, 1, ws + w.tiles, sm_count, Launch::kFirst, nodes + 2 * few_nodes(sm_count), &split, s);
  if (e != cudaSuccess) return e;
  bb = b;
  bb.seqs = own;
  bb.from = from;
  aa.prior = aa.state;
  aa.state = nullptr;
  aa.Gp = a.G;
  return launch_attend_few(p, bb, aa, kind, INT32_MAX, ws + w.few, sm_count, Launch::kAfter, nodes + few_nodes(sm_count),
                           &split, s);
}

}  // namespace gtkv
