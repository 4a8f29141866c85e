// Attention of few rows a sequence (decode steps, drafted tokens): at most 16 rows (8-bit and 4-bit caches: 32) on
// average, a row being a (token, query head) pair of one KV head, in tiles of 8 or 16; a sequence with more takes
// several tiles, each of which reads its keys and values again. A tile reads them once for a handful of rows, so the
// bound is memory; the work is laid out so that nothing stands between the loads. Behind shared prefixes the kernel
// takes the own tokens of all sequences, however many rows they have, and prefixes of groups of few rows
// (kv_attend_shared.cu has the limits).
//
// One warp owns one KV head over its own run of keys, 16 keys a step, and never talks to another warp. Both products
// run as mma m16n8k16 with the CACHE as the 16-row operand, S^T = K Q^T and O^T = V^T P^T, rows as the 8 (or 16)
// columns, so 4 query heads fill half of an instruction instead of a quarter. The order of the summed index is free, so
// operand registers are filled from whole 16-byte pieces of the rows as they lie in the cache: lane (g, c) = (lane / 4,
// lane % 4) takes pieces of keys g and g + 8 for K, and its eighth of the elements of keys 2c, 2c + 1, 2c + 8, 2c + 9
// for V, where byte permutes pair up two keys. Rows come by cp.async into a ring of the warp's own, whole rows an
// instruction. No transpose, no bank conflict, no barrier. Codes become fp16 (exact) on the way into the registers; P^T
// comes out of the score registers by movmatrix.
//
// Softmax: the running reference m moves only when a score exceeds it by 2^8 (a vote per step), so the common step has
// no shuffle. Weights are 2^(t - m), t = score * log2(e) + log2(value scale): the scale of an 8-bit value is part of
// its weight, so that weights stay in one range, and the denominator adds weight / scale. Weights meet the values as
// the sum of two 16-bit parts and keep 16 bits (bf16) or 22 (fp16, lifted by 2^6 so that 2^-30 of the largest still
// counts): the result's error is then the output's own rounding and no more, where one part alone adds 40 % to it (fp16
// output, 4096 keys, root mean square: 5.39e-6 and 7.54e-6). Under 16-bit caches the second product is free, memory
// being the bound. Of 8-bit caches read into bf16, whose 8 bits hide the 11 of one fp16 part (8.73e-5 and 8.79e-5), the
// weights are one part, and so they are of 4-bit caches (the result's whole error grows by 0.8 %): drafts in 8 bits
// take 334 us so and 377 with two, 256 x 4096 tokens in 4 bits 320 and 337. Queries for 8-bit caches are fp16 after a
// power-of-two scaling per row, exact for all bits that matter (2^-29 of the row's largest).
//
// Measured: 256 sequences of 4096 tokens (bf16, 8 KV heads of 128, 4.3 GB) 680 to 698 us from one GPU to another, 91 to
// 93 % of the copy rate; 40 sequences of 9 to 40 961 tokens with drafts (8-bit, 1.68 GB) 332 us, 74 %, bound by latency
// inside a warp (codes into fp16, products, weights, one after the other) with three warps a scheduler; one sequence of
// 203 tokens 14 us, latency.
//
// 4-bit caches. A lane's piece of a key is a quarter of the head (two blocks of 16 and their scale bytes), its part of
// a value an eighth (one block, or half of one). Two elements become fp16 by one conversion and one product with the
// block's scale, exactly; codes of two values share a byte before that, so that no halves are exchanged. That is 64
// conversions (at half rate) and 64 products a lane and step, beside some 300 other instructions; latency bounds the
// kernel (issue slots 60 % busy): 256 x 4096 tokens (1.2 GB) 320 us, 56 % of the copy rate. What it is sensitive to, in
// us: one block of keys a round instead of two 324; shared memory that leaves little of L1, where the heads of a block
// find each other's scale sectors, rings of six stages 393; three blocks an SM 319, five, which spill, 494. 16 columns
// need all registers of two blocks an SM (drafts of 9 to 40 961 tokens, fp16, 377 us; with three blocks, which spill,
// 398).
//
// Workers (as many warps as share a step's heads) take equal shares of all steps of the batch (kv_attend_split.cuh);
// units cut at a border are joined by k_attend_join from 32-bit partial sums in the workspace.
#pragma once

#include "kv_attend_launch.h"
#include "kv_attend_split.cuh"

namespace gtkv {

namespace {

constexpr int kUnitCost = kFewUnitCost;
template <class C>
struct FewType {
  static constexpr int kSize = 2;       // bytes per cached element
  static constexpr float kLift = 6.0f;  // log2 of the weights' lift
};
template <>
struct FewType<CodeE4M3> {
  static constexpr int kSize = 1;
  static constexpr float kLift = 6.0f;
};
template <>
struct FewType<CodeE2M1> {
  static constexpr float kLift = 6.0f;
};
template <>
struct FewType<__nv_bfloat16> {
  static constexpr int kSize = 2;
  static constexpr float kLift = 0.0f;
};

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// d (+)= A B; `first`: d starts from zero.
template <class C>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, bool first = false) {
  const float z0 = first ? 0.0f : d[0], z1 = first ? 0.0f : d[1], z2 = first ? 0.0f : d[2], z3 = first ? 0.0f : d[3];
  if constexpr (std::is_same_v<C, __nv_bfloat16>)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
}

// 8x8 transpose of 16-bit elements over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <class C, int D>
struct FewShape {
  static constexpr int row_of() {
    if constexpr (std::is_same_v<C, CodeE2M1>)
      return D / 2;
    else
      return D * FewType<C>::kSize;
  }
  static constexpr bool kE2M1 = std::is_same_v<C, CodeE2M1>;
  static constexpr int kRow = row_of();       // bytes of a head's row (4-bit caches: of its codes)
  static constexpr int kKC = kRow / 64;       // 16-byte pieces of a key that a lane holds
  static constexpr int kScaleRow = kE2M1 ? D / 16 : 0;  // bytes of a head's scales in a row
  static constexpr int kVB = kRow / 8;        // bytes of a value that a lane holds
  static constexpr int kVC = kVB < 16 ? 1 : kVB / 16;  // pieces of it, 128 bytes apart
  static constexpr int kK = 16 * kRow;        // bytes of a step's K, and of its V
  static constexpr int kLPR = kRow / 16;       // lanes that copy a row
  static constexpr int kRPR = 32 / kLPR;       // rows a round
  static constexpr int kRounds = 16 / kRPR;
  // what round `it` adds to the swap of V's pieces, in bytes of the address
  static __device__ __forceinline__ constexpr uint32_t flip_v(int it) {
    return kRow >= 256 ? (it & 3) * 32 : kRow >= 128 ? (it & 1) * 64 : 0;
  }
  // 4-bit caches: the scale bytes of 16 keys and values, else 32 scales; the mask of live keys behind them
  static constexpr int kMeta = (kE2M1 ? 32 * kScaleRow : 128) + 16;
  static constexpr int kLive = 2 * kK + kMeta - 16;
  static constexpr int kStage = 2 * kK + kMeta;
  // Stages of a warp's ring: as many as shared memory holds with all the
  // blocks that fit an SM, or, for calls of one block an SM, whose time is latency, six.
  static constexpr int kStages = kRow >= 256 ? 2 : kRow >= 128 ? 3 : kE2M1 && D == 128 ? 4 : 6;
  static constexpr int kDeep = 6;
  // blocks of 16 keys a round of the loop: two of a 4-bit cache, whose loads and softmax are little beside what a
  // round costs anyway, and whose conversions are chains that then overlap (256 x 4096 tokens 320 us, with one 324)
  static __host__ __device__ constexpr int blocks(int nt) { return kE2M1 && nt == 1 ? 2 : 1; }
  static constexpr int kKS = D / 16;          // k16 steps of the score product
  // bytes of a warp's queries in shared memory: of 4-bit caches and 8 columns, whose registers they would not leave
  static __host__ __device__ constexpr int queries(int nt) { return kE2M1 && nt == 1 ? D * 16 : 0; }
  static constexpr int kMT = D / 16;          // 16-element tiles of the output
};

// P16: the page size is a multiple of 16, so a step's keys share a page and a
// lane looks up the pages of 32 steps ahead at once; otherwise every key's entry is
// read on its own, one step ahead. 256 x 4096 tokens in pages of 16, bf16, on one GPU: 686 us against
// 698 by keys; 8-bit, pages of 32: the same within 1 %.

// TWO: weights in two parts. SHARED: a pass over prefixes, whose sums it leaves in a.state, or the one
// over sequences' own tokens, which takes them up from a.prior (kv_attend_shared.cu); instances of their own, since
// their code costs the plain ones 1 % (decode) to 6 % (k_attend_tile, prompts).
template <class C, int D, int NT, bool P16, bool TWO, bool SHARED>
__global__ void __launch_bounds__(kFewBlock, few_blocks(FewShape<C, D>::kRow, NT, FewShape<C, D>::kE2M1))
    k_attend_few(DevPool p, Batch b, AttendArgs a, Split w) {
  using Sh = FewShape<C, D>;
  constexpr bool kE4M3 = std::is_same_v<C, CodeE4M3>, kE2M1 = Sh::kE2M1;
  constexpr bool kCodes = kE4M3 || kE2M1;
  constexpr float kLift = FewType<C>::kLift;
  constexpr int NQ = 8 * NT;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ ShareStart loc[kFewWarps];
  __shared__ int64_t tmp[kFewWarps];
  if (SHARED && w.first) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int kw = kFewWarps / w.hw;             // workers of the block
  const int wk = warp / w.hw;                  // this warp's worker in the block
  const int hw = warp - wk * w.hw;             // its head of the worker's group
  const int32_t n_groups = a.H / w.hw;
  const int32_t Gp = SHARED ? a.Gp : a.G;      // rows of a sequence's position
  int bits = 0;

  auto tiles_of = [&](const Seq& q) { return q.n == 0 || q.n > w.max_new ? 0 : (q.n * a.G + NQ - 1) / NQ; };
  auto span_of = [&](const Seq& q, int32_t s, int32_t t) {
    const int32_t f0 = t * NQ, f1 = min(f0 + NQ, q.n * a.G);
    KeySpan k = key_span<16>(a, q.a + f0 / Gp, q.a + (f1 - 1) / Gp);
    if (SHARED && b.from) k.b0 = __ldcg(b.from + s) >> 4;
    return k;
  };
  const int32_t worker0 = static_cast<int32_t>(blockIdx.x) * kw;
  const int64_t share = find_shares<kFewBlock, kFewWarps>(
      b.n_seqs, worker0, w.n_workers, w.min_share, loc, tmp, [&](int32_t s) -> int64_t {
        int err = 0;
        const Seq q = seq_of<SHARED>(p, b, s, err);
        if (blockIdx.x == 0) bits |= err;
        int64_t n = 0;
        if (w.whole) return static_cast<int64_t>(tiles_of(q)) * n_groups;
        for (int32_t t = 0; t < tiles_of(q); ++t) n += span_of(q, s, t).steps() + kUnitCost;
        return n * n_groups;
      });
  const int32_t worker = worker0 + wk;
  SplitRecord rec{-1, 0, 0, 0, 0, 0, 0};
  ShareStart at = loc[wk];
  if (worker >= w.n_workers) at.s = -1;

  // The warp's ring. A row's 16-byte pieces are permuted within it so that the
  // reads below meet no bank twice: K's piece p of row r sits at p ^ 4 (r % 2),
  // V's at p ^ 2 (r / 2 % 4) (64-byte rows: p and p ^ (r / 2 % 4); of 32-byte rows
  // V's stay whole, row r at r ^ (r / 4 % 2)).
  const int cr = lane / Sh::kLPR, cp = lane % Sh::kLPR;  // row of a round and piece that the lane copies
  const uint32_t put_k = cr * Sh::kRow + (Sh::kRow > 64 ? cp ^ (cr & 1) * 4 : cp) * 16;
  const uint32_t put_v =
      Sh::kRow == 32 ? (cr ^ (cr >> 2 & 1)) * 32 + cp * 16
                     : cr * Sh::kRow +
                           (Sh::kRow >= 256 ? cp : Sh::kRow > 64 ? cp ^ (cr >> 1) * 2 : cp ^ (cr >> 1 & 3)) * 16;
  const uint32_t get_k = g * Sh::kRow + (Sh::kRow > 64 ? c ^ (g & 1) * 4 : c) * (Sh::kRow == 32 ? 8 : 16);  // ^ 64 ch, + 8 rows
  const uint32_t get_v =
      Sh::kRow == 32 ? (2 * c + (c >> 1)) * 32 + g * 4
                     : 2 * c * Sh::kRow + (Sh::kRow > 64 ? (g ^ 2 * c) * 16 : ((g >> 1) ^ c) * 16 + (g & 1) * 8);
  // where the lane's part of values 2c, 2c + 1, 2c + 8, 2c + 9 lies
  auto value_at = [&](int kk) {
    return Sh::kRow == 32 ? (get_v ^ (kk & 1) * 32) + 8 * (kk >> 1) * 32 : get_v + ((kk & 1) + 8 * (kk >> 1)) * Sh::kRow;
  };
  const int stages = w.deep ? Sh::kDeep : Sh::kStages;
  const uint32_t ring0 = shared_u32(ring) + warp * stages * Sh::kStage;
  constexpr bool kQShared = Sh::queries(NT) > 0;
  const uint32_t qs = shared_u32(ring) + kFewWarps * stages * Sh::kStage + warp * Sh::queries(NT) + lane * 16;  // + 512 for two steps
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.base);
  const int32_t row_bytes = static_cast<int32_t>(p.vpr * 16);

  int64_t left = at.s < 0 ? 0 : share;
  int32_t s = at.s, tile = 0, group = 0;
  int32_t step0 = 0;
  int64_t in_unit = 0;  // SHARED: of the share's first unit, what of its line lies before the share
  Seq q{0, 0, 0};
  KeySpan span{0, 0, 0};
  if (left > 0) {  // the unit and step where the share begins
    int err = 0;
    q = seq_of<SHARED>(p, b, s, err);
    int64_t off = at.off;
    for (;;) {
      span = span_of(q, s, tile);
      const int64_t n = static_cast<int64_t>(w.whole ? 1 : span.steps() + kUnitCost) * n_groups;
      if (off < n) break;
      off -= n;
      ++tile;
    }
    if (w.whole) {
      group = static_cast<int32_t>(off);
    } else {
      const int32_t unit = span.steps() + kUnitCost;
      group = static_cast<int32_t>(off / unit);
      const int32_t in = static_cast<int32_t>(off - static_cast<int64_t>(group) * unit);
      step0 = in < kUnitCost ? 0 : in - kUnitCost;
      in_unit = in;
      left -= in < kUnitCost ? kUnitCost - in : 0;
    }
  }

  while (left > 0) {
    const int32_t n_steps = span.steps();
    const int32_t end = !w.whole && left < n_steps - step0 ? step0 + static_cast<int32_t>(left) : n_steps;
    const int32_t h = group * w.hw + hw;
    const int32_t f0 = tile * NQ;
    const int32_t nf = min(NQ, q.n * a.G - f0);  // rows of the tile
    const int32_t i0 = q.a + f0 / Gp, i1 = q.a + (f0 + nf - 1) / Gp;

    // ---- issue of a step's loads
    // the lane's piece of row 0 of a page, in the layer's block of keys; rows are below 2^31
    const uint8_t* from = pool + (2 * static_cast<int64_t>(a.layer) * p.ps + cr) * row_bytes + h * Sh::kRow + cp * 16;
    const int32_t page_rows = static_cast<int32_t>(p.stride), ps = static_cast<int32_t>(p.ps);
    const float* scale_at = kE4M3 ? a.scales + 2 * static_cast<int64_t>(a.layer) * a.H + h : nullptr;  // of page 0
    const int32_t page_scales = p.blocks * a.H;
    // from the lane's piece of row 0 to the scale bytes of its key or value of a step
    const int64_t scales4 = code_bytes(a.H, D) + h * Sh::kScaleRow - (h * Sh::kRow + cp * 16) + ((lane & 15) - cr) * static_cast<int64_t>(row_bytes) +
                            (lane >> 4) * p.ps * row_bytes;
    const int64_t round_bytes = Sh::kRPR * static_cast<int64_t>(row_bytes), v_bytes = p.ps * row_bytes;
    uint32_t whole_stages = 0;  // bit s: all 16 keys of stage s are tokens
    int32_t ent = 0;  // P16: page of step seg_base + lane (0: tombstone); else: raw entry of key lane % 16 of the next step
    auto page_of_step = [&](int32_t i) -> int32_t {
      if (i >= end) return 0;
      const int64_t k = div_ps(p, static_cast<int64_t>(span.block(i)) * 16);
      return static_cast<int32_t>(
          page_of_entry(p, b, __ldg(b.table + static_cast<int64_t>(s) * b.max_pages + k), bits));
    };
    auto entry_of_key = [&](int32_t i) -> int32_t {  // general: table entry of key `lane % 16` of step i
      const int64_t j = static_cast<int64_t>(span.block(i < end ? i : step0)) * 16 + (lane & 15);
      return i < end && j <= i1 && some_row_sees(a, i0, j, j) ? __ldg(b.table + static_cast<int64_t>(s) * b.max_pages + div_ps(p, j)) : 0;
    };
    int32_t seg_base = step0;  // P16: `ent` covers steps [seg_base, seg_base + 32)
    int32_t ent_next = 0;
    if constexpr (P16) {
      ent = page_of_step(step0 + lane);
      ent_next = page_of_step(step0 + 32 + lane);
    } else {
      ent = entry_of_key(step0);
    }
    auto issue = [&](int32_t i, int stage) {
      if (i < end) {
        const uint32_t st = ring0 + stage * Sh::kStage;
        const int32_t j0 = span.block(i) * 16;
        int32_t page;     // of the step (P16) or of key lane % 16
        int32_t rk;       // row of key 0, or of key lane % 16
        uint32_t live;    // bit k: key k is a token of the cache
        if constexpr (P16) {
          if (i >= seg_base + 32) {
            seg_base += 32;
            ent = ent_next;
            ent_next = page_of_step(seg_base + 32 + lane);
          }
          page = __shfl_sync(kFull, ent, i - seg_base);
          live = page == 0 ? 0 : i1 - j0 >= 15 ? 0xffffu : (2u << (i1 - j0)) - 1;
          rk = page * page_rows + (p.ps_shift >= 0 ? j0 & (ps - 1) : j0 % ps);
        } else {
          const int32_t e = ent;
          ent = entry_of_key(i + 1);
          const int32_t j = j0 + (lane & 15);
          page = (lane & 15) <= i1 - j0 ? static_cast<int32_t>(page_of_entry(p, b, e, bits)) : 0;
          rk = page * page_rows + (page != 0 ? j % ps : 0);
          live = __ballot_sync(kFull, page != 0) & 0xffffu;
        }
        const bool all = P16 && live == 0xffffu;
        whole_stages = (whole_stages & ~(1u << stage)) | static_cast<uint32_t>(all) << stage;
        const uint8_t* base = from;
        if (all) {  // every key is a token: one base address and constant offsets
          base += static_cast<int64_t>(rk) * row_bytes;
#pragma unroll
          for (int it = 0; it < Sh::kRounds; ++it) copy_async<16>(st + put_k + it * 512, base + it * round_bytes);
          base += v_bytes;
#pragma unroll
          for (int it = 0; it < Sh::kRounds; ++it)
            copy_async<16>(st + Sh::kK + (put_v ^ Sh::flip_v(it)) + it * 512, base + it * round_bytes);
        } else {
#pragma unroll
          for (int it = 0; it < Sh::kRounds; ++it) {
            const int key = it * Sh::kRPR + cr;
            const int32_t r = P16 ? rk + it * Sh::kRPR : __shfl_sync(kFull, rk, key) - cr;
            const bool ok = live >> key & 1;
            const uint8_t* src = ok ? base + static_cast<int64_t>(r) * row_bytes : pool;
            copy_async<16>(st + put_k + it * 512, src, ok);
            copy_async<16>(st + Sh::kK + (put_v ^ Sh::flip_v(it)) + it * 512, src + (ok ? v_bytes : 0), ok);
          }
          if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + Sh::kLive), "r"(live) : "memory");
        }
        if constexpr (kE2M1) {  // lanes 0-15: a key's scales, 16-31: a value's
          if (all) {
            copy_async<Sh::kScaleRow>(st + 2 * Sh::kK + lane * Sh::kScaleRow, from + static_cast<int64_t>(rk) * row_bytes + scales4);
          } else {
            const bool ok = live >> (lane & 15) & 1;
            const int64_t r = P16 ? rk : rk - (lane & 15);
            copy_async<Sh::kScaleRow>(st + 2 * Sh::kK + lane * Sh::kScaleRow, ok ? from + r * row_bytes + scales4 : pool, ok);
          }
        } else if constexpr (kE4M3 && P16) {  // one scale of K (lane 0) and one of V (lane 1)
          if (lane < 2)
            copy_async<4>(st + 2 * Sh::kK + lane * 4,
                          scale_at + static_cast<int64_t>(page) * page_scales + lane * a.H);
        } else if constexpr (kE4M3) {  // lanes 0-15: scales of K, 16-31: of V
          const bool ok = live >> (lane & 15) & 1;
          copy_async<4>(st + 2 * Sh::kK + lane * 4,
                        scale_at + (ok ? static_cast<int64_t>(page) * page_scales + (lane >> 4) * a.H : 0), ok);
        }
      }
      copy_commit();
    };
    constexpr int KB = Sh::blocks(NT);
    for (int i = 0; i < stages - KB; ++i) issue(step0 + i, i);

    // ---- the queries, while the first loads are in flight
    uint32_t qf[NT][kQShared ? 2 : Sh::kKS][2];
    float cq[NT][2];
    int32_t pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int32_t f = f0 + nt * 8 + g;
      const bool ok = nt * 8 + g < nf;
      const int64_t q0 = ok ? (q.row0 + f / a.G) * a.q_stride + static_cast<int64_t>(h * a.G + f % a.G) * D : 0;
      float row_c = a.scale_log2;
      if constexpr (!kCodes) {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + q0;
#pragma unroll
        for (int ch = 0; ch < Sh::kKC; ++ch) {
          const uint16_t* e = src + ch * 32 + c * 8;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (ok) {
            if (w.q_wide) {
              v = __ldg(reinterpret_cast<const uint4*>(e));
            } else {
              uint16_t* d = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
              for (int k = 0; k < 8; ++k) d[k] = __ldg(e + k);
            }
          }
          qf[nt][2 * ch][0] = v.x, qf[nt][2 * ch][1] = v.y;
          qf[nt][2 * ch + 1][0] = v.z, qf[nt][2 * ch + 1][1] = v.w;
        }
      } else {
        // the lane's elements of a key, in the order of its codes: sixteen of every 64, or (4-bit caches) a quarter of
        // the head
        constexpr int NV = D / 32;  // in vectors of eight
        float x[8 * NV];
        float amax = 0.0f;
#pragma unroll
        for (int vec = 0; vec < NV; ++vec) {
          const int e0 = kE2M1 ? c * (D / 4) + vec * 8 : vec / 2 * 64 + c * 16 + vec % 2 * 8;
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + q0 + e0;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (ok && w.q_wide) {
            v = __ldg(reinterpret_cast<const uint4*>(src));
          } else if (ok) {
            uint32_t e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = __ldg(src + k);
            v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
          }
          const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = a.type == KV_TYPE_BF16 ? make_float2(__uint_as_float(vw[k] << 16), __uint_as_float(vw[k] & 0xffff0000u))
                                                    : halves(vw[k]);
            x[vec * 8 + 2 * k] = f.x;
            x[vec * 8 + 2 * k + 1] = f.y;
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        // amax * 2^k in [2^14, 2^15)
        int k = 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23);
        k = amax > 0.0f ? max(-100, min(100, k)) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        row_c *= __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
        for (int ks = 0; ks < Sh::kKS; ++ks) {
          const int at = kQShared ? ks & 1 : ks;
          qf[nt][at][0] = pack_h(x[4 * ks] * up, x[4 * ks + 1] * up);
          qf[nt][at][1] = pack_h(x[4 * ks + 2] * up, x[4 * ks + 3] * up);
          if constexpr (kQShared)  // (a lane reads what it wrote)
            if (ks & 1)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(qs + ks / 2 * 512), "r"(qf[nt][0][0]), "r"(qf[nt][0][1]),
                           "r"(qf[nt][1][0]), "r"(qf[nt][1][1])
                           : "memory");
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // columns 2c and 2c + 1 of the scores
        cq[nt][e] = __shfl_sync(kFull, row_c, (2 * c + e) * 4);
        pos[nt][e] = q.a + min(f0 + nt * 8 + 2 * c + e, f0 + nf - 1) / Gp;
      }
    }

    float o[Sh::kMT][NT][4];
    // exponents are taken below `low` = reference - lift; they may reach `high`
    // before the reference moves (-inf: no key seen yet, so any key moves it)
    float low[NT][2], high[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < Sh::kMT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.0f;
      low[nt][0] = low[nt][1] = 0.0f;
      high[nt][0] = high[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.0f;
    }

    int stage = 0;
    for (int32_t i = step0; i < end; i += KB) {
#pragma unroll
      for (int hb = 0; hb < KB; ++hb) {
        int ahead = stage + stages - KB + hb;
        if (ahead >= stages) ahead -= stages;
        issue(i + stages - KB + hb, ahead);
      }
      if (w.deep)
        copy_wait<Sh::kDeep - KB>();
      else
        copy_wait<Sh::kStages - KB>();
      __syncwarp();
      uint32_t st[KB], live[KB];
      int32_t j0[KB];
      bool mask = false;  // some row may not see some key
#pragma unroll
      for (int hb = 0; hb < KB; ++hb) {
        st[hb] = ring0 + (stage + hb) * Sh::kStage;
        live[hb] = whole_stages >> (stage + hb) & 1 ? 0xffffu : lds32(st[hb] + Sh::kLive);
        j0[hb] = span.block(i + hb) * 16;
        if (hb > 0 && i + hb >= end) live[hb] = 0;  // past the last: nothing was copied
        mask = mask || live[hb] != 0xffffu || j0[hb] + 15 > i0 || (a.window && j0[hb] <= i1 - a.window);
      }

      // ---- scores
      // two sums for one tile of columns, so that products wait half as long for one another
      constexpr bool kTwo = NT == 1;
      float x[KB][NT][4];
      uint32_t s01[KB], s23[KB];  // 4-bit caches: the scales of the lane's part of its four values, as pairs of fp16
#pragma unroll
      for (int hb = 0; hb < KB; ++hb) {
        float x2[NT][4];
        float(&xb)[NT][4] = x[hb];
        if constexpr (kE2M1) {
          const uint32_t at = st[hb] + 2 * Sh::kK;
          // the lane's scale bytes of keys g and g + 8, a key's in a half
          const uint32_t ka = at + g * Sh::kScaleRow + c * (D / 64);
          uint32_t kb;
          if constexpr (D == 128)
            kb = lds16(ka) | lds16(ka + 8 * Sh::kScaleRow) << 16;
          else
            kb = lds8(ka) | lds8(ka + 8 * Sh::kScaleRow) << 16;
          const uint32_t va = at + (16 + 2 * c) * Sh::kScaleRow + (D == 128 ? g : g >> 1);
          s01[hb] = lds8(va) * 0x80u + lds8(va + Sh::kScaleRow) * 0x800000u;
          s23[hb] = lds8(va + 8 * Sh::kScaleRow) * 0x80u + lds8(va + 9 * Sh::kScaleRow) * 0x800000u;
          if (const uint32_t bad = above_max(kb)) kb |= (bad >> 7) * 0xffu;
          constexpr int W = D / 32;  // words of codes
          uint32_t uu[W], vv[W];
          if constexpr (W == 4) {
            const uint4 u = lds128(st[hb] + get_k), v = lds128(st[hb] + get_k + 8 * Sh::kRow);
            uu[0] = u.x, uu[1] = u.y, uu[2] = u.z, uu[3] = u.w;
            vv[0] = v.x, vv[1] = v.y, vv[2] = v.z, vv[3] = v.w;
          } else {
            const uint2 u = lds64(st[hb] + get_k), v = lds64(st[hb] + get_k + 8 * Sh::kRow);
            uu[0] = u.x, uu[1] = u.y;
            vv[0] = v.x, vv[1] = v.y;
          }
          uint32_t sa[W / 2], sb[W / 2];  // a block's scale, twice
#pragma unroll
          for (int blk = 0; blk < W / 2; ++blk) {
            sa[blk] = __byte_perm(kb, 0, blk ? 0x4141 : 0x4040) * 0x80u;
            sb[blk] = __byte_perm(kb, 0, blk ? 0x4343 : 0x4242) * 0x80u;
          }
#pragma unroll
          for (int wd = 0; wd < W; ++wd) {
            uint32_t y[4], z[4];
            codes8(uu[wd], y);
            codes8(vv[wd], z);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[k] = mul_h2(y[k], sa[wd / 2]);
              z[k] = mul_h2(z[k], sb[wd / 2]);
            }
            uint4 qq = make_uint4(0, 0, 0, 0);
            if constexpr (kQShared) qq = lds128(qs + wd * 512);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<C>(kTwo && half ? x2[nt] : xb[nt], y[2 * half], z[2 * half], y[2 * half + 1], z[2 * half + 1],
                       kQShared ? (half ? qq.z : qq.x) : qf[nt][kQShared ? 0 : 2 * wd + half][0],
                       kQShared ? (half ? qq.w : qq.y) : qf[nt][kQShared ? 0 : 2 * wd + half][1], 2 * wd + half < 1 + kTwo);
          }
        }
#pragma unroll
        for (int ch = 0; ch < (kE2M1 ? 0 : Sh::kKC); ++ch) {
          const uint4 u = lds128(st[hb] + (get_k ^ ch * 64)), v = lds128(st[hb] + (get_k ^ ch * 64) + 8 * Sh::kRow);
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
          if constexpr (kE4M3) {
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) {
              const uint32_t a0 = codes_lo(uu[wd]), a1 = codes_lo(vv[wd]), a2 = codes_hi(uu[wd]), a3 = codes_hi(vv[wd]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<C>(kTwo && wd & 1 ? x2[nt] : xb[nt], a0, a1, a2, a3, qf[nt][ch * 4 + wd][0], qf[nt][ch * 4 + wd][1],
                       ch * 4 + wd < 1 + kTwo);
            }
          } else {
#pragma unroll
            for (int wd = 0; wd < 2; ++wd)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<C>(kTwo && wd & 1 ? x2[nt] : xb[nt], uu[2 * wd], vv[2 * wd], uu[2 * wd + 1], vv[2 * wd + 1],
                       qf[nt][ch * 2 + wd][0], qf[nt][ch * 2 + wd][1], ch * 2 + wd < 1 + kTwo);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (kTwo) xb[nt][e] += x2[nt][e];
      }

      // ---- weights; x[.][0], [1]: key g, columns 2c, 2c + 1; [2], [3]: key g + 8
      float lv[2] = {0.0f, 0.0f}, iv[2] = {1.0f, 1.0f}, sk[2] = {1.0f, 1.0f};
      if constexpr (kE4M3) {
        if constexpr (P16) {
          const uint2 kv = lds64(st[0] + 2 * Sh::kK);
          sk[0] = sk[1] = __uint_as_float(kv.x);
          lv[0] = lv[1] = lg2(__uint_as_float(kv.y));
          iv[0] = iv[1] = rcp(__uint_as_float(kv.y));
        }
#pragma unroll
        for (int e = 0; e < (P16 ? 0 : 2); ++e) {
          sk[e] = __uint_as_float(lds32(st[0] + 2 * Sh::kK + (g + 8 * e) * 4));
          const float sv = __uint_as_float(lds32(st[0] + 2 * Sh::kK + 64 + (g + 8 * e) * 4));
          lv[e] = lg2(sv);
          iv[e] = rcp(sv);
        }
      }
#pragma unroll
      for (int hb = 0; hb < KB; ++hb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[hb][nt][e] = kE4M3 ? fmaf(x[hb][nt][e], cq[nt][e & 1] * sk[e >> 1], lv[e >> 1] - low[nt][e & 1])
                                 : fmaf(x[hb][nt][e], cq[nt][e & 1], -low[nt][e & 1]);
      // apart from the common step, where as predicates they were a third of its instructions (8-bit drafts 363 us, 332
      // so)
      if (mask) {
#pragma unroll
        for (int hb = 0; hb < KB; ++hb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = g + 8 * (e >> 1);
              if (!(live[hb] >> key & 1) || !in_sight(a, pos[nt][e & 1], j0[hb] + key)) x[hb][nt][e] = -INFINITY;
            }
      }
      bool over = false;
#pragma unroll
      for (int hb = 0; hb < KB; ++hb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) over = over || x[hb][nt][e] > high[nt][e & 1];
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
            if constexpr (KB > 1) m = fmaxf(m, fmaxf(x[KB - 1][nt][e], x[KB - 1][nt][e + 2]));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            if (m > kLift || (m > -INFINITY && high[nt][e] == -INFINITY)) {  // the maximum becomes the reference
              const float up = m - kLift;
              const float keep = high[nt][e] == -INFINITY ? 0.0f : ex2(-up);
              low[nt][e] += up;
              high[nt][e] = kLift + 8.0f;
#pragma unroll
              for (int hb = 0; hb < KB; ++hb) {
                x[hb][nt][e] -= up;
                x[hb][nt][e + 2] -= up;
              }
              sum[nt][e] *= keep;
#pragma unroll
              for (int mt = 0; mt < Sh::kMT; ++mt) {
                o[mt][nt][e] *= keep;
                o[mt][nt][e + 2] *= keep;
              }
            }
          }
      }
      uint32_t pb[KB][NT][2], pl[KB][NT][2];
#pragma unroll
      for (int hb = 0; hb < KB; ++hb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = ex2(x[hb][nt][e]);
            // a dead key adds nothing, whatever its zero-filled scale's inverse is
            if constexpr (kE4M3 && !P16)
              sum[nt][e & 1] += live[hb] >> (g + 8 * (e >> 1)) & 1 ? y[e] * iv[e >> 1] : 0.0f;
            else if constexpr (!kE4M3)
              sum[nt][e & 1] += y[e];
          }
          if constexpr (kE4M3 && P16) {
            if (live[hb]) {
              sum[nt][0] = fmaf(y[0] + y[2], iv[0], sum[nt][0]);
              sum[nt][1] = fmaf(y[1] + y[3], iv[0], sum[nt][1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            constexpr bool kBf16 = std::is_same_v<C, __nv_bfloat16>;
            const uint32_t hi = pack16<kBf16>(y[2 * e], y[2 * e + 1]);
            pb[hb][nt][e] = transpose8(hi);
            if constexpr (TWO) {
              const float2 h = unpack16<kBf16>(hi);
              pl[hb][nt][e] = transpose8(pack16<kBf16>(y[2 * e] - h.x, y[2 * e + 1] - h.y));
            }
          }
        }

      // ---- values: registers of keys 2c, 2c + 1 (a0, a1) and 2c + 8, 2c + 9 (a2, a3)
      auto tile_mma = [&](int hb, int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma<C>(o[mt][nt], a0, a1, a2, a3, pb[hb][nt][0], pb[hb][nt][1]);
          if constexpr (TWO) mma<C>(o[mt][nt], a0, a1, a2, a3, pl[hb][nt][0], pl[hb][nt][1]);
        }
      };
      // rows that see a key whose value was zeroed are done again
      auto redo = [&](int hb, uint32_t keys) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (keys >> (g + 8 * (e >> 1)) & 1 && x[hb][nt][e] != -INFINITY) sum[nt][e & 1] = NAN;
      };
#pragma unroll
      for (int hb = 0; hb < (kE2M1 ? KB : 0); ++hb) {
        uint32_t v[4][D == 128 ? 2 : 1];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (D == 128) {
            const uint2 u = lds64(st[hb] + Sh::kK + value_at(kk));
            v[kk][0] = u.x, v[kk][1] = u.y;
          } else {
            v[kk][0] = lds32(st[hb] + Sh::kK + value_at(kk));
          }
        }
        // scales above the largest: NaN, or, where some row may not see some key, zeroed as below
        const uint32_t bad = above_max_pair(s01[hb]) | above_max_pair(s23[hb]) >> 1;  // bits 15, 31 and 14, 30
        if (mask) {
          const uint32_t own = (bad >> 15 & 1) | (bad >> 30 & 2) | (bad >> 6 & 0x100) | (bad >> 21 & 0x200);
          const uint32_t keys = __reduce_or_sync(kFull, own << 2 * c);
          if (bad) {
            s01[hb] &= ~((bad >> 15 & 0x10001u) * 0xffffu);
            s23[hb] &= ~((bad >> 14 & 0x10001u) * 0xffffu);
          }
          if (keys) redo(hb, keys);
        } else if (bad) {
          s01[hb] |= (bad >> 15 & 0x10001u) * 0x7fffu;
          s23[hb] |= (bad >> 14 & 0x10001u) * 0x7fffu;
        }
        // Codes of a pair of values share a byte before they become a pair of fp16, so that no halves are exchanged.
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          uint32_t a0[4], a1[4], a2[4], a3[4];
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          codes8((v[0][wd] & kLow) | (v[1][wd] << 4 & ~kLow), a0);
          codes8((v[0][wd] >> 4 & kLow) | (v[1][wd] & ~kLow), a1);
          codes8((v[2][wd] & kLow) | (v[3][wd] << 4 & ~kLow), a2);
          codes8((v[2][wd] >> 4 & kLow) | (v[3][wd] & ~kLow), a3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tile_mma(hb, 4 * wd + k, mul_h2(a0[k], s01[hb]), mul_h2(a1[k], s01[hb]), mul_h2(a2[k], s23[hb]),
                     mul_h2(a3[k], s23[hb]));
        }
      }
      constexpr int VC = kE2M1 ? 0 : Sh::kVC;
      constexpr int VW = Sh::kVB >= 16 ? 4 : 2;             // words of a piece
#pragma unroll
      for (int ch = 0; ch < VC; ++ch) {
        uint32_t v[4][VW];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (VW == 4) {
            const uint4 u = lds128(st[0] + Sh::kK + value_at(kk) + ch * 128);
            v[kk][0] = u.x, v[kk][1] = u.y, v[kk][2] = u.z, v[kk][3] = u.w;
          } else {
            const uint2 u = lds64(st[0] + Sh::kK + value_at(kk));
            v[kk][0] = u.x, v[kk][1] = u.y;
          }
        }
        // A value that is not finite must reach the rows that see its key and no
        // other, but 0 * NaN would spread it. Where some row may not see some
        // key, such elements are zeroed here and the rows that do see the key
        // get a NaN denominator: they are done again, key by key, at the end.
        if (mask) {
          uint32_t keys = 0;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int wd = 0; wd < VW; ++wd) {
              const uint32_t bad = not_finite<C>(v[kk][wd]);
              v[kk][wd] &= ~bad;
              if (bad) keys |= 1u << (2 * c + (kk & 1) + 8 * (kk >> 1));
            }
          keys = __reduce_or_sync(kFull, keys);
          if (keys) redo(0, keys);
        }
#pragma unroll
        for (int wd = 0; wd < VW; ++wd) {
          if constexpr (kE4M3) {
            const uint32_t x0 = __byte_perm(v[0][wd], v[1][wd], 0x5140), y0 = __byte_perm(v[0][wd], v[1][wd], 0x7362);
            const uint32_t x1 = __byte_perm(v[2][wd], v[3][wd], 0x5140), y1 = __byte_perm(v[2][wd], v[3][wd], 0x7362);
            tile_mma(0, ch * 8 + 2 * wd, codes_lo(x0), codes_hi(x0), codes_lo(x1), codes_hi(x1));
            tile_mma(0, ch * 8 + 2 * wd + 1, codes_lo(y0), codes_hi(y0), codes_lo(y1), codes_hi(y1));
          } else {
            tile_mma(0, ch * 4 + wd, __byte_perm(v[0][wd], v[1][wd], 0x5410), __byte_perm(v[0][wd], v[1][wd], 0x7632),
                     __byte_perm(v[2][wd], v[3][wd], 0x5410), __byte_perm(v[2][wd], v[3][wd], 0x7632));
          }
        }
      }
      stage += KB;
      if (stage == stages) stage = 0;
      __syncwarp();  // the stage's scales and mask are free for the next issue
    }
    copy_wait<0>();

    // ---- the segment's end. o[mt][nt]: elements element(mt) (+ 1: [2], [3]) of columns 2c, 2c + 1
    auto element = [&](int mt) { return Sh::kVC == 1 ? g * (D / 8) + 2 * mt : mt / 4 * 64 + g * 8 + mt % 4 * 2; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[nt][e] += __shfl_xor_sync(kFull, sum[nt][e], 4);
        sum[nt][e] += __shfl_xor_sync(kFull, sum[nt][e], 8);
        sum[nt][e] += __shfl_xor_sync(kFull, sum[nt][e], 16);
      }
    bool whole = step0 == 0 && end == n_steps;
    if constexpr (SHARED) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (high[nt][e] == -INFINITY) low[nt][e] = kNoRef;
      // adds sums of the same rows, in the layout of a.state and of partial results: at(col) their place
      auto add = [&](const float* base, int64_t refs, int64_t sums, auto at, bool first) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int64_t r = at(nt * 8 + 2 * c + e);
            const float ref = __ldcg(base + refs + r), other = __ldcg(base + sums + r);
            const float top = fmaxf(ref, low[nt][e]), k1 = ex2(low[nt][e] - top), k2 = ex2(ref - top);
            low[nt][e] = top;
            auto sum_of = [&](float own, float oth) {  // left + right, whoever holds them
              return first ? __fmaf_rn(own, k1, __fmul_rn(oth, k2)) : __fmaf_rn(oth, k2, __fmul_rn(own, k1));
            };
            sum[nt][e] = sum_of(sum[nt][e], other);
#pragma unroll
            for (int mt = 0; mt < Sh::kMT; mt += 2) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(base + r * D + element(mt)));
              o[mt][nt][e] = sum_of(o[mt][nt][e], x.x);
              o[mt][nt][e + 2] = sum_of(o[mt][nt][e + 2], x.y);
              o[mt + 1][nt][e] = sum_of(o[mt + 1][nt][e], x.z);
              o[mt + 1][nt][e + 2] = sum_of(o[mt + 1][nt][e + 2], x.w);
            }
          }
      };
      auto leave = [&](float* base, int64_t refs, int64_t sums, auto at, int32_t cols) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * c + e;
            if (col >= cols) continue;
            const int64_t r = at(col);
#pragma unroll
            for (int mt = 0; mt < Sh::kMT; mt += 2)
              *reinterpret_cast<float4*>(base + r * D + element(mt)) =
                  make_float4(o[mt][nt][e], o[mt][nt][e + 2], o[mt + 1][nt][e], o[mt + 1][nt][e + 2]);
            if (g == 0) {
              base[refs + r] = low[nt][e];
              base[sums + r] = sum[nt][e];
            }
          }
      };
      if (!whole) {
        TreePlace tree;
        if (step0 == 0)
          tree.begin(worker, 1 + static_cast<int32_t>((n_steps - end + share - 1) / share));
        else
          tree.go_on(worker, share, in_unit, n_steps, kUnitCost);
        auto part_of = [&](int32_t wk) {
          return w.part + ((static_cast<int64_t>(wk) * w.hw + hw) * 2 + (wk == tree.worker0 ? 1 : 0)) * static_cast<int64_t>(NQ * (D + 2));
        };
        auto same = [](int col) -> int64_t { return col; };
        whole = true;
        while (tree.up()) {
          int32_t other;
          if (!meet(w.nodes + static_cast<int64_t>(tree.node) * w.hw + hw, worker, &other,
                    [&]() { leave(part_of(worker), NQ * D, NQ * (D + 1), same, NQ); })) {
            whole = false;
            break;
          }
          add(part_of(other), NQ * D, NQ * (D + 1), same, tree.left);
          tree.joined();
        }
      }
      auto row_at = [&](int col) -> int64_t {
        const int32_t f = f0 + min(col, nf - 1);
        return (q.row0 + f / a.G) * a.Q + h * a.G + f % a.G;
      };
      if (whole && a.state) {
        leave(a.state, a.state_rows * D, a.state_rows * (D + 1), row_at, nf);
        whole = false;
      } else if (whole && a.prior && __ldcg(b.from + s) != 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        add(a.prior, a.state_rows * D, a.state_rows * (D + 1), row_at, false);
      }
    }
    if (whole) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = nt * 8 + 2 * c + e;
          const int32_t f = f0 + col;
          const float inv = sum[nt][e] == 0.0f ? 0.0f : rcp(sum[nt][e]);
          bool bad = !(sum[nt][e] <= 3.402823466e38f);
          const int64_t r = q.row0 + f / a.G;
          const int32_t qh = h * a.G + f % a.G;
#pragma unroll
          for (int mt = 0; mt < Sh::kMT; ++mt) {
            const float y0 = o[mt][nt][e] * inv, y1 = o[mt][nt][e + 2] * inv;
            bad = bad || !(fabsf(y0) <= 3.402823466e38f) || !(fabsf(y1) <= 3.402823466e38f);
            if (col < nf) {
              const uint32_t y = a.type == KV_TYPE_BF16 ? pack_b(y0, y1) : pack_h(y0, y1);
              uint16_t* out = static_cast<uint16_t*>(a.out) + (r * a.Q + qh) * D + element(mt);
              if (w.out_wide) {
                *reinterpret_cast<uint32_t*>(out) = y;
              } else {
                out[0] = static_cast<uint16_t>(y);
                out[1] = static_cast<uint16_t>(y >> 16);
              }
            }
          }
          if (a.lse && g == 0 && col < nf)
            a.lse[r * a.Q + qh] = sum[nt][e] == 0.0f ? -INFINITY : (low[nt][e] + log2f(sum[nt][e])) * kLn2;
          // columns with anything not finite are done again, key by key
          const uint32_t again = __ballot_sync(kFull, bad && col < nf);
          if (again) {
            __syncwarp();
            for (int k = 0; k < 4; ++k)
              if (again & (0x11111111u << k)) {
                const int32_t ff = f0 + nt * 8 + 2 * k + e;
                attend_row<C>(p, b, a, s, q.a + ff / a.G, q.row0 + ff / a.G, h * a.G + ff % a.G, &bits);
              }
          }
        }
    } else if constexpr (!SHARED) {
      const int slot = step0 == 0 ? 1 : 0;
      float* part = w.part + ((static_cast<int64_t>(worker) * w.hw + hw) * 2 + slot) * static_cast<int64_t>(NQ * (D + 2));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = nt * 8 + 2 * c + e;
#pragma unroll
          for (int mt = 0; mt < Sh::kMT; mt += 2)
            *reinterpret_cast<float4*>(part + col * D + element(mt)) =
                make_float4(o[mt][nt][e], o[mt][nt][e + 2], o[mt + 1][nt][e], o[mt + 1][nt][e + 2]);
          if (g == 0) {
            part[NQ * D + col] = high[nt][e] == -INFINITY ? kNoRef : low[nt][e];
            part[NQ * (D + 1) + col] = sum[nt][e];
          }
        }
      if (slot == 1)
        rec = SplitRecord{s, q.a, f0, nf, group, worker + static_cast<int32_t>((n_steps - end + share - 1) / share), q.row0};
    }
    left -= w.whole ? 1 : end - step0 + kUnitCost;  // and the head of the next unit

    // ---- the next unit
    step0 = 0;
    if (left > 0 && ++group == n_groups) {
      group = 0;
      ++tile;
      while (tile >= tiles_of(q)) {
        tile = 0;
        if (++s >= b.n_seqs) break;
        int err = 0;
        q = seq_of<SHARED>(p, b, s, err);
      }
      if (s >= b.n_seqs) break;
      span = span_of(q, s, tile);
    }
  }
  if (!SHARED && worker < w.n_workers && hw == 0 && lane == 0) w.rec[worker] = rec;
  store_bits(p, bits);
  // whoever waits for this kernel waits for those before it
  if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class C, int D, int NT, bool SHARED>
cudaError_t launch(const DevPool& p, const Batch& b, const AttendArgs& a, Split w, bool after, cudaStream_t s) {
  using Sh = FewShape<C, D>;
  constexpr bool kOne = std::is_same_v<C, CodeE4M3> || std::is_same_v<C, CodeE2M1>;  // one part will do for a bf16 output
  const bool one = kOne && a.type == KV_TYPE_BF16;
  auto kernel = p.ps % 16 == 0
                    ? (one ? k_attend_few<C, D, NT, true, !kOne, SHARED> : k_attend_few<C, D, NT, true, true, SHARED>)
                    : (one ? k_attend_few<C, D, NT, false, !kOne, SHARED> : k_attend_few<C, D, NT, false, true, SHARED>);
  const int smem = kFewWarps * ((w.deep ? Sh::kDeep : Sh::kStages) * Sh::kStage + Sh::queries(NT));
  if (after) return launch_overlapped(kernel, dim3(w.blocks), kFewBlock, smem, s, p, b, a, w);
  kernel<<<w.blocks, kFewBlock, smem, s>>>(p, b, a, w);
  return cudaGetLastError();
}

template <class C, int D, int NT, bool SHARED>
cudaError_t prepare_one(bool p16) {
  using Sh = FewShape<C, D>;
  constexpr int kBytes = kFewWarps * (Sh::kDeep * Sh::kStage + Sh::queries(NT));
  auto set = [](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes); };
  cudaError_t e = set(p16 ? k_attend_few<C, D, NT, true, true, SHARED> : k_attend_few<C, D, NT, false, true, SHARED>);
  if constexpr (std::is_same_v<C, CodeE4M3> || std::is_same_v<C, CodeE2M1>)
    if (e == cudaSuccess) e = set(p16 ? k_attend_few<C, D, NT, true, false, SHARED> : k_attend_few<C, D, NT, false, false, SHARED>);
  return e;
}

}  // namespace

template <class C, bool SHARED>
cudaError_t launch_few(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, int nt, bool after,
                       cudaStream_t s) {
  if (a.D == 64) return nt == 1 ? launch<C, 64, 1, SHARED>(p, b, a, w, after, s) : launch<C, 64, 2, SHARED>(p, b, a, w, after, s);
  return nt == 1 ? launch<C, 128, 1, SHARED>(p, b, a, w, after, s) : launch<C, 128, 2, SHARED>(p, b, a, w, after, s);
}

template <class C, bool SHARED>
cudaError_t prepare_few(int32_t D, bool p16) {
  const cudaError_t e = D == 64 ? prepare_one<C, 64, 1, SHARED>(p16) : prepare_one<C, 128, 1, SHARED>(p16);
  return e != cudaSuccess ? e : D == 64 ? prepare_one<C, 64, 2, SHARED>(p16) : prepare_one<C, 128, 2, SHARED>(p16);
}

// One pair of instances a file (kv_attend_few_*.cu), so that they compile side by side.
#define GTKV_FEW_INSTANCES(C, SHARED)                                                                                     \
  template cudaError_t launch_few<C, SHARED>(const DevPool&, const Batch&, const AttendArgs&, const Split&, int, bool,  \
                                             cudaStream_t);                                                            \
  template cudaError_t prepare_few<C, SHARED>(int32_t, bool);

}  // namespace gtkv
