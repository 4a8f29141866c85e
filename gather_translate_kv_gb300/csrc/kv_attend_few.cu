// Attention of few rows a sequence (decode steps, drafted tokens): at most 16
// rows (8-bit caches: 32) on average, a row being a (token, query head) pair of one KV head, in
// tiles of 8 or 16; a sequence with more takes several tiles. Every key and
// value is read once and meets a handful of rows, so the bound is memory; the
// work is laid out so that nothing stands between the loads.
//
// One warp owns one KV head over its own run of keys, 16 keys a step, and never
// talks to another warp. Both products run as mma m16n8k16 with the CACHE as
// the 16-row operand, S^T = K Q^T and O^T = V^T P^T, rows as the 8 (or 16)
// columns, so 4 query heads fill half of an instruction instead of a quarter.
// The order of the summed index is free, so operand registers are filled from
// whole 16-byte pieces of the rows as they lie in the cache: lane (g, c) =
// (lane / 4, lane % 4) takes pieces of keys g and g + 8 for K, and its eighth
// of the elements of keys 2c, 2c + 1, 2c + 8, 2c + 9 for V, where byte
// permutes pair up two keys. Rows come by cp.async into a ring of the warp's
// own, whole rows an instruction. No transpose, no bank conflict, no barrier. Codes become fp16 (exact) on the
// way into the registers; P^T comes out of the score registers by movmatrix.
//
// Softmax: the running reference m moves only when a score exceeds it by
// 2^8 (a vote per step), so the common step has no shuffle. Weights are
// 2^(t - m), t = score * log2(e) + log2(value scale): the scale of an 8-bit
// value is part of its weight, so that weights stay in one range, and the
// denominator adds weight / scale. Weights meet the values as the sum of two 16-bit
// parts and keep 16 bits (bf16) or 22 (fp16, lifted by 2^6 so that 2^-30 of the largest
// still counts): the result's error is then the output's own rounding and no more, where one part
// alone adds 40 % to it (fp16 output, 4096 keys, root mean square: 5.39e-6 and 7.54e-6). Under
// 16-bit caches the second product is free, memory being the bound. Of 8-bit caches read
// into bf16, whose 8 bits hide the 11 of one fp16 part (8.73e-5 and 8.79e-5), the weights are
// one part: drafts take 364 us so and 405 with two. Queries for 8-bit caches are fp16 after a power-of-two scaling per row, exact for all
// bits that matter (2^-29 of the row's largest).
//
// Measured: 256 sequences of 4096 tokens (bf16, 8 KV heads of 128, 4.3 GB) 680 to 698
// us from one GPU to another, 91 to 93 % of the copy rate; 40 sequences of 9 to 40 961 tokens with drafts
// (8-bit, 1.68 GB) 364 us, 68 %, bound by latency inside a warp (codes into fp16, products,
// weights, one after the other) with three warps a scheduler; one sequence of 203 tokens 14 us, latency.
//
// Workers (as many warps as share a step's heads) take equal shares of all
// steps of the batch (kv_attend_split.cuh); units cut at a border are joined by
// k_attend_join from 32-bit partial sums in the workspace.
#include "kv_attend_launch.h"
#include "kv_attend_split.cuh"

namespace gtkv {

namespace {

constexpr int kFewWarps = 4;
constexpr int kFewBlock = 32 * kFewWarps;
constexpr int kFewBlocksPerSM = 4;  // at most
constexpr int kUnitCost = 2;  // steps' worth of a unit's queries and output
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
  static constexpr int kSize = FewType<C>::kSize;
  static constexpr int kRow = D * kSize;      // bytes of a head's row
  static constexpr int kKC = kRow / 64;       // 16-byte pieces of a key that a lane holds
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
  static constexpr int kMeta = 144;           // 32 scales, the mask of live keys
  static constexpr int kStage = 2 * kK + kMeta;
  // Stages of a warp's ring: as many as shared memory holds with all the
  // blocks that fit an SM, or, for calls of one block an SM, whose time is latency, six.
  static constexpr int kStages = kRow >= 256 ? 2 : kRow >= 128 ? 3 : 6;
  static constexpr int kDeep = 6;
  static constexpr int kKS = D / 16;          // k16 steps of the score product
  static constexpr int kMT = D / 16;          // 16-element tiles of the output
};

// P16: the page size is a multiple of 16, so a step's keys share a page and a
// lane looks up the pages of 32 steps ahead at once; otherwise every key's entry is
// read on its own, one step ahead. 256 x 4096 tokens in pages of 16, bf16, on one GPU: 686 us against
// 698 by keys; 8-bit, pages of 32: the same within 1 %.
// Resident blocks: shared memory for 256-byte rows, registers for 16 columns allow three.
constexpr int few_blocks(int row, int nt) { return row >= 256 || nt > 1 ? 3 : kFewBlocksPerSM; }

// TWO: weights in two parts.
template <class C, int D, int NT, bool P16, bool TWO>
__global__ void __launch_bounds__(kFewBlock, few_blocks(FewShape<C, D>::kRow, NT))
    k_attend_few(DevPool p, Batch b, AttendArgs a, Split w) {
  using Sh = FewShape<C, D>;
  constexpr bool kE4M3 = std::is_same_v<C, CodeE4M3>;
  constexpr float kLift = FewType<C>::kLift;
  constexpr int NQ = 8 * NT;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ ShareStart loc[kFewWarps];
  __shared__ int64_t tmp[kFewWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int kw = kFewWarps / w.hw;             // workers of the block
  const int wk = warp / w.hw;                  // this warp's worker in the block
  const int hw = warp - wk * w.hw;             // its head of the worker's group
  const int32_t n_groups = a.H / w.hw;
  int bits = 0;

  auto tiles_of = [&](const Seq& q) { return q.n == 0 || q.n > w.max_new ? 0 : (q.n * a.G + NQ - 1) / NQ; };
  auto span_of = [&](const Seq& q, int32_t t) {
    const int32_t f0 = t * NQ, f1 = min(f0 + NQ, q.n * a.G);
    return key_span<16>(a, q.a + f0 / a.G, q.a + (f1 - 1) / a.G);
  };
  const int32_t worker0 = static_cast<int32_t>(blockIdx.x) * kw;
  const int64_t share = find_shares<kFewBlock, kFewWarps>(
      b.n_seqs, worker0, w.n_workers, w.min_share, loc, tmp, [&](int32_t s) -> int64_t {
        int err = 0;
        const Seq q = seq_of(p, b, s, err);
        if (blockIdx.x == 0) bits |= err;
        int64_t n = 0;
        if (w.whole) return static_cast<int64_t>(tiles_of(q)) * n_groups;
        for (int32_t t = 0; t < tiles_of(q); ++t) n += span_of(q, t).steps() + kUnitCost;
        return n * n_groups;
      });
  const int32_t worker = worker0 + wk;
  SplitRecord rec{-1, 0, 0, 0, 0, 0, 0};
  ShareStart at = loc[wk];
  if (worker >= w.n_workers) at.s = -1;

  // The warp's ring. A row's 16-byte pieces are permuted within it so that the
  // reads below meet no bank twice: K's piece p of row r sits at p ^ 4 (r % 2),
  // V's at p ^ 2 (r / 2 % 4) (64-byte rows: p and p ^ (r / 2 % 4)).
  const int cr = lane / Sh::kLPR, cp = lane % Sh::kLPR;  // row of a round and piece that the lane copies
  const uint32_t put_k = cr * Sh::kRow + (Sh::kRow > 64 ? cp ^ (cr & 1) * 4 : cp) * 16;
  const uint32_t put_v = cr * Sh::kRow + (Sh::kRow >= 256 ? cp : Sh::kRow > 64 ? cp ^ (cr >> 1) * 2 : cp ^ (cr >> 1 & 3)) * 16;
  const uint32_t get_k = g * Sh::kRow + (Sh::kRow > 64 ? c ^ (g & 1) * 4 : c) * 16;  // ^ 64 ch, + 8 rows
  const uint32_t get_v = 2 * c * Sh::kRow + (Sh::kRow > 64 ? (g ^ 2 * c) * 16 : ((g >> 1) ^ c) * 16 + (g & 1) * 8);
  auto key_at = [](int kk) { return ((kk & 1) + 8 * (kk >> 1)) * Sh::kRow; };  // of keys 2c, 2c + 1, 2c + 8, 2c + 9
  const int stages = w.deep ? Sh::kDeep : Sh::kStages;
  const uint32_t ring0 = shared_u32(ring) + warp * stages * Sh::kStage;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.base);
  const int32_t row_bytes = static_cast<int32_t>(p.vpr * 16);

  int64_t left = at.s < 0 ? 0 : share;
  int32_t s = at.s, tile = 0, group = 0;
  int32_t step0 = 0;
  Seq q{0, 0, 0};
  KeySpan span{0, 0, 0};
  if (left > 0) {  // the unit and step where the share begins
    int err = 0;
    q = seq_of(p, b, s, err);
    int64_t off = at.off;
    for (;;) {
      span = span_of(q, tile);
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
      left -= in < kUnitCost ? kUnitCost - in : 0;
    }
  }

  while (left > 0) {
    const int32_t n_steps = span.steps();
    const int32_t end = !w.whole && left < n_steps - step0 ? step0 + static_cast<int32_t>(left) : n_steps;
    const int32_t h = group * w.hw + hw;
    const int32_t f0 = tile * NQ;
    const int32_t nf = min(NQ, q.n * a.G - f0);  // rows of the tile
    const int32_t i0 = q.a + f0 / a.G, i1 = q.a + (f0 + nf - 1) / a.G;

    // ---- issue of a step's loads
    // the lane's piece of row 0 of a page, in the layer's block of keys; rows are below 2^31
    const uint8_t* from = pool + (2 * static_cast<int64_t>(a.layer) * p.ps + cr) * row_bytes + h * Sh::kRow + cp * 16;
    const int32_t page_rows = static_cast<int32_t>(p.stride), ps = static_cast<int32_t>(p.ps);
    const float* scale_at = kE4M3 ? a.scales + 2 * static_cast<int64_t>(a.layer) * a.H + h : nullptr;  // of page 0
    const int32_t page_scales = p.blocks * a.H;
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
          if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + 2 * Sh::kK + 128), "r"(live) : "memory");
        }
        if constexpr (kE4M3 && P16) {  // one scale of K (lane 0) and one of V (lane 1)
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
    for (int i = 0; i < stages - 1; ++i) issue(step0 + i, i);

    // ---- the queries, while the first loads are in flight
    uint32_t qf[NT][Sh::kKS][2];
    float cq[NT][2];
    int32_t pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int32_t f = f0 + nt * 8 + g;
      const bool ok = nt * 8 + g < nf;
      const int64_t q0 = ok ? (q.row0 + f / a.G) * a.q_stride + static_cast<int64_t>(h * a.G + f % a.G) * D : 0;
      float row_c = a.scale_log2;
      constexpr int EC = 16 / Sh::kSize;  // elements of a lane's piece
      if constexpr (!kE4M3) {
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
        float x[Sh::kKC][EC];
        float amax = 0.0f;
#pragma unroll
        for (int ch = 0; ch < Sh::kKC; ++ch)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + q0 + ch * 64 + c * 16 + half * 8;
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
              x[ch][half * 8 + 2 * k] = f.x;
              x[ch][half * 8 + 2 * k + 1] = f.y;
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
        for (int ch = 0; ch < Sh::kKC; ++ch)
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            qf[nt][ch * 4 + wd][0] = pack_h(x[ch][4 * wd] * up, x[ch][4 * wd + 1] * up);
            qf[nt][ch * 4 + wd][1] = pack_h(x[ch][4 * wd + 2] * up, x[ch][4 * wd + 3] * up);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // columns 2c and 2c + 1 of the scores
        cq[nt][e] = __shfl_sync(kFull, row_c, (2 * c + e) * 4);
        pos[nt][e] = q.a + min(f0 + nt * 8 + 2 * c + e, f0 + nf - 1) / a.G;
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
    for (int32_t i = step0; i < end; ++i) {
      {
        int ahead = stage + stages - 1;
        if (ahead >= stages) ahead -= stages;
        issue(i + stages - 1, ahead);
      }
      if (w.deep)
        copy_wait<Sh::kDeep - 1>();
      else
        copy_wait<Sh::kStages - 1>();
      __syncwarp();
      const uint32_t st = ring0 + stage * Sh::kStage;
      const uint32_t live = whole_stages >> stage & 1 ? 0xffffu : lds32(st + 2 * Sh::kK + 128);
      const int32_t j0 = span.block(i) * 16;

      // ---- scores
      // two sums for one tile of columns, so that products wait half as long for one another
      constexpr bool kTwo = NT == 1;
      float x[NT][4], x2[NT][4];
#pragma unroll
      for (int ch = 0; ch < Sh::kKC; ++ch) {
        const uint4 u = lds128(st + (get_k ^ ch * 64)), v = lds128(st + (get_k ^ ch * 64) + 8 * Sh::kRow);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
        if constexpr (kE4M3) {
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            const uint32_t a0 = codes_lo(uu[wd]), a1 = codes_lo(vv[wd]), a2 = codes_hi(uu[wd]), a3 = codes_hi(vv[wd]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<C>(kTwo && wd & 1 ? x2[nt] : x[nt], a0, a1, a2, a3, qf[nt][ch * 4 + wd][0], qf[nt][ch * 4 + wd][1],
                     ch * 4 + wd < 1 + kTwo);
          }
        } else {
#pragma unroll
          for (int wd = 0; wd < 2; ++wd)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<C>(kTwo && wd & 1 ? x2[nt] : x[nt], uu[2 * wd], vv[2 * wd], uu[2 * wd + 1], vv[2 * wd + 1],
                     qf[nt][ch * 2 + wd][0], qf[nt][ch * 2 + wd][1], ch * 2 + wd < 1 + kTwo);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kTwo) x[nt][e] += x2[nt][e];

      // ---- weights; x[.][0], [1]: key g, columns 2c, 2c + 1; [2], [3]: key g + 8
      float lv[2] = {0.0f, 0.0f}, iv[2] = {1.0f, 1.0f}, sk[2] = {1.0f, 1.0f};
      if constexpr (kE4M3) {
        if constexpr (P16) {
          const uint2 kv = lds64(st + 2 * Sh::kK);
          sk[0] = sk[1] = __uint_as_float(kv.x);
          lv[0] = lv[1] = lg2(__uint_as_float(kv.y));
          iv[0] = iv[1] = rcp(__uint_as_float(kv.y));
        }
#pragma unroll
        for (int e = 0; e < (P16 ? 0 : 2); ++e) {
          sk[e] = __uint_as_float(lds32(st + 2 * Sh::kK + (g + 8 * e) * 4));
          const float sv = __uint_as_float(lds32(st + 2 * Sh::kK + 64 + (g + 8 * e) * 4));
          lv[e] = lg2(sv);
          iv[e] = rcp(sv);
        }
      }
      const bool mask = live != 0xffffu || j0 + 15 > i0 || (a.window && j0 <= i1 - a.window);
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float t = kE4M3 ? fmaf(x[nt][e], cq[nt][e & 1] * sk[e >> 1], lv[e >> 1] - low[nt][e & 1])
                          : fmaf(x[nt][e], cq[nt][e & 1], -low[nt][e & 1]);
          if (mask) {
            const int key = g + 8 * (e >> 1);
            if (!(live >> key & 1) || !in_sight(a, pos[nt][e & 1], j0 + key)) t = -INFINITY;
          }
          x[nt][e] = t;
          over = over || t > high[nt][e & 1];
        }
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(x[nt][e], x[nt][e + 2]);
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            if (m > kLift || (m > -INFINITY && high[nt][e] == -INFINITY)) {  // the maximum becomes the reference
              const float up = m - kLift;
              const float keep = high[nt][e] == -INFINITY ? 0.0f : ex2(-up);
              low[nt][e] += up;
              high[nt][e] = kLift + 8.0f;
              x[nt][e] -= up;
              x[nt][e + 2] -= up;
              sum[nt][e] *= keep;
#pragma unroll
              for (int mt = 0; mt < Sh::kMT; ++mt) {
                o[mt][nt][e] *= keep;
                o[mt][nt][e + 2] *= keep;
              }
            }
          }
      }
      uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = ex2(x[nt][e]);
          // a dead key adds nothing, whatever its zero-filled scale's inverse is
          if constexpr (kE4M3 && !P16)
            sum[nt][e & 1] += live >> (g + 8 * (e >> 1)) & 1 ? y[e] * iv[e >> 1] : 0.0f;
          else if constexpr (!kE4M3)
            sum[nt][e & 1] += y[e];
        }
        if constexpr (kE4M3 && P16) {
          if (live) {
            sum[nt][0] = fmaf(y[0] + y[2], iv[0], sum[nt][0]);
            sum[nt][1] = fmaf(y[1] + y[3], iv[0], sum[nt][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          constexpr bool kBf16 = std::is_same_v<C, __nv_bfloat16>;
          const uint32_t hi = pack16<kBf16>(y[2 * e], y[2 * e + 1]);
          pb[nt][e] = transpose8(hi);
          if constexpr (TWO) {
            const float2 h = unpack16<kBf16>(hi);
            pl[nt][e] = transpose8(pack16<kBf16>(y[2 * e] - h.x, y[2 * e + 1] - h.y));
          }
        }
      }

      // ---- values: registers of keys 2c, 2c + 1 (a0, a1) and 2c + 8, 2c + 9 (a2, a3)
      auto tile_mma = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma<C>(o[mt][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          if constexpr (TWO) mma<C>(o[mt][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
        }
      };
      constexpr int VC = Sh::kVC;
      constexpr int VW = Sh::kVB >= 16 ? 4 : 2;             // words of a piece
#pragma unroll
      for (int ch = 0; ch < VC; ++ch) {
        uint32_t v[4][VW];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (VW == 4) {
            const uint4 u = lds128(st + Sh::kK + get_v + key_at(kk) + ch * 128);
            v[kk][0] = u.x, v[kk][1] = u.y, v[kk][2] = u.z, v[kk][3] = u.w;
          } else {
            const uint2 u = lds64(st + Sh::kK + get_v + key_at(kk));
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
          if (keys) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (keys >> (g + 8 * (e >> 1)) & 1 && x[nt][e] != -INFINITY) sum[nt][e & 1] = NAN;
          }
        }
#pragma unroll
        for (int wd = 0; wd < VW; ++wd) {
          if constexpr (kE4M3) {
            const uint32_t x0 = __byte_perm(v[0][wd], v[1][wd], 0x5140), y0 = __byte_perm(v[0][wd], v[1][wd], 0x7362);
            const uint32_t x1 = __byte_perm(v[2][wd], v[3][wd], 0x5140), y1 = __byte_perm(v[2][wd], v[3][wd], 0x7362);
            tile_mma(ch * 8 + 2 * wd, codes_lo(x0), codes_hi(x0), codes_lo(x1), codes_hi(x1));
            tile_mma(ch * 8 + 2 * wd + 1, codes_lo(y0), codes_hi(y0), codes_lo(y1), codes_hi(y1));
          } else {
            tile_mma(ch * 4 + wd, __byte_perm(v[0][wd], v[1][wd], 0x5410), __byte_perm(v[0][wd], v[1][wd], 0x7632),
                     __byte_perm(v[2][wd], v[3][wd], 0x5410), __byte_perm(v[2][wd], v[3][wd], 0x7632));
          }
        }
      }
      if (++stage == stages) stage = 0;
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
    const bool whole = step0 == 0 && end == n_steps;
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
    } else {
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
        q = seq_of(p, b, s, err);
      }
      if (s >= b.n_seqs) break;
      span = span_of(q, tile);
    }
  }
  if (worker < w.n_workers && hw == 0 && lane == 0) w.rec[worker] = rec;
  store_bits(p, bits);
}

template <class C, int D, int NT>
cudaError_t launch(const DevPool& p, const Batch& b, const AttendArgs& a, Split w, cudaStream_t s) {
  using Sh = FewShape<C, D>;
  constexpr bool kOne = std::is_same_v<C, CodeE4M3>;  // one part will do for a bf16 output
  const bool one = kOne && a.type == KV_TYPE_BF16;
  auto kernel = p.ps % 16 == 0 ? (one ? k_attend_few<C, D, NT, true, !kOne> : k_attend_few<C, D, NT, true, true>)
                               : (one ? k_attend_few<C, D, NT, false, !kOne> : k_attend_few<C, D, NT, false, true>);
  kernel<<<w.blocks, kFewBlock, kFewWarps * (w.deep ? Sh::kDeep : Sh::kStages) * Sh::kStage, s>>>(p, b, a, w);
  return cudaGetLastError();
}

template <class C>
cudaError_t launch_c(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, int nt, cudaStream_t s) {
  if (a.D == 64) return nt == 1 ? launch<C, 64, 1>(p, b, a, w, s) : launch<C, 64, 2>(p, b, a, w, s);
  return nt == 1 ? launch<C, 128, 1>(p, b, a, w, s) : launch<C, 128, 2>(p, b, a, w, s);
}

template <class C, int D, int NT>
cudaError_t prepare_one(bool p16) {
  constexpr int kBytes = kFewWarps * FewShape<C, D>::kDeep * FewShape<C, D>::kStage;
  auto set = [](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes); };
  cudaError_t e = set(p16 ? k_attend_few<C, D, NT, true, true> : k_attend_few<C, D, NT, false, true>);
  if constexpr (std::is_same_v<C, CodeE4M3>)
    if (e == cudaSuccess) e = set(p16 ? k_attend_few<C, D, NT, true, false> : k_attend_few<C, D, NT, false, false>);
  return e;
}

template <class C>
cudaError_t prepare_c(int32_t D, bool p16) {
  const cudaError_t e = D == 64 ? prepare_one<C, 64, 1>(p16) : prepare_one<C, 128, 1>(p16);
  return e != cudaSuccess ? e : D == 64 ? prepare_one<C, 64, 2>(p16) : prepare_one<C, 128, 2>(p16);
}

constexpr int kWhole = 24;    // steps up to which units are not cut where they fill the GPU; a third of it where they do not
constexpr int kMinShare = 4;  // steps of 16 keys below which a worker's share is not cut

int heads_of_worker(int32_t H) { return H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1; }

}  // namespace

cudaError_t prepare_attend_few(int32_t D, bool e4m3, bool p16) {
  if (e4m3) return prepare_c<CodeE4M3>(D, p16);
  const cudaError_t e = prepare_c<__half>(D, p16);
  return e == cudaSuccess ? prepare_c<__nv_bfloat16>(D, p16) : e;
}

int64_t attend_few_workspace(int32_t D, int sm_count) {
  const int64_t warps = static_cast<int64_t>(sm_count) * kFewBlocksPerSM * kFewWarps;
  return split_record_bytes(warps) + warps * 2 * 16 * (D + 2) * 4;
}

cudaError_t launch_attend_few(const DevPool& p, const Batch& b, const AttendArgs& a, bool e4m3, int32_t max_new,
                              void* workspace, int sm_count, Split* out, cudaStream_t s) {
  Split w{};
  w.hw = heads_of_worker(a.H);
  w.max_new = max_new;
  const int kw = kFewWarps / w.hw;
  // one tile of 8 columns when the sequences' rows of a KV head fit on average, else 16 (4 rows, 256 x 4096 tokens, on one
  // GPU: 686 us with 8 columns, 803 with 16)
  const int nt = b.n_rows * a.G <= 8 * static_cast<int64_t>(b.n_seqs) ? 1 : 2;
  // steps of one unit at most, and of all units
  int64_t most = static_cast<int64_t>(b.max_pages) * p.ps / 16 + 1;
  if (a.window) {
    const int64_t seen = (static_cast<int64_t>(a.window) + 16) / 16 + 2 + (a.sinks + 15) / 16;
    most = seen < most ? seen : most;
  }
  const int64_t tiles = (b.n_rows * a.G) / (8 * nt) + b.n_seqs;  // row tiles of all sequences
  int64_t cap = static_cast<int64_t>(sm_count) * few_blocks(a.D * (e4m3 ? 1 : 2), nt) * kw;
  // units that are short anyway are never cut, and then there is nothing to join: 512 sequences of 300 tokens (8-bit,
  // D = 64) 52 us against 63 cut, 4 of 128 tokens 15.0 against 15.2
  w.whole = most <= (tiles * (a.H / w.hw) >= cap ? kWhole : kWhole / 3);
  const int64_t all = (w.whole ? 1 : most + kUnitCost) * tiles * (a.H / w.hw);
  cap = cap < kMaxWorkers ? cap : kMaxWorkers;
  w.min_share = w.whole ? 1 : kMinShare;
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
  *out = w;
  if (e4m3) return launch_c<CodeE4M3>(p, b, a, w, nt, s);
  if (a.type == KV_TYPE_BF16) return launch_c<__nv_bfloat16>(p, b, a, w, nt, s);
  return launch_c<__half>(p, b, a, w, nt, s);
}

}  // namespace gtkv
