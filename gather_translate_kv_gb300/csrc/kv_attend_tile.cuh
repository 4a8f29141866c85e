// Attention of many rows a sequence (prompts, chunks, long drafts) on the 5th-generation tensor cores.
//
// A block owns a unit: up to 256 rows of one KV head of a sequence, a row being a (token, query head of the group)
// pair, as two tiles of 128 rows. For each 128 keys
//   S_w = Q_w K^T   (tile w of rows; both operands in shared memory)
//   P_w = 2^(t - m) (softmax warps; written over S_w in tensor memory)
//   O_w += P_w V    (P_w from tensor memory, V as the M/N-major operand)
// with S_0, S_1, O_0, O_1 filling the 512 columns of tensor memory. The two tiles alternate: while four warps turn S_0
// into P_0 the tensor cores work on tile 1 and the other way round, which is what bounds the kernel: per 128 keys and
// tile 4 * 128 * 128 * D operations (6 with weights in two parts) on the tensor cores against 128 * 128 exponentials.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, one row a thread (no shuffles). Warps 8-11: loaders; they look up the
// pages, copy keys and values into the 128-byte-swizzled operand layout with cp.async (16-bit caches) or through
// registers, turning codes into fp16 (8-bit and 4-bit caches), and zero what is no live token. Pages of any size end
// anywhere in a tile, so keys are placed row by row rather than by a tensor map. Warp 12 issues the products.
//
// The running reference m of a row moves only when a tile's maximum exceeds it by 2^8; only then is O read back and
// scaled. A first pass over the scores finds that maximum, a second turns them into weights in place. Weights meet the
// values as two parts of the cache's 16-bit type (bf16, or fp16 lifted by 2^6 for fp16 and 8-bit caches), rounded and
// what the rounding left, so that the result's error is the output's own rounding: 1.479e-4 (root mean square, prompts
// of 2048 tokens in bf16), as the formula in 32 bits has it, where one part gave 1.903e-4 for 582 us instead of 757. Of
// 8-bit and 4-bit caches read into bf16, whose 8 bits hide fp16's 11, one part is enough (7.45e-5 and 7.39e-5; chunks
// of ~1000 tokens in 8 bits 452 us, with two parts 561, in 4 bits 440 and 524). Denominators add the 32-bit weights.
// The scale of an 8-bit value is part of its weight, t = score * log2(e) + log2(scale), and the denominator adds weight
// / scale. Queries for 8-bit caches become fp16 after a power-of-two scaling per row.
//
// Work is cut as in kv_attend_split.cuh, 128 keys a step.
//
// Measured: 16 prompts of 2048 tokens (bf16, 8 KV and 32 query heads of 128, 550 GFLOP) 752 to 766 us, 38 % of the
// measured cuBLAS burst; 4 of 8192 tokens 2240 us; the 16 prompts in 8 bits 952, in 4 bits 890 us. Chunks of ~1000
// tokens on 6001 to 8190: 16-bit 457 us, 8-bit 451, 4-bit 440, so that what bounds them is no longer the loaders but
// the chain from scores through weights to the second product. The kernel is at the limit of 128 registers a thread,
// and the code that its warps run through in a step is larger than the instruction caches near them: where loops of the
// loaders (3 to 5 %) and of the softmax (7 to 15 %) are written out only in part it is faster (figures beside them). A
// unit costs ~13 us beside its steps, for its queries, masked last step and output.
#pragma once

#include "kv_attend_split.cuh"
#include "kv_umma.cuh"

namespace gtkv {

namespace {

constexpr int kTileThreads = 416;  // 13 warps
constexpr int kRows = kTileRows, kKeys = kTileKeys;
constexpr int kSlots = 8;          // steps whose scales and masks are kept
constexpr int kUnitCost = kTileUnitCost;

// What the softmax warps need to know of a step's keys.
struct Masks {
  uint32_t live[4];  // keys that are tokens
  uint32_t nan[4];   // keys whose value had elements that are not finite (zeroed)
};
struct Scales {
  float ks[kKeys];  // scale of the key
  float lv[kKeys];  // log2 of the value's scale
  float iv[kKeys];  // its inverse
};

// Tiles of keys and values pass through one ring of operand tiles, K of step n
// as tile 2n and V as tile 2n + 1; codes of 8-bit caches through a ring of raw tiles before it.
template <class C, int D>
struct TileSmem {
  static constexpr bool kE4M3 = std::is_same_v<C, CodeE4M3>, kE2M1 = std::is_same_v<C, CodeE2M1>;
  static constexpr bool kCodes = kE4M3 || kE2M1;
  static constexpr int kOperand = 128 * D * 2;  // a tile of Q, K or V
  static constexpr int kRing = D == 64 ? 8 : kE4M3 ? 3 : kE2M1 ? 4 : 5;
  static constexpr int kRawRing = kCodes ? 3 : 0;
  static constexpr int kRawTile = kOperand / (kE2M1 ? 4 : 2);
  static constexpr int kQ = 0;  // two tiles
  static constexpr int kTiles = 2 * kOperand;
  static constexpr int kRaw = kTiles + kRing * kOperand;
  // 4-bit caches: scale bytes as they were copied, of this step and the next: per key K's and V's
  static constexpr int kRawScale = kE2M1 ? D / 16 : 0;
  static constexpr int kRawScales = kRaw + kRawRing * kRawTile;
  static constexpr int kMasks = kRawScales + 2 * 128 * 2 * kRawScale;
  static constexpr int kScales = kMasks + kSlots * static_cast<int>(sizeof(Masks));
  static constexpr int kQScale = kScales + (kE4M3 ? kSlots * static_cast<int>(sizeof(Scales)) : 0);
  static constexpr int kBar = kQScale + (kCodes ? 2 * kRows * 4 : 0);  // of this unit's and the next one's rows
  enum Bar { kFull, kFree = kFull + kRing, kQFull = kFree + kRing, kQFree = kQFull + 2, kSFull = kQFree + 2,
             kPReady = kSFull + 2, kODone = kPReady + 2, kDrain = kODone + 2, kBars };
  static constexpr int kMisc = kBar + kBars * 8;   // tensor memory address, stop word
  static constexpr int kBytes = kMisc + 16 + 1024;  // + room to align to the swizzle's 1024 bytes
};
static_assert(TileSmem<__half, 128>::kBytes <= 227 * 1024 && TileSmem<CodeE4M3, 128>::kBytes <= 227 * 1024 &&
              TileSmem<CodeE2M1, 128>::kBytes <= 227 * 1024);

// One segment of a block's share: steps [step0, end) of a unit.
struct Segment {
  Seq q;
  KeySpan span;
  int32_t s, tile, h;
  int32_t step0, end;
  int32_t f0, nf;  // rows
  int32_t i0, i1;  // positions of the first and the last
  int32_t in;      // of the share's first unit, what of its line lies before the share
};

template <bool SHARED>
struct TileWalk {
  const DevPool& p;
  const Batch& b;
  const AttendArgs& a;
  const Split& w;
  int64_t left;
  Segment g;

  __device__ __forceinline__ int32_t tiles() const {
    return g.q.n < w.min_new || g.q.n == 0 ? 0 : static_cast<int32_t>((static_cast<int64_t>(g.q.n) * a.G + kRows - 1) / kRows);
  }
  __device__ __forceinline__ void shape() {
    g.f0 = g.tile * kRows;
    g.nf = min(kRows, g.q.n * a.G - g.f0);
    g.i0 = g.q.a + g.f0 / (SHARED ? a.Gp : a.G);
    g.i1 = g.q.a + (g.f0 + g.nf - 1) / (SHARED ? a.Gp : a.G);
    g.span = key_span<kKeys>(a, g.i0, g.i1);
  }
  __device__ __forceinline__ bool cut() {
    if (left <= 0) return false;
    const int32_t n = g.span.steps() - g.step0;
    g.end = g.step0 + static_cast<int32_t>(left < n ? left : n);
    return true;
  }
  // The first segment of a share; false when there is none.
  __device__ bool start(const ShareStart& at, int64_t share) {
    left = at.s < 0 ? 0 : share;
    if (left == 0) return false;
    int err = 0;
    g.s = at.s;
    g.tile = 0;
    g.q = seq_of<SHARED>(p, b, g.s, err);
    int64_t off = at.off;
    for (;;) {
      shape();
      const int64_t n = static_cast<int64_t>(g.span.steps() + kUnitCost) * a.H;
      if (off < n) break;
      off -= n;
      ++g.tile;
    }
    const int32_t unit = g.span.steps() + kUnitCost;
    g.h = static_cast<int32_t>(off / unit);
    const int32_t in = static_cast<int32_t>(off - static_cast<int64_t>(g.h) * unit);
    g.step0 = in < kUnitCost ? 0 : in - kUnitCost;
    g.in = in;
    left -= in < kUnitCost ? kUnitCost - in : 0;
    return cut();
  }
  __device__ bool next() {
    left -= g.end - g.step0 + kUnitCost;  // and the head of the next unit
    if (left <= 0) return false;
    g.step0 = 0;
    if (++g.h == a.H) {
      g.h = 0;
      ++g.tile;
      while (g.tile >= tiles()) {
        g.tile = 0;
        if (++g.s >= b.n_seqs) return false;
        int err = 0;
        g.q = seq_of<SHARED>(p, b, g.s, err);
      }
      shape();
    }
    return cut();
  }
};

// The warp's earlier writes are seen by whoever waits on the barrier.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}

// Byte offset of 16-byte piece `ch` (of D / 8) of row `row` in a swizzled operand tile.
__device__ __forceinline__ uint32_t piece_at(int row, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (128 * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// 16 codes as two pieces of 8 fp16.
__device__ __forceinline__ void decode16(const uint4& v, uint4& lo, uint4& hi) {
  lo = make_uint4(codes_lo(v.x), codes_hi(v.x), codes_lo(v.y), codes_hi(v.y));
  hi = make_uint4(codes_lo(v.z), codes_hi(v.z), codes_lo(v.w), codes_hi(v.w));
}

__device__ __forceinline__ float2 ffma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}

__device__ __forceinline__ float2 fadd2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// P16: the page size is a multiple of 16, so 16 keys share the scales of an 8-bit cache.
// TWO: weights in two parts. SHARED: a pass over prefixes (kv_attend_few.cuh).
template <class C, int D, bool P16, bool TWO, bool SHARED>
__global__ void __launch_bounds__(kTileThreads, 1) k_attend_tile(DevPool p, Batch b, AttendArgs a, Split w) {
  using Sm = TileSmem<C, D>;
  constexpr bool kE4M3 = Sm::kE4M3, kE2M1 = Sm::kE2M1, kCodes = Sm::kCodes;
  constexpr bool kBf16 = std::is_same_v<C, __nv_bfloat16>;
  constexpr float kLift = kBf16 ? 0.0f : 6.0f;
  constexpr int kPieces = D / 8;  // 16-byte pieces of a 16-bit row
  extern __shared__ uint8_t dyn[];
  __shared__ ShareStart loc[1];
  __shared__ int64_t tmp[kTileThreads / 32];
  if (SHARED && w.first) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t base = (shared_u32(dyn) + 1023u) & ~1023u;
  uint8_t* gen = dyn + (base - shared_u32(dyn));
  volatile int* stop = reinterpret_cast<volatile int*>(gen + Sm::kMisc + 8);
  Masks* masks = reinterpret_cast<Masks*>(gen + Sm::kMasks);
  Scales* scales = reinterpret_cast<Scales*>(gen + Sm::kScales);  // 8-bit caches
  float* qscale = reinterpret_cast<float*>(gen + Sm::kQScale);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) -> uint32_t { return base + Sm::kBar + i * 8; };
  int bits = 0;

  if (warp == 12) tmem_alloc(base + Sm::kMisc, 512);
  if (tid == 0) {
    stop[0] = 0;
    stop[1] = 0;  // some row is not finite
    for (int i = 0; i < Sm::kBars; ++i) {
      const bool warps4 = i < Sm::kFree || (i >= Sm::kPReady && i < Sm::kODone);  // one arrival a warp
      const bool warps2 = i >= Sm::kQFull && i < Sm::kQFree;
      const int test = i >= Sm::kPReady && i < Sm::kODone ? GTKV_TEST_EXTRA_ARRIVALS : 0;
      mbar_init_n(bar(i), (warps4 ? 4 : warps2 ? 2 : 1) + test);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  TileWalk<SHARED> walk{p, b, a, w, 0, {}};
  const int64_t share = find_shares<kTileThreads, 1>(b.n_seqs, blockIdx.x, w.n_workers, w.min_share, loc, tmp,
                                                     [&](int32_t s) -> int64_t {
                                                       int err = 0;
                                                       walk.g.q = seq_of<SHARED>(p, b, s, err);
                                                       if (blockIdx.x == 0) bits |= err;
                                                       int64_t n = 0;
                                                       for (walk.g.tile = 0; walk.g.tile < walk.tiles(); ++walk.g.tile) {
                                                         walk.shape();
                                                         n += walk.g.span.steps() + kUnitCost;
                                                       }
                                                       return n * a.H;
                                                     });
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gen + Sm::kMisc);
  bool more = walk.start(loc[0], share);
  const Segment& g = walk.g;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const int wt = warp >> 2;                       // tile of rows
    const int r = tid & 127;                        // row of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + wt * 128, tO = lanes + 256 + wt * D;
    uint32_t n = 0;       // steps of the block so far
    uint32_t mine = 0;    // of them, steps of this tile
    uint32_t done = 0;    // units of this tile
    SplitRecord rec{-1, 0, 0, 0, 0, 0, 0};
    // the queries carry the scale's sign; a scale of 0 must keep -inf * c = -inf
    const float c0 = fmaxf(fabsf(a.scale_log2), 1e-37f);
    bool ok = true;
    for (; more && ok; more = walk.next()) {
      const bool here = wt * 128 < g.nf;  // the unit has rows in this tile
      if (g.step0 == 0 && g.end < g.span.steps())
        rec = SplitRecord{g.s, g.q.a, g.f0, g.nf, g.h,
                          static_cast<int32_t>(blockIdx.x + (g.span.steps() - g.end + share - 1) / share), g.q.row0};
      if (!here) {
        n += g.end - g.step0;
        continue;
      }
      const int32_t f = g.f0 + wt * 128 + r;
      const int32_t fc = min(f, g.f0 + g.nf - 1);
      const bool row_ok = f < g.f0 + g.nf;
      const int32_t pos = g.q.a + fc / (SHARED ? a.Gp : a.G);
      float c = c0;
      float ref = kNoRef;
      float2 sum = make_float2(0.0f, 0.0f);
      for (int32_t i = g.step0; i < g.end && ok; ++i, ++n, ++mine) {
        ok = wait_or_stop(bar(Sm::kSFull + wt), mine & 1, stop);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tmem_after_sync();
        const Masks& mk = masks[n % kSlots];
        const Scales& sl = scales[n % kSlots];
        const int32_t j0 = g.span.block(i) * kKeys;
        if (kCodes && i == g.step0) c = c0 * qscale[(done & 1) * kRows + wt * 128 + r];
        const uint4 live = *reinterpret_cast<const uint4*>(mk.live);
        // by the unit's rows, as the loaders decide it, so that no zeroed value is missed
        const bool cut = j0 + kKeys - 1 > g.i0 || (a.window && j0 <= g.i1 - a.window);
        const bool dead = (live.x & live.y & live.z & live.w) != 0xffffffffu;
        if (cut || dead) {
          // scores out of sight become -inf in place, so that the steps below need no masks
          const int hi = pos - j0;  // columns [lo, hi] and those below `first` are in sight
          const int lo = a.window ? pos - a.window + 1 - j0 : -1;
          const int first = a.window ? a.sinks - j0 : 0;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t x[32];
            tmem_load32(tS + 32 * k, x);
            const uint32_t lw = k == 0 ? live.x : k == 1 ? live.y : k == 2 ? live.z : live.w;
            uint32_t sight = lw;
            const int h = hi - 32 * k, l = lo - 32 * k, z = first - 32 * k;
            sight &= h >= 31 ? kFull : h < 0 ? 0 : (2u << h) - 1;
            sight &= (l <= 0 ? kFull : l > 31 ? 0 : ~((1u << l) - 1)) | (z <= 0 ? 0 : z > 31 ? kFull : (1u << z) - 1);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(sight >> e & 1)) x[e] = 0xff800000u;
            tmem_store32(tS + 32 * k, x);
          }
          tmem_wait_st();
          // values that are not finite were zeroed; rows that see such a key are done again at the end
          ok = wait_or_stop(bar(Sm::kFull + (2 * n + 1) % Sm::kRing), (2 * n + 1) / Sm::kRing & 1, stop);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          const uint4 nan4 = *reinterpret_cast<const uint4*>(mk.nan);
          if (nan4.x | nan4.y | nan4.z | nan4.w) {
            const uint32_t nw[4] = {nan4.x, nan4.y, nan4.z, nan4.w};
#pragma unroll 1
            for (int e = 0; e < kKeys; ++e)
              if (nw[e >> 5] >> (e & 31) & 1 && in_sight(a, pos, j0 + e)) sum.x = NAN;
          }
        }
        auto log_scale = [&](int e, float off, float2& m, float2& o) {  // exponents of columns e, e + 1: x m + o
          const float2 ks = *reinterpret_cast<const float2*>(sl.ks + e), lv = *reinterpret_cast<const float2*>(sl.lv + e);
          m = make_float2(ks.x * c, ks.y * c);
          o = make_float2(lv.x + off, lv.y + off);
        };
        // the step's largest exponent
        float m = -INFINITY;
        if constexpr (!kE4M3) {  // the loads' own maximum
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t x[32];
            float top;
            tmem_load32_max(tS + 32 * k, x, top);
            tmem_wait_ld(x);
            tmem_tie(x, top);
            m = fmaxf(m, top);
          }
          m *= c;
        } else if constexpr (P16) {
#pragma unroll 2
          for (int key = 0; key < kKeys; key += 16)
            m = fmaxf(m, fmaf(tmem_max16(tS + key), c * sl.ks[key], sl.lv[key]));
        } else {
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t x[32];
            tmem_load32(tS + 32 * k, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 mm, oo;
              log_scale(32 * k + e, 0.0f, mm, oo);
              const float2 t = ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mm, oo);
              m = fmaxf(m, fmaxf(t.x, t.y));
            }
          }
        }
        const bool move = m > ref + 8.0f;  // (always so for a row's first keys)
        if (__any_sync(kFull, move)) {
          const float next = move ? m : ref;
          const float keep = ex2(ref - next);
          ref = next;
          sum.x *= keep;
          sum.y *= keep;
          if (i > g.step0) {  // the products so far are done: the score product was issued after them
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t x[32];
              tmem_load32(tO + 32 * k, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * keep);
              tmem_store32(tO + 32 * k, x);
            }
          }
        }
        // Weights over the scores of their keys: the 16 columns of 16 keys take their 8 words of
        // rounded weights and, with TWO, 8 words of what the rounding left.
        const float off = kLift - (ref == kNoRef ? 0.0f : ref);  // (kNoRef itself would swallow the scores)
        {
          float2 add = make_float2(0.0f, 0.0f);
          uint32_t ra[32], rb[32];
          auto buf = [&](int k) -> uint32_t(&)[32] { return k & 1 ? rb : ra; };
          tmem_load32(tS, ra);
          tmem_wait_ld(ra);
          // Half of it written out: what both tiles' warps run through stays nearer to the instruction caches (8
          // prompts of 2048 tokens, written out / half: 16-bit 458 / 409 us, 8-bit 564 / 508, 4-bit 520 / 484; fp16
          // output 458 / 408, 697 / 598, 644 / 546). Prefixes of one tile of rows have the whole chain to wait for
          // instead (24 groups of 64 rows behind 8192 tokens: 210 / 212, 8-bit 221 / 223, fp16 267 / 279, 4-bit fp16
          // 248 / 292, but 4-bit bf16 283 / 232).
          constexpr int kWritten = SHARED && (!kE2M1 || TWO) ? 4 : 2;
#pragma unroll kWritten
          for (int k = 0; k < 4; ++k) {
            uint32_t(&x)[32] = buf(k);
            if (k < 3) tmem_load32(tS + 32 * (k + 1), buf(k + 1));
            uint32_t P[32];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int key = 32 * k + 16 * z;
              float2 ms = make_float2(c, c), os = make_float2(off, off), part = make_float2(0.0f, 0.0f);
              if constexpr (kE4M3 && P16) {  // 16 keys share a page, so their scales
                ms.x = ms.y = c * sl.ks[key];
                os.x = os.y = off + sl.lv[key];
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if constexpr (kE4M3 && !P16) log_scale(key + 2 * e, off, ms, os);
                const float2 t = ffma2(make_float2(__uint_as_float(x[16 * z + 2 * e]),
                                                   __uint_as_float(x[16 * z + 2 * e + 1])), ms, os);
                const float2 y = make_float2(ex2(t.x), ex2(t.y));
                if constexpr (kE4M3 && P16)
                  part = fadd2(part, y);
                else if constexpr (kE4M3)
                  add = ffma2(y, *reinterpret_cast<const float2*>(sl.iv + key + 2 * e), add);
                else
                  add = fadd2(add, y);
                const uint32_t hi = pack16<kBf16>(y.x, y.y);
                P[16 * z + e] = hi;
                if constexpr (TWO) {
                  const float2 lo = ffma2(unpack16<kBf16>(hi), make_float2(-1.0f, -1.0f), y);
                  P[16 * z + 8 + e] = pack16<kBf16>(lo.x, lo.y);
                }
              }
              if constexpr (kE4M3 && P16) add = ffma2(part, make_float2(sl.iv[key], sl.iv[key]), add);
              if constexpr (!TWO) tmem_store8(tS + key, &P[16 * z]);
            }
            if constexpr (TWO) tmem_store32(tS + 32 * k, P);
            if (k < 3) tmem_wait_ld(buf(k + 1));
          }
          sum = fadd2(sum, add);
        }
        tmem_wait_st();
        tmem_before_sync();
        warp_arrive(bar(Sm::kPReady + wt));
      }
      if (!ok) break;
      // ---- the unit's rows
      ok = __all_sync(kFull, wait_or_stop(bar(Sm::kODone + wt), done & 1, stop));
      if (!ok) break;
      ++done;
      tmem_after_sync();
      const float total = sum.x + sum.y;
      const bool whole = g.step0 == 0 && g.end == g.span.steps();
      const int64_t orow = g.q.row0 + fc / a.G;
      const int32_t qh = g.h * a.G + fc % a.G;
      if constexpr (SHARED) {
        // The rows' sums go to the state, a cut unit's through the other segments', warp by warp; they stay in
        // tensor memory meanwhile. What a warp leaves for another lies by elements, four of all its rows
        // together, so that a lane's row is not a stride for the others.
        const int row = wt * 128 + r;
        const int32_t me = blockIdx.x;
        float ref2 = ref, total2 = total;
        bool all = true, put_out = false;  // the warp holds all segments; the sums are in the state
        TreePlace tree;
        if (!whole) {
          if (g.step0 == 0)
            tree.begin(me, 1 + static_cast<int32_t>((g.span.steps() - g.end + share - 1) / share));
          else
            tree.go_on(me, share, g.in, g.span.steps(), kUnitCost);
        }
        auto part_of = [&](int32_t wk) {
          return w.part + (static_cast<int64_t>(wk) * 2 + (wk == tree.worker0 ? 1 : 0)) * (static_cast<int64_t>(kRows) * (D + 2));
        };
        float* state = a.state + (orow * a.Q + qh) * D;
        auto put = [&](int k, const uint32_t (&x)[32]) {  // whole 32-byte sectors
          if (!row_ok) return;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(state + 32 * k + e), "r"(x[e]), "r"(x[e + 1]),
                         "r"(x[e + 2]), "r"(x[e + 3]), "r"(x[e + 4]), "r"(x[e + 5]), "r"(x[e + 6]), "r"(x[e + 7])
                         : "memory");
        };
        // (Loads from and stores to tensor memory are the whole warp's.)
        while (!whole && tree.up()) {
          int32_t other;
          if (!meet(w.nodes + static_cast<int64_t>(tree.node) * 8 + warp, me, &other, [&]() {
                float* to = part_of(me);
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                  uint32_t x[32];
                  tmem_load32(tO + 32 * k, x);
                  tmem_wait_ld(x);
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    reinterpret_cast<uint4*>(to)[(8 * k + e) * kRows + row] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                }
                to[kRows * D + row] = ref2;
                to[kRows * (D + 1) + row] = total2;
              })) {
            all = false;
            break;
          }
          const float* from = part_of(other);
          const float oref = __ldcg(from + kRows * D + row), ototal = __ldcg(from + kRows * (D + 1) + row);
          const float top = fmaxf(ref2, oref), k1 = ex2(ref2 - top), k2 = ex2(oref - top);
          auto sum_of = [&](float x, float y) {  // left + right, whoever holds them
            return tree.left ? __fmaf_rn(x, k1, __fmul_rn(y, k2)) : __fmaf_rn(y, k2, __fmul_rn(x, k1));
          };
          ref2 = top;
          total2 = sum_of(total2, ototal);
          put_out = 2 * tree.s >= tree.n;  // the root
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t x[32];
            float4 y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __ldcg(reinterpret_cast<const float4*>(from) + (8 * k + e) * kRows + row);
            tmem_load32(tO + 32 * k, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[4 * e] = __float_as_uint(sum_of(__uint_as_float(x[4 * e]), y[e].x));
              x[4 * e + 1] = __float_as_uint(sum_of(__uint_as_float(x[4 * e + 1]), y[e].y));
              x[4 * e + 2] = __float_as_uint(sum_of(__uint_as_float(x[4 * e + 2]), y[e].z));
              x[4 * e + 3] = __float_as_uint(sum_of(__uint_as_float(x[4 * e + 3]), y[e].w));
            }
            if (put_out)
              put(k, x);
            else
              tmem_store32(tO + 32 * k, x);
          }
          tmem_wait_st();
          tree.joined();
        }
        if (all && !put_out) {
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t x[32];
            tmem_load32(tO + 32 * k, x);
            tmem_wait_ld(x);
            put(k, x);
          }
        }
        if (all && row_ok) {  // (the reference of weights is lifted, the state's is not)
          a.state[a.state_rows * D + orow * a.Q + qh] = ref2 - kLift;
          a.state[a.state_rows * (D + 1) + orow * a.Q + qh] = total2;
        }
      } else if (whole) {
        bool bad = !(total <= 3.402823466e38f);
        const float inv = bad ? NAN : total == 0.0f ? 0.0f : rcp(total);
        uint16_t* out = static_cast<uint16_t*>(a.out) + (orow * a.Q + qh) * D;
        const float2 inv2 = make_float2(inv, inv), none = make_float2(0.0f, 0.0f);
        float2 zero = none;  // stays 0 while all values are finite
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t raw[32];
          tmem_load32(tO + 32 * k, raw);
          tmem_wait_ld(raw);
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 v = ffma2(make_float2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])), inv2, none);
            zero = ffma2(v, none, zero);
            y[e] = a.type == KV_TYPE_BF16 ? pack_b(v.x, v.y) : pack_h(v.x, v.y);
          }
          if (row_ok) {
            if (w.out_wide) {
#pragma unroll
              for (int e = 0; e < 16; e += 8)  // whole 32-byte sectors: a lane's row is its own
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + 32 * k + 2 * e), "r"(y[e]),
                             "r"(y[e + 1]), "r"(y[e + 2]), "r"(y[e + 3]), "r"(y[e + 4]), "r"(y[e + 5]), "r"(y[e + 6]),
                             "r"(y[e + 7])
                             : "memory");
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                out[32 * k + 2 * e] = static_cast<uint16_t>(y[e]);
                out[32 * k + 2 * e + 1] = static_cast<uint16_t>(y[e] >> 16);
              }
            }
          }
        }
        if (a.lse && row_ok) a.lse[orow * a.Q + qh] = total == 0.0f ? -INFINITY : (ref - kLift + log2f(total)) * kLn2;
        bad = bad || !(zero.x + zero.y == 0.0f);
        if (bad && row_ok) stop[1] = 1;
      } else {
        const int slot = g.step0 == 0 ? 1 : 0;
        const int row = wt * 128 + r;
        float* part = w.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * (static_cast<int64_t>(kRows) * (D + 2));
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t raw[32];
          tmem_load32(tO + 32 * k, raw);
          tmem_wait_ld(raw);
          if (row_ok) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4*>(part + row * D + 32 * k)[e] =
                  make_uint4(raw[4 * e], raw[4 * e + 1], raw[4 * e + 2], raw[4 * e + 3]);
          }
        }
        part[kRows * D + row] = ref;
        part[kRows * (D + 1) + row] = total;
      }
    }
    if (!SHARED && tid == 0) w.rec[blockIdx.x] = ok ? rec : SplitRecord{-1, 0, 0, 0, 0, 0, 0};
    // rows that came out with anything not finite are done again, key by key
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (stop[1] && !*stop && walk.start(loc[0], share)) do {
      if (g.step0 > 0 || g.end < g.span.steps()) continue;  // the join's
      for (int32_t k = warp; k < g.nf; k += 8) {
        const int32_t f = g.f0 + k;
        const int64_t orow = g.q.row0 + f / a.G;
        const int32_t qh = g.h * a.G + f % a.G;
        const uint16_t* out = static_cast<const uint16_t*>(a.out) + (orow * a.Q + qh) * D;
        bool bad = false;
        const int exponent = a.type == KV_TYPE_BF16 ? 0x7f80 : 0x7c00;
        for (int e = lane; e < D; e += 32) bad = bad || (out[e] & exponent) == exponent;
        if (__any_sync(kFull, bad)) attend_row<C>(p, b, a, g.s, g.q.a + f / a.G, orow, qh, &bits);
      }
    } while (walk.next());
  } else if (warp < 12) {
    // ------------------------------------------------------------- loaders
    const int lw = warp - 8;
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(p.base);
    constexpr int RB = kE2M1 ? D / 2 : kE4M3 ? D : 2 * D;  // bytes of a head's row (4-bit caches: of its codes)
    constexpr int LPR = RB / 16 < 8 ? RB / 16 : 8;  // lanes a row
    constexpr int RPI = 32 / LPR;                   // rows a round
    constexpr int PPR = RB / 16 / LPR;              // pieces of a row a lane
    constexpr int IT = 32 / RPI;
    const int lr = lane / LPR, lc = lane % LPR;
    uint32_t n = 0;   // steps of the block so far
    uint32_t u = 0;   // units with rows in the warp's tile of queries
    const int qt = lw >> 1;
    bool ok = true;
    // (positions and rows are below 2^31)
    auto page_index = [&](uint32_t j) { return p.ps_shift >= 0 ? j >> p.ps_shift : j / static_cast<uint32_t>(p.ps); };
    // the loader's 32 keys of a step: key lw * 32 + lane is this lane's
    auto entry = [&](int32_t i) -> int32_t {
      if (i >= g.end) return 0;
      const uint32_t j = static_cast<uint32_t>(g.span.block(i)) * kKeys + lw * 32 + lane;
      // (keys that share the scales of 16 share their page too, so all of them are looked up or none)
      constexpr int64_t kShared = kE4M3 && P16 ? 15 : 0;
      if (j > static_cast<uint32_t>(g.i1) || !some_row_sees(a, g.i0, j & ~kShared, j | kShared)) return 0;
      return __ldg(b.table + static_cast<int64_t>(g.s) * b.max_pages + page_index(j));
    };
    struct Keys {
      int32_t row, page;  // this lane's key; row -1: no token
      uint32_t live;
      bool partial;       // some row may not see some key
    };
    auto keys_of = [&](int32_t i, int32_t ent) -> Keys {
      Keys k;
      const int32_t j0 = g.span.block(i) * kKeys;
      const uint32_t j = static_cast<uint32_t>(j0) + lw * 32 + lane, ps = static_cast<uint32_t>(p.ps);
      k.page = static_cast<int32_t>(page_of_entry(p, b, ent, bits));
      k.row = k.page == 0 ? -1
                          : static_cast<int32_t>(static_cast<uint32_t>(k.page) * static_cast<uint32_t>(p.stride) + 2 * a.layer * ps +
                                                 (p.ps_shift >= 0 ? j & (ps - 1) : j % ps));
      k.live = __ballot_sync(kFull, k.page != 0);
      k.partial = j0 + kKeys - 1 > g.i0 || (a.window && j0 <= g.i1 - a.window) || k.live != kFull;
      return k;
    };
    auto wait = [&](uint32_t at, uint32_t parity) {
      ok = __all_sync(kFull, wait_or_stop(at, parity, stop));
      return ok;
    };

    // the unit's queries: 64 rows a warp, the row's address looked up by a lane each
    auto query_rows = [&](int64_t& qa, int64_t& qb) {
      auto q_at = [&](int32_t f) -> int64_t {
        const int32_t ff = g.f0 + f;
        return f < g.nf ? (g.q.row0 + ff / a.G) * a.q_stride + static_cast<int64_t>(g.h * a.G + ff % a.G) * D : -1;
      };
      qa = q_at(lw * 64 + lane);
      qb = q_at(lw * 64 + 32 + lane);
    };
    auto load_queries = [&](int64_t qa, int64_t qb) {
      constexpr int QP = kPieces / 8;  // pieces of a row a lane; 8 lanes a row, 4 rows a round
      const int ql = lane >> 3, qc = lane & 7;
      auto q_tile = [&](int rr) { return base + Sm::kQ + ((lw * 64 + rr) >> 7) * Sm::kOperand; };
      if (!kCodes && w.q_wide && a.scale_log2 >= 0.0f) {
#pragma unroll
        for (int it = 0; it < 16; ++it) {
          const int rr = it * 4 + ql;
          const int64_t at = __shfl_sync(kFull, it < 8 ? qa : qb, rr & 31);
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + (at >= 0 ? at : 0) + qc * 8;
#pragma unroll
          for (int k = 0; k < QP; ++k)
            copy_async<16>(q_tile(rr) + piece_at((lw * 64 + rr) & 127, qc + k * 8), src + k * 64, at >= 0);
        }
        return;
      }
      constexpr int B = 4;  // rounds whose loads are in flight together
#pragma unroll 1
      for (int it0 = 0; it0 < 16; it0 += B) {
        uint4 v[B][QP];
#pragma unroll
        for (int z = 0; z < B; ++z) {
          const int rr = (it0 + z) * 4 + ql;
          const int64_t va = __shfl_sync(kFull, qa, rr & 31), vb = __shfl_sync(kFull, qb, rr & 31);
          const int64_t at = rr < 32 ? va : vb;
#pragma unroll
          for (int k = 0; k < QP; ++k) {
            v[z][k] = make_uint4(0, 0, 0, 0);
            if (at >= 0) {
              const uint16_t* src = static_cast<const uint16_t*>(a.q) + at + (qc + k * 8) * 8;
              if (w.q_wide) {
                v[z][k] = __ldg(reinterpret_cast<const uint4*>(src));
              } else {
                uint32_t e[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) e[y] = __ldg(src + y);
                v[z][k] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
              }
            }
          }
        }
#pragma unroll
        for (int z = 0; z < B; ++z) {
          const int rr = (it0 + z) * 4 + ql;
          if constexpr (kCodes) {  // fp16 after a power of two that brings the row's largest to [2^14, 2^15)
            float x[QP][8];
            float amax = 0.0f;
#pragma unroll
            for (int k = 0; k < QP; ++k) {
              const uint32_t e[4] = {v[z][k].x, v[z][k].y, v[z][k].z, v[z][k].w};
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const uint32_t h = y & 1 ? e[y >> 1] >> 16 : e[y >> 1] & 0xffffu;
                x[k][y] = a.type == KV_TYPE_BF16 ? __uint_as_float(h << 16)
                                                 : __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
                amax = fmaxf(amax, fabsf(x[k][y]));
              }
            }
#pragma unroll
            for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            int ex = 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23);
            ex = amax > 0.0f ? max(-100, min(100, ex)) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
            if (qc == 0) qscale[(u & 1) * kRows + lw * 64 + rr] = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
            for (int k = 0; k < QP; ++k)
              v[z][k] = make_uint4(pack_h(x[k][0] * up, x[k][1] * up), pack_h(x[k][2] * up, x[k][3] * up),
                                   pack_h(x[k][4] * up, x[k][5] * up), pack_h(x[k][6] * up, x[k][7] * up));
          }
          const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0;
#pragma unroll
          for (int k = 0; k < QP; ++k)
            sts128(q_tile(rr) + piece_at((lw * 64 + rr) & 127, qc + k * 8),
                   make_uint4(v[z][k].x ^ flip, v[z][k].y ^ flip, v[z][k].z ^ flip, v[z][k].w ^ flip));
        }
      }
    };

    auto full = [&](uint32_t t) { return bar(Sm::kFull + t % Sm::kRing); };
    auto operand = [&](uint32_t t) { return base + Sm::kTiles + t % Sm::kRing * Sm::kOperand; };
    // waits until tile t - kRing has been used
    auto claim = [&](uint32_t t) { return wait(bar(Sm::kFree + t % Sm::kRing), (t / Sm::kRing & 1) ^ 1); };
    const int32_t row_bytes = static_cast<int32_t>(p.vpr * 16);
    // Copies 32 rows (of round `it` the lane's ro[it]) of K, or of V when `v`; at(round, piece): where a lane's piece
    // goes.
    auto rows_of = [&](int32_t row_of_lane, int32_t* ro) {  // all shuffles together: their latencies overlap
#pragma unroll
      for (int it = 0; it < IT; ++it) ro[it] = __shfl_sync(kFull, row_of_lane, it * RPI + lr);
    };
    auto copy = [&](auto at, const int32_t* ro, bool v) {
      const uint8_t* from = pool + static_cast<int64_t>(g.h) * RB + lc * 16 + (v ? p.ps * row_bytes : 0);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const bool ok = ro[it] >= 0;
        const uint8_t* src = from + static_cast<int64_t>(ok ? ro[it] : 0) * row_bytes;
#pragma unroll
        for (int z = 0; z < PPR; ++z) copy_async<16>(at(it, z), src + z * LPR * 16, ok);
      }
      copy_commit();
    };
    if constexpr (kCodes) {
      // A step's codes are copied one step ahead; a lane turns the very pieces
      // that it copied into fp16, so the raw ring needs no barrier. Order of
      // a step: copy K(n + 1), turn K(n), copy V(n + 1), turn V(n); the raw
      // tile that a copy overwrites is the one turned just before it.
      struct Step {
        Keys k;
        float ks, vs;         // 8-bit caches: the scales of the lane's key
        bool first, queries;  // first of its unit; the unit has rows in the warp's tile
      };
      const uint32_t raw0 = base + Sm::kRaw + lw * 32 * RB + lane * 16;
      // 4-bit caches: scales of step n, of the warp's keys, K's and V's; in shared memory, since a key has 8 to 16
      // bytes of them and the kernel no register to spare. (The two scales of an 8-bit cache's key are held by its
      // lane.)
      constexpr int SB = Sm::kRawScale;
      const uint32_t scales0 = base + Sm::kRawScales + lw * 32 * 2 * SB;
      auto raw_scales = [&](uint32_t n) { return scales0 + (n & 1) * (128 * 2 * SB); };
      auto raw = [&](uint32_t t, int it) { return raw0 + t % 3 * Sm::kRawTile + it * 512; };
      int64_t qa = -1, qb = -1;
      // the step after the one in `walk`, as far as its lookups go
      int32_t i = more ? g.step0 : 0, ent = more ? entry(g.step0) : 0;
      bool have = more;
      auto look = [&]() -> Step {
        Step s;
        s.k = keys_of(i, ent);
        s.first = i == g.step0;
        s.queries = qt * 128 < g.nf;
        ent = entry(i + 1);
        s.ks = s.vs = 0.0f;
        if (kE4M3 && s.k.page != 0) {
          const int64_t at = (static_cast<int64_t>(s.k.page) * p.blocks + 2 * a.layer) * a.H + g.h;
          s.ks = __ldg(a.scales + at);
          s.vs = __ldg(a.scales + at + a.H);
        }
        return s;
      };
      // copies a step's scales, in the group of its keys
      auto copy_scales = [&](uint32_t n, const Keys& k) {
        if constexpr (kE2M1) {
          const bool live = k.page != 0;
          const uint32_t to = raw_scales(n) + lane * 2 * SB;
          const uint8_t* from = pool + code_bytes(a.H, D) + g.h * SB + static_cast<int64_t>(live ? k.row : 0) * row_bytes;
          copy_async<SB>(to, from, live);
          copy_async<SB>(to + SB, from + (live ? p.ps * row_bytes : 0), live);
        }
      };
      auto advance = [&]() {
        if (++i == g.end) {
          have = walk.next();
          if (have) {
            i = g.step0;
            ent = entry(i);
          }
        }
      };
      // In batches whose loads come first, and in a loop: the warps of a scheduler run through more code a step than
      // its instruction cache holds, and what is written out is fetched every time (chunks, written out / in a loop:
      // 8-bit 474 / 450 us, 4-bit 454 / 440).
      auto turn_tile = [&](uint32_t t, bool check) -> uint32_t {
        uint32_t bad_rows = 0;
        const uint32_t to = operand(t);
        if constexpr (kE2M1) {
          constexpr int B = 2;
#pragma unroll 1
          for (int it0 = 0; it0 < IT; it0 += B) {
            uint32_t s4[B];
            uint4 codes[B];
#pragma unroll
            for (int ib = 0; ib < B; ++ib) {
              codes[ib] = lds128(raw(t, it0 + ib));
              s4[ib] = lds16(raw_scales(t >> 1) + (((it0 + ib) * RPI + lr) * 2 + (t & 1)) * SB + lc * 2);
            }
#pragma unroll
            for (int ib = 0; ib < B; ++ib) {
              const int it = it0 + ib;
              const uint4 v = codes[ib];
              uint32_t bytes = s4[ib];
              const uint32_t bad = bad_scales(bytes);
              if (!check) {
                bytes |= bad;
              } else if (bad) {
                bad_rows |= 1u << (it * RPI + lr);
                bytes &= ~bad;
              }
              const uint32_t sc[2] = {__byte_perm(bytes, 0, 0x4040) << 7, __byte_perm(bytes, 0, 0x4141) << 7};
              const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
              const int rr = lw * 32 + it * RPI + lr;
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                uint32_t y[4];
                codes8(w4[z], y);
                sts128(to + piece_at(rr, 4 * lc + z), make_uint4(mul_h2(y[0], sc[z >> 1]), mul_h2(y[1], sc[z >> 1]),
                                                                 mul_h2(y[2], sc[z >> 1]), mul_h2(y[3], sc[z >> 1])));
              }
            }
          }
        } else {
          constexpr int B = 4;
#pragma unroll 1
          for (int it0 = 0; it0 < IT; it0 += B) {
            uint4 codes[B];
#pragma unroll
            for (int ib = 0; ib < B; ++ib) codes[ib] = lds128(raw(t, it0 + ib));
#pragma unroll
            for (int ib = 0; ib < B; ++ib) {
              const int it = it0 + ib;
              uint4 v = codes[ib];
              if (check) {
                const uint4 z = make_uint4(not_finite<C>(v.x), not_finite<C>(v.y), not_finite<C>(v.z), not_finite<C>(v.w));
                if (z.x | z.y | z.z | z.w) {
                  bad_rows |= 1u << (it * RPI + lr);
                  v = make_uint4(v.x & ~z.x, v.y & ~z.y, v.z & ~z.z, v.w & ~z.w);
                }
              }
              uint4 lo, hi;
              decode16(v, lo, hi);
              const int rr = lw * 32 + it * RPI + lr;
              sts128(to + piece_at(rr, 2 * lc), lo);
              sts128(to + piece_at(rr, 2 * lc + 1), hi);
            }
          }
        }
        fence_async_shared();
        return bad_rows;
      };
      if (have) {
        Step cur = look();
        copy_scales(0, cur.k);
        int32_t ro[IT];
        rows_of(cur.k.row, ro);
        copy([&](int it, int) { return raw(0, it); }, ro, false);
        copy([&](int it, int) { return raw(1, it); }, ro, true);
        query_rows(qa, qb);
        for (bool go = true; go;) {
          int64_t na = -1, nb = -1;
          advance();
          go = have;
          Step next{};
          if (have) {
            next = look();
            copy_scales(n + 1, next.k);
            rows_of(next.k.row, ro);
            if (next.first) {
              query_rows(na, nb);
              for (int k = 0; k < 2 * D; k += 128) {  // on their way when the unit begins
                if (na >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.q) + 2 * na + k));
                if (nb >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.q) + 2 * nb + k));
              }
            }
          }
          bool gone = false;
#pragma unroll
          for (uint32_t v = 0; v < 2; ++v) {
            if (gone) break;
            const uint32_t t = 2 * n + v;
            if (have)
              copy([&](int it, int) { return raw(t + 2, it); }, ro, v != 0);
            else
              copy_commit();
            copy_wait<2>();
            if constexpr (kE2M1) __syncwarp();  // scales that other lanes copied
            gone = !claim(t);
            if (gone) break;
            if (v == 0) {
              if constexpr (kE4M3) {
                Scales& sl = scales[n % kSlots];
                sl.ks[lw * 32 + lane] = cur.k.page != 0 ? cur.ks : 1.0f;  // no token: 2^-inf through lv, whatever the score
                sl.lv[lw * 32 + lane] = lg2(cur.vs);
                sl.iv[lw * 32 + lane] = cur.k.page != 0 ? rcp(cur.vs) : 0.0f;
              }
              if (lane == 0) masks[n % kSlots].live[lw] = cur.k.live;
            }
            const uint32_t bad_rows = turn_tile(t, v != 0 && cur.k.partial);
            if (v != 0) {
              const uint32_t nan = __reduce_or_sync(kFull, bad_rows);
              if (lane == 0) masks[n % kSlots].nan[lw] = nan;
            }
            warp_arrive(full(t));
            if (v == 0 && cur.first && cur.queries) {
              gone = !wait(bar(Sm::kQFree + qt), (u & 1) ^ 1);
              if (gone) break;
              load_queries(qa, qb);
              fence_async_shared();
              warp_arrive(bar(Sm::kQFull + qt));
              ++u;
            }
          }
          if (gone) break;
          if (next.first) {
            qa = na;
            qb = nb;
          }
          cur = next;
          ++n;
        }
      }
      copy_wait<0>();
    } else {
      // One more copy is always in flight: a tile is announced after the next
      // one has been asked for.
      bool pending = false, pending_partial = false;
      auto put = [&](uint32_t t, const Keys& k) {
        const uint32_t to = operand(t);
        int32_t ro[IT];
        rows_of(k.row, ro);
        copy([&](int it, int z) { return to + piece_at(lw * 32 + it * RPI + lr, lc + z * LPR); }, ro, t & 1);
      };
      auto announce_v = [&](uint32_t m) {  // V of step m has arrived
        uint32_t bad_rows = 0;
        if (pending_partial) {
          const uint32_t vt = operand(2 * m + 1);
#pragma unroll
          for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int z = 0; z < PPR; ++z) {
              const uint32_t at = vt + piece_at(lw * 32 + it * RPI + lr, lc + z * LPR);
              const uint4 v = lds128(at);
              const uint4 x = make_uint4(not_finite<C>(v.x), not_finite<C>(v.y), not_finite<C>(v.z), not_finite<C>(v.w));
              if (x.x | x.y | x.z | x.w) {
                bad_rows |= 1u << (it * RPI + lr);
                sts128(at, make_uint4(v.x & ~x.x, v.y & ~x.y, v.z & ~x.z, v.w & ~x.w));
              }
            }
        }
        bad_rows = __reduce_or_sync(kFull, bad_rows);
        if (lane == 0) masks[m % kSlots].nan[lw] = bad_rows;
        fence_async_shared();
        warp_arrive(full(2 * m + 1));
        pending = false;
      };
      for (; more && ok; more = walk.next()) {
        const bool queries = qt * 128 < g.nf;
        int32_t ent = entry(g.step0);
        for (int32_t i = g.step0; i < g.end; ++i, ++n) {
          const Keys cur = keys_of(i, ent);
          ent = entry(i + 1);
          if (!claim(2 * n)) break;
          if (lane == 0) masks[n % kSlots].live[lw] = cur.live;
          put(2 * n, cur);
          if (pending) {
            copy_wait<1>();
            announce_v(n - 1);
          }
          if (i == g.step0 && queries) {
            if (!wait(bar(Sm::kQFree + qt), (u & 1) ^ 1)) break;
            int64_t qa, qb;
            query_rows(qa, qb);
            load_queries(qa, qb);
            copy_commit();
          }
          if (!claim(2 * n + 1)) break;
          put(2 * n + 1, cur);
          pending = true;
          pending_partial = cur.partial;
          copy_wait<1>();
          fence_async_shared();
          warp_arrive(full(2 * n));
          if (i == g.step0 && queries) {
            warp_arrive(bar(Sm::kQFull + qt));
            ++u;
          }
        }
      }
      copy_wait<0>();
      if (pending && ok) announce_v(n - 1);
    }
  } else {
    if (warp == 12) {
      // All lanes run along, so that operands and waits stay warp-uniform (a lone
      // lane's operands would be moved to uniform registers one by one, which
      // took 85 cycles a product against its 64); one elected lane issues.
      // ------------------------------------------------------------- products
      constexpr uint32_t kQK = umma_f16(kBf16, kKeys, false), kPV = umma_f16(kBf16, D, true);
      const bool elected = elect_one();
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      uint32_t n = 0;
      uint32_t weights[2] = {0, 0}, queries[2] = {0, 0};  // phases of each tile's barriers
      bool ok = true;
      auto slot_of = [&](uint32_t t) { return t % Sm::kRing; };
      auto wait = [&](uint32_t at, uint32_t parity) { return __all_sync(kFull, wait_or_stop(at, parity, stop)) != 0; };
      auto full = [&](uint32_t t) { return wait(bar(Sm::kFull + slot_of(t)), t / Sm::kRing & 1); };
      const uint32_t ub = __shfl_sync(kFull, base, 0);
      const uint32_t q0 = smem_operand_lo(ub + Sm::kQ, 16), k0 = smem_operand_lo(ub + Sm::kTiles, 16);
      const uint32_t v0 = smem_operand_lo(ub + Sm::kTiles, 128 * 128);
      auto qk = [&](int wt, uint32_t t) {
        const uint32_t qd = q0 + wt * (Sm::kOperand >> 4), kd = k0 + slot_of(t) * (Sm::kOperand >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
          umma_ss(elected, tm + wt * 128, qd + at, kd + at, kQK, k > 0);
        }
        umma_commit(elected, bar(Sm::kSFull + wt));
      };
      auto pv = [&](int wt, uint32_t t, bool add) {
        const uint32_t vd = v0 + slot_of(t) * (Sm::kOperand >> 4);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) {
          umma_ts(elected, tm + 256 + wt * D, tm + wt * 128 + k * 16, vd + (k * 2048 >> 4), kPV, add || k > 0);
          if constexpr (TWO)
            umma_ts(elected, tm + 256 + wt * D, tm + wt * 128 + k * 16 + 8, vd + (k * 2048 >> 4), kPV, true);
        }
      };
      auto scores = [&](int wt, uint32_t t, bool first, bool last) {
        if (first) ok = wait(bar(Sm::kQFull + wt), queries[wt]++ & 1);
        if (!ok) return;
        tmem_after_sync();
        qk(wt, t);
        if (last) umma_commit(elected, bar(Sm::kQFree + wt));
      };
      // Runs on from unit to unit: behind a tile's O += P V comes its next S,
      // be it the next unit's first.
      more = __any_sync(kFull, more);
      int nt = __shfl_sync(kFull, g.nf > 128 ? 2 : 1, 0);
      int32_t i = 0, steps = __shfl_sync(kFull, g.end - g.step0, 0);
      if (more) {
        ok = full(0);
        scores(0, 0, true, steps == 1);
        if (ok && nt > 1) scores(1, 0, true, steps == 1);
        umma_commit(elected, bar(Sm::kFree));
      }
#pragma unroll 1
      while (more && ok) {
        const bool last = i + 1 == steps;
        int next_nt = nt;
        int32_t next_i = i + 1, next_steps = steps;
        if (last) {
          more = __any_sync(kFull, walk.next());
          next_nt = __shfl_sync(kFull, !more ? 0 : g.nf > 128 ? 2 : 1, 0);
          next_i = 0;
          next_steps = __shfl_sync(kFull, g.end - g.step0, 0);
        }
        // V of this step and K of the next are there long before the weights as a rule
        ok = full(2 * n + 1) && (!more || full(2 * n + 2));
#pragma unroll
        for (int wt = 0; wt < 2; ++wt) {
          if (ok && wt < nt) {
            ok = wait(bar(Sm::kPReady + wt), weights[wt]++ & 1);
            if (ok) {
              tmem_after_sync();
              pv(wt, 2 * n + 1, i > 0);
              if (last) umma_commit(elected, bar(Sm::kODone + wt));
            }
          }
          if (ok && wt < next_nt) scores(wt, 2 * n + 2, next_i == 0, next_i + 1 == next_steps);
        }
        if (!ok) break;
        umma_commit(elected, bar(Sm::kFree + slot_of(2 * n + 1)));
        if (more) umma_commit(elected, bar(Sm::kFree + slot_of(2 * n + 2)));
        i = next_i;
        steps = next_steps;
        nt = next_nt;
        ++n;
      }
      umma_commit(elected, bar(Sm::kDrain));  // tensor memory is freed when nothing is in flight
      const long long t0 = clock64();
      while (!mbar_try(bar(Sm::kDrain), 0) && clock64() - t0 < kWaitClocks) {
      }
    }
    __syncwarp();
  }
  tmem_before_sync();
  __syncthreads();
  tmem_after_sync();
  // launched over the tail of the few-rows kernel: the join waits for this
  // kernel alone, so this kernel ends after that one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 12) tmem_free(tmem, 512);
  if (tid == 0 && *stop) bits |= KV_DEV_ERR_TIMEOUT;
  store_bits(p, bits);
}

template <class C, bool P16, bool TWO, bool SHARED>
cudaError_t prepare_one(int32_t D) {
  auto set = [](auto kernel, int bytes) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); };
  return D == 64 ? set(k_attend_tile<C, 64, P16, TWO, SHARED>, TileSmem<C, 64>::kBytes)
                 : set(k_attend_tile<C, 128, P16, TWO, SHARED>, TileSmem<C, 128>::kBytes);
}

template <class C, bool P16, bool TWO, bool SHARED>
cudaError_t launch_one(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, bool after, cudaStream_t s) {
  auto kernel = a.D == 64 ? k_attend_tile<C, 64, P16, TWO, SHARED> : k_attend_tile<C, 128, P16, TWO, SHARED>;
  const int smem = a.D == 64 ? TileSmem<C, 64>::kBytes : TileSmem<C, 128>::kBytes;
  if (after) return launch_overlapped(kernel, dim3(w.blocks), kTileThreads, smem, s, p, b, a, w);
  kernel<<<w.blocks, kTileThreads, smem, s>>>(p, b, a, w);
  return cudaGetLastError();
}

// Caches of codes: one part of the weights will do for a bf16 output; in 8 bits the page size matters.
template <class C>
constexpr bool kIsCode = std::is_same_v<C, CodeE4M3> || std::is_same_v<C, CodeE2M1>;
template <class C>
constexpr bool kPaged = std::is_same_v<C, CodeE4M3>;

}  // namespace

template <class C, bool SHARED>
cudaError_t launch_tile(const DevPool& p, const Batch& b, const AttendArgs& a, const Split& w, bool after, cudaStream_t s) {
  constexpr bool kOne = kIsCode<C>;
  const bool one = kOne && a.type == KV_TYPE_BF16;
  if (kPaged<C> && p.ps % 16 == 0)
    return one ? launch_one<C, kPaged<C>, !kOne, SHARED>(p, b, a, w, after, s)
               : launch_one<C, kPaged<C>, true, SHARED>(p, b, a, w, after, s);
  return one ? launch_one<C, false, !kOne, SHARED>(p, b, a, w, after, s) : launch_one<C, false, true, SHARED>(p, b, a, w, after, s);
}

template <class C, bool SHARED>
cudaError_t prepare_tile(int32_t D, bool p16) {
  constexpr bool kOne = kIsCode<C>;
  const bool paged = kPaged<C> && p16;
  const cudaError_t e = paged ? prepare_one<C, kPaged<C>, true, SHARED>(D) : prepare_one<C, false, true, SHARED>(D);
  if (e != cudaSuccess || !kOne) return e;
  return paged ? prepare_one<C, kPaged<C>, !kOne, SHARED>(D) : prepare_one<C, false, !kOne, SHARED>(D);
}

// One pair of instances a file (kv_attend_tile_*.cu), so that they compile side by side.
#define GTKV_TILE_INSTANCES(C, SHARED)                                                                                    \
  template cudaError_t launch_tile<C, SHARED>(const DevPool&, const Batch&, const AttendArgs&, const Split&, bool,       \
                                              cudaStream_t);                                                            \
  template cudaError_t prepare_tile<C, SHARED>(int32_t, bool);

}  // namespace gtkv
