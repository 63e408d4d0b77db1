// Attention of a batch's new tokens over a paged key/value cache.
//
// For a query row q and the keys j it sees, with x_j = scale q . k_j (bounded by
// softcap * tanh(x / softcap) when asked for):
//   o = sum_j e^{x_j} v_j / sum_j e^{x_j},   lse = log sum_j e^{x_j},
// in one pass over the keys: a reference m, the sum l of 2^{x - m} and the
// unnormalised output, all in fp32 and in log2 units.  Any reference gives the same
// quotient as long as nothing overflows or vanishes, so it need not be the maximum:
// chunks take it from the first keys a row sees (in fp16 they move it when a weight
// grows large, l and o multiplied by 2^{m - m'}), and compute a share again, with a
// reference that follows the maximum, in the rare case that this did not hold;
// decode moves it when a score exceeds m by more than kSlack.
//
// Products on 32x32x16 MFMAs, transposed so that a query row is a lane's column:
//   S^T [keys x rows] = K Q^T     A = K rows from LDS, B = Q rows from registers
//   O^T [dims x rows] += V^T P^T  A = V columns (transposed LDS reads), B = P^T
// S^T leaves its accumulator with 16 keys of one row in each lane, which is
// what the next product's B operand holds (the keys in an order that the reads
// of V follow), so P never leaves the lane, and l, m and o's scaling are a
// lane's own.
//
// The query rows of all q-heads of a kv-head and of consecutive tokens share a
// workgroup's tile (row = token * group + head): K and V are read once for them.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gdn_internal.h"

namespace gdn {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr float kNoScore = -__FLT_MAX__;  // reference before the first score
constexpr float kLn2 = 0.6931471805599453f;

// Element types.  References lie kBias below the highest score at hand, so that
// scores far below it keep a weight: fp16 has none under 2^-25, and 2^17 keys at
// that weight may hold all the values beside one heavy key that holds none.
// 2^(kBias + kSlack) stays in the type's range.  Decode takes a new reference when a
// score exceeds its own by kBias + kSlack.  Chunks take theirs from the first block a
// row sees and keep it in bf16 (whose weights have fp32's range) while the row's
// weights sum to at most kHigh and nothing overflows; in fp16 (kMoves) they take a
// new one when 16 weights sum to more than 2^(kBias + kSlack).  Over 32,768 scores
// spread by 2 (by 4) that is so in 2 (22) of a wave's 1,024 blocks.  kOne is 1 in the
// type, kExp and kCarry find values that are not finite in a packed pair.
struct Bf {
  static constexpr float kBias = 0.f, kSlack = 8.f, kHigh = 0x1p100f;
  static constexpr bool kMoves = false;
  static constexpr uint32_t kOne = 0x3f80u, kExp = 0x7f807f80u, kCarry = 0x00800080u;
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return f2bf2(a, b); }
  // two e4m3 codes (of the low or the high half), times a power of two
  static __device__ __forceinline__ uint32_t lo8(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
  }
  static __device__ __forceinline__ uint32_t hi8(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true));
  }
};
struct Hf {
  static constexpr float kBias = 7.f, kSlack = 8.f, kHigh = 0x1p100f, kMost = 0x1p15f;
  static constexpr bool kMoves = true;
  static constexpr uint32_t kOne = 0x3c00u, kExp = 0x7c007c00u, kCarry = 0x04000400u;
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  }
  static __device__ __forceinline__ uint32_t lo8(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false));
  }
  static __device__ __forceinline__ uint32_t hi8(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true));
  }
};

// 8 codes as 8 values of the element type, the first 4 times a, the others times b.
template <class E>
__device__ __forceinline__ u32x4 values8(u32x2 w, float a, float b) {
  return u32x4{E::lo8(w[0], a), E::hi8(w[0], a), E::lo8(w[1], b), E::hi8(w[1], b)};
}

// The value the other half of the wave (lane ^ 32) holds.
__device__ __forceinline__ float other_half(float x) {
  return __shfl_xor(x, 32, 64);
}

// An output taken to another reference: an infinity stays one, however far the
// references lie apart (0 * inf would make it NaN).
__device__ __forceinline__ float rescaled(float x, float f) { return __builtin_isinf(x) ? x : x * f; }
__device__ __forceinline__ f32x4 rescaled(f32x4 x, float f) {
  return f32x4{rescaled(x[0], f), rescaled(x[1], f), rescaled(x[2], f), rescaled(x[3], f)};
}

// Whether any of 8 values is an infinity or a NaN.
template <class E>
__device__ __forceinline__ bool has_odd(u32x4 v) {
  uint32_t odd = 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) odd |= (v[x] & E::kExp) + E::kCarry;
  return (odd & 0x80008000u) != 0;
}
// Takes the infinities and NaN out of 8 values and leaves ones in their places: in
// `plus`, in `minus`, or for a NaN in both.
template <class E>
__device__ __forceinline__ void take_odd(u32x4& v, u32x4& plus, u32x4& minus) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    plus[x] = minus[x] = 0u;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint32_t w = (v[x] >> (16 * y)) & 0xffffu, big = E::kExp & 0x7fffu;
      if ((w & 0x7fffu) >= big) {
        if (w != (big | 0x8000u)) plus[x] |= E::kOne << (16 * y);
        if (w != big) minus[x] |= E::kOne << (16 * y);
        v[x] &= y ? 0x0000ffffu : 0xffff0000u;
      }
    }
  }
}

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2* lds_i32x2;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) const u32x4* lds_u32x4;

// Where piece c (8 values, 16 bytes) of row r of a K or V tile lies in LDS.
// K fragments read one piece of 16 consecutive rows at a time, V fragments four
// pieces of 4 consecutive rows: the piece's place within the row is turned by the
// row's number so that either read touches every bank once.
template <int D>
__device__ __forceinline__ int k_at(int r, int c) {
  return r * (2 * D) + ((c ^ (D == 64 ? (r >> 1) & 7 : r & 15)) << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int r, int c) {
  return r * (2 * D) + ((c ^ (D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2)) << 4);
}

__device__ __forceinline__ uint32_t lds_of(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// One 16-byte global->LDS load a lane: lane l's bytes land at byte 16 l of the
// 1 KiB block at `lds`.  In assembly, so that the compiler neither drains every
// LDS read for it nor counts it; its completion is awaited explicitly.  (One wait
// state between the M0 write and the load that reads it.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <bool NT>
__device__ __forceinline__ void dma16(uint32_t lds, const void* src) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(at), "v"(src)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src)
                 : "memory", "m0");
}
// One 4-byte load a lane, to byte 4 l of the 256 bytes at `lds`.
__device__ __forceinline__ void dma4(uint32_t lds, const void* src) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}
// The same from a wave-uniform address and a 32-bit byte offset of each lane.
__device__ __forceinline__ void dma16_at(uint32_t lds, const void* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// A value that every lane of the wave holds, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ const u32x4 g_zero = {0u, 0u, 0u, 0u};  // read in place of keys outside a run
__device__ const float g_one = 1.f;                // and of their scales

// Caps of scores: none; kCapShort, by 1 - 2 / (e^{2y} + 1) for tanh(y), which is off
// by up to 2^-21 of the cap, near zero too; kCap, where scores under a quarter of the
// cap go by the series of tanh, off by 2^-19 of the score at most.  Chunks take the
// short form for caps up to kMostShort, where it is off by 3e-5 at most, a tenth of
// what rounding the weights to fp16 is (2,048 tokens over 32,768: 1,154 us, 1,758 in
// the long form, 912 without a cap); decode, bound by memory, always the long one.
enum Cap { kNoCap, kCapShort, kCap };
constexpr float kMostShort = 64.f;

// How far a capped score lies under the cap, over twice the cap: with
// p.scale = 2 log2(e) scale / softcap, tanh(y) = 1 - 2 / (e^{2y} + 1).
__device__ __forceinline__ float under_cap(const AttnParams& p, float x) {
  return __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * p.scale) + 1.f);
}

// Score in log2 units.
template <Cap CAP>
__device__ __forceinline__ float score(const AttnParams& p, float x) {
  if constexpr (CAP == kNoCap) return x * p.scale;
  const float far = __builtin_fmaf(under_cap(p, x), -2.f * p.cap, p.cap);
  if constexpr (CAP == kCapShort) return far;
  const float y = x * p.scale * (0.5f * kLn2), t = y * y;
  const float r = __builtin_fmaf(__builtin_fmaf(t, -17.f / 315.f, 2.f / 15.f), t, -1.f / 3.f);
  const float near_ = p.cap * __builtin_fmaf(r * t, y, y);  // (what is left out: 62/2835 y^9)
  return fabsf(y) < 0.25f ? near_ : far;
}

// ------------------------------------------------------------------ chunks
//
// The tiles of kRows query rows, each against its own run of key tiles, are listed
// with the running total of their key tiles (make_plan).  The total over all
// kv-heads is cut into equal shares, one a workgroup and one workgroup a compute
// unit, so the chip is full and even whatever the batch: a run that crosses shares
// is joined afterwards from its parts' (m, l, o).  Starting and ending a tile of
// rows counts as kTileCost keys (a whole prompt of 16,384 tokens, tiles of 1 to 256
// key tiles: 1,318 us without, 988 with).
//
// A workgroup is four waves, one a SIMD, with 32 NQ rows each; at NQ = 2 a K or V
// fragment read from LDS feeds two products, which keeps the LDS reads at half
// the matrix time.  Nothing else runs on the SIMD, so a wave overlaps its own
// work: beside the exponentials of a block of 32 keys, the matrix unit works on
// the block before's product with V and on the block after's scores.  Keys arrive
// by global->LDS loads three tiles ahead, values two, with one barrier a tile.
//
// Bound by the matrix unit and, beside it, the vector operations: at D 128 a wave
// has 64 products of 32 cycles a tile, and beside them 64 exponentials of 12 cycles
// and 167 other operations of 4 to 8.
// Measured over several cards, bf16: 2,048 tokens over 32,768, 32 q-heads on 8 of 128
// values, 911 to 959 us, 1,182 to 1,244 TFLOP/s (a library matrix product of 8192^3
// reaches 1,347), of 64 values 600 to 605 us, 938 to 943; 4 ragged prompts, 16 q-heads
// on 2 of 256 values, 231 to 244 us, 909 to 960; 17 tokens over 1,000 21 us, most of
// it start and join.  In fp16, whose references move: 1,040 to 1,096 us (1,034 to
// 1,090 TFLOP/s), 655 to 670 and 252 to 261.
//
// Weights enter the product with V rounded to the element type: a second product
// for what the rounding loses would cost a third of the time, and the rounding adds
// 1.5e-3 of the output (bf16; in the mean) to the 1.6e-3 of the output's own.  In fp16
// it adds 1.7e-4 to 2.1e-4, and besides up to 2^-32 of the row's sum a weight, the
// type's least step: 2^17 keys that share 2% of a row are off by 1.5e-3 at most.

// Sizes of the chunk kernel.
template <int D, bool Q8>
struct Chunk {
  static constexpr int kNQ = D == 256 ? 1 : 2;      // 32-row blocks of a wave
  static constexpr int kRows = 32 * kNQ * kWaves;   // query rows of a tile
  static constexpr int kKeys = D == 256 ? 32 : 64;  // keys of a tile
  // tiles of K and of V in LDS: K's loads run three tiles ahead, V's two; the keys of a tile's later
  // blocks are still read while its first is worked on
  static constexpr int kSlotsK = Q8 || kKeys == 32 ? 3 : 4, kSlotsV = Q8 ? 2 : 3;
  static constexpr int kPlaces = Q8 ? 1024 : 2048;  // places of rows staged at a time (see `places`)
  // A load instruction brings kLoadRows rows into one block of 1 KiB.  In a block of K a row's 16-byte
  // pieces stay in order, but for the lowest bits of their number, turned by the row's; blocks lie
  // kPadK bytes further apart than 1 KiB: 16 rows of one piece then touch every bank once, and a
  // fragment's address is one of kTurnsK registers and an immediate.  In a block of V the 64-byte
  // quarter-, half- or eighth-rows that one product takes lie together, row by row, so that the
  // transposed read of four rows covers 256 bytes in one piece.
  static constexpr int kLoadRows = 512 / D;
  static constexpr int kTurnsK = D == 256 ? 1 : 2;
  static constexpr int kBlockK = 1024 + (D == 256 ? 32 : 64), kBlockV = 1024 + (D == 256 ? 128 : 0);
  static constexpr int kBlocks = kKeys / kLoadRows;  // of a tile
  static constexpr int kSlotK = kBlocks * kBlockK, kSlotV = kBlocks * kBlockV;  // bytes of a tile
  // Codes of a wave's rows of a tile, of the keys or the values: bytes, load instructions, rows and 16-code pieces of
  // one of those, and tiles on the way.
  static constexpr int kCodes = Q8 ? kKeys / kWaves * D : 0, kCodeLoads = kCodes / 1024;
  static constexpr int kCodeRows = 1024 / D, kCodePieces = D / 16, kCodeTiles = 2;
  static __device__ __forceinline__ int turn_k(int r) { return D == 64 ? (r >> 1) & 3 : D == 128 ? r & 3 : r & 1; }
  // piece c of row r of a tile
  static __device__ __forceinline__ int k_at(int r, int c) {
    return r / kLoadRows * kBlockK + r % kLoadRows * 2 * D + ((c ^ turn_k(r)) << 4);
  }
  static __device__ __forceinline__ int v_at(int r, int c) {
    return r / kLoadRows * kBlockV + (c >> 2) * (64 * kLoadRows) + r % kLoadRows * 64 + ((c & 3) << 4);
  }
  // A batch that may have more tiles than these is planned by a kernel of its own; otherwise every
  // workgroup lists them for itself, which saves the launch (17 tokens over 1,000: 26.3 -> 24.6 us).
  static constexpr int kFewTiles = 64 * kWaves;
  static constexpr int kPlanLds = kFewTiles * (32 + 8 + 20) + 8;  // (TileRec, running totals, SeqRec)
  static constexpr int kPlaceBytes = Q8 ? 16 : 8;
  static constexpr int kLds = kPlanLds + kSlotsK * kSlotK + kSlotsV * kSlotV + kPlaces * kPlaceBytes +
                              2 * kCodeTiles * kWaves * kCodes;
  static_assert(kLds <= 160 * 1024);
};

// A tile of query rows: its first row in its sequence, the keys it sees, and the
// sequence's new tokens, tokens and first page.  Where first tokens stay visible
// beside a window (sinks) and the window of some row begins behind them, the tile has
// their tiles of keys first, which show them alone, and then the window's, which show
// the rest: key numbers from `firsts` on, the end of their tiles, are the tokens' less
// `gap` (kNoGap: not so; -1 tile: one of both is read twice).
struct TileRec {
  int row0, key_begin, key_end, tok0, n, len, first_page, gap;
};
constexpr int kNoGap = INT32_MIN;
__device__ __forceinline__ int end_of_firsts(const AttnParams& p, int keys) { return (p.sinks + keys - 1) / keys * keys; }
// What plan_kernel says of the list: tiles, what each costs besides its key tiles,
// and what one kv-head costs in all.
struct PlanHead {
  int tiles, cost;
  int64_t per_head;
};
// A sequence: tiles before its own, first new token and their number, first page,
// and tokens.
struct SeqRec {
  int before, tok0, n, first_page, len;
};
// A tile that a share leaves unfinished: how many parts it has (0: none), the
// share that starts it, its first row, its sequence's first new token and their
// number, and its kv-head.
struct Unfinished {
  int parts, share, row0, tok0, n, hk, unused[2];
};

constexpr int kTileCost = 512;  // what starting and ending a tile costs, in keys
constexpr int kMinShare = 2;    // key tiles of a share at least: fewer parts to join

// a / b of units: 32 bits, but for a batch of 2^31 units and more
__device__ __forceinline__ int64_t div_units(int64_t a, int64_t b) {
  return (a | b) >> 31 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// One workgroup lists every sequence's tiles and the running total of their key
// tiles (of one kv-head), [tiles + 1].  seqs: room for B.
__device__ __forceinline__ PlanHead make_plan(const AttnParams& p, int rows, int keys, int shares, SeqRec* seqs,
                                              TileRec* tiles, int64_t* before) {
  const int B = p.kv.B, G = (int)p.group.d, threads = blockDim.x;
  // tiles before each sequence
  const int per = (B + threads - 1) / threads;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int tok0 = p.cu[b], tok1 = p.cu[b + 1], f = p.kv.ptr[b], e = p.kv.ptr[b + 1], last = p.kv.lpl[b];
    const int n = max(0, tok1 - tok0);
    seqs[b] = SeqRec{mine, tok0, n, f, e > f ? (e - f - 1) * (int)p.kv.page.d + last : 0};
    mine += (int)(((int64_t)n * G + rows - 1) / rows);
  }
  int total;
  const int at = block_exclusive_scan(mine, &total);
  for (int b = b0; b < b1; ++b) seqs[b].before += at;
  __syncthreads();
  int64_t run = 0;
  for (int i0 = 0; i0 < total; i0 += threads) {
    const int i = i0 + (int)threadIdx.x;
    int x = 0;
    if (i < total) {
      int lo = 0, hi = B - 1;  // the last sequence that starts at tile i or before has it
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seqs[mid].before <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const SeqRec q = seqs[lo];
      TileRec r{(i - q.before) * rows, 0, 0, q.tok0, q.n, q.len, q.first_page, kNoGap};
      const int past = r.len - r.n;
      const int first = (int)div_by((uint32_t)r.row0, p.group);
      const int last = min(r.n - 1, (int)div_by((uint32_t)r.row0 + rows - 1, p.group));
      r.key_end = p.causal ? max(0, min(past + last + 1, r.len)) : r.len;
      r.key_begin = p.window > 0 ? min(r.key_end, max(0, past + first - p.window + 1) / keys * keys) : 0;
      if (p.sinks > 0) {  // (with a window)
        if (past + last - p.window + 1 > p.sinks && r.key_end > p.sinks) {
          r.gap = max(r.key_begin, p.sinks / keys * keys) - end_of_firsts(p, keys);
          r.key_end -= r.gap;
        }
        r.key_begin = 0;
      }
      tiles[i] = r;
      x = max(1, (r.key_end - r.key_begin + keys - 1) / keys);  // a tile without keys still writes its rows
    }
    int sum;
    const int so_far = block_exclusive_scan(x, &sum);
    if (i < total) before[i] = run + so_far;
    run += sum;
  }
  if (threadIdx.x == 0) before[total] = run;
  // a tile costs as many key tiles more than it has, or less where shares are small
  const int cost = (int)min((int64_t)(kTileCost / keys), div_units(run * p.Hkv, 4 * (int64_t)shares));
  return PlanHead{total, cost, run + (int64_t)total * cost};
}

// The plan of a batch with more tiles than a workgroup lists by itself.
__global__ __launch_bounds__(1024) void plan_kernel(AttnParams p, int rows, int keys, int shares) {
  __shared__ SeqRec few[1024];
  const PlanHead h = make_plan(p, rows, keys, shares, p.kv.B <= 1024 ? few : (SeqRec*)p.seqs,
                               (TileRec*)p.tiles, p.before);
  if (threadIdx.x == 0) *(PlanHead*)p.head = h;
}

// The last tile that starts at most x in, each `cost` more than its key tiles (the whole wave searches).
__device__ __forceinline__ int find_tile(const int64_t* before, int tiles, int cost, int64_t x) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = tiles - 1;  // among before[1 .. tiles - 1]
  while (n > 0) {
    const int step = (n + 63) >> 6;
    const int64_t at = int64_t(lane + 1) * step;
    const int64_t i = lo + (at <= n ? at : 1);
    const int c = __popcll(__ballot(at <= n && before[i] + i * cost <= x));
    lo += c * step;
    n = step == 1 ? 0 : min(step - 1, n - c * step);
  }
  return lo;
}

// A lane's column of output (row in_tile of the tile, half of its values): the
// finished row, or, into part `part` >= 0, what the join needs.  A row that sees no
// token has a sum of -1, in its parts too; one whose scores are all -inf a sum of 0,
// and by the formula 0 / 0 for its output.
template <class E, int D>
__device__ __forceinline__ void store_rows(const AttnParams& p, const TileRec& rec, int hk, int in_tile,
                                           int64_t part, const f32x16 (&o)[D / 32], float m, float sum) {
  const int half = (threadIdx.x & 63) >> 5, row = rec.row0 + in_tile;
  const int tok0 = rec.tok0, tok = (int)div_by(row, p.group), g = row - tok * (int)p.group.d;
  if (tok >= rec.n) return;
  if (part < 0) {
    const bool none = sum < 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int64_t h = (int64_t)hk * p.group.d + g;
    u16* dst = (u16*)p.o.p + (int64_t)(tok0 + tok) * p.o.ts + h * p.o.hs;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(u32x2*)(dst + 32 * d + 8 * i + 4 * half) = u32x2{E::pack(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                                                           E::pack(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
    if (p.lse && half == 0)
      p.lse[(int64_t)(tok0 + tok) * p.Hq + h] = none ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * kLn2;
  } else {
    float* dst = p.part_o + (part * p.part_rows + in_tile) * D;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(f32x4*)(dst + 32 * d + 8 * i + 4 * half) = f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (half == 0) {
      p.part_ml[(part * p.part_rows + in_tile) * 2] = m;
      p.part_ml[(part * p.part_rows + in_tile) * 2 + 1] = sum;
    }
  }
}

// The first argument of the kernel, its fields loaded anew where they are asked for:
// what is needed once a run does not stay in scalar registers in between, of which the
// chunk kernel with sinks has too few.
__device__ __forceinline__ const AttnParams& reloaded() {
  typedef const AttnParams __attribute__((address_space(4))) * Args;
  Args p = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnParams*)p;
}

// EVEN: a wave's rows of a tile lie in one page (see launch_chunk).
// Q8: the cache holds e4m3 codes.  A wave loads its rows' codes into LDS of its own,
// and a tile ahead writes them as values, times their scales, to the slots that the
// products read: exact (a power of two times 4 bits), once a tile and workgroup, where
// codes as operands would be converted by each of the four waves.  The results are
// those of a 16-bit cache of the same values, bit for bit.  The conversions and their
// LDS traffic stand beside the products: 2,048 tokens over 32,768 978 to 1,070 us over
// several cards, 980 where a 16-bit cache takes 927 (188 M vector instructions against
// 165 M).  Their writes of V meet in the banks; laid
// out so that they do not, they took the same time.
// SINKS: first tokens stay visible beside a window.  A run is then its first tokens' key
// tiles and those of the window, in one row of tiles (TileRec): the parts of one run
// share a softmax and need no join of their own.  Kernels of their own: the questions
// cost the scalar registers that calls without sinks need (their chunks were 2% slower).
// 3,007 new tokens of two sequences with a window of 2,000 and 64 first tokens 132 to 143
// us, 0 to 4 of them the first tokens'.
template <class E, int D, Cap CAP, bool EVEN, bool Q8, bool SINKS>
__global__ __launch_bounds__(64 * kWaves, 1) void chunk_kernel(AttnParams p) {
  typedef Chunk<D, Q8> C;
  static_assert(EVEN || !Q8);
  constexpr int NQ = C::kNQ, NSK = C::kSlotsK, NSV = C::kSlotsV, KB = C::kKeys / 32;
  constexpr int kSteps = D / 16;   // MFMA steps over D
  constexpr int kBlocks = D / 32;  // 32-wide blocks of the output
  constexpr int kLoads = C::kBlocks / kWaves;  // load instructions of a wave for a tile of K or V
  constexpr int kRowsW = C::kKeys / kWaves;    // rows they cover
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  // Where rows of the run's keys lie in the caches, in bytes from the start of their kv-head: of every
  // kRowsW-th row, or of every row when pages may end between them
  int64_t* places = (int64_t*)(smem + NSK * C::kSlotK + NSV * C::kSlotV);
  // (of codes: with the scales of the keys and of the values, which a wave's rows of a tile share)
  struct Place8 {
    int64_t at;
    float k, v;
  };
  Place8* places8 = (Place8*)places;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = (int)p.group.d;

  char* own_plan = smem + NSK * C::kSlotK + NSV * C::kSlotV + C::kPlaces * C::kPlaceBytes;
  const TileRec* tile_recs = (const TileRec*)p.tiles;
  const int64_t* tile_before = p.before;
  PlanHead plan;
  if (p.head) {
    plan = *(const PlanHead*)p.head;
  } else {
    TileRec* recs = (TileRec*)own_plan;
    int64_t* before = (int64_t*)(own_plan + C::kFewTiles * sizeof(TileRec));
    plan = make_plan(p, C::kRows, C::kKeys, gridDim.x, (SeqRec*)(before + C::kFewTiles + 1), recs, before);
    tile_recs = recs;
    tile_before = before;
    __syncthreads();
  }
  const int num_tiles = uniform(plan.tiles), cost = uniform(plan.cost);
  const int64_t per_head = uniform64(plan.per_head), units = per_head * p.Hkv;
  const int64_t share = max((int64_t)kMinShare, div_units(units + gridDim.x - 1, gridDim.x));
  // neighbouring shares on one XCD (workgroup x runs on XCD x % 8)
  const int shares8 = gridDim.x >> 3;
  const int me = (gridDim.x & 7) ? blockIdx.x : (blockIdx.x & 7) * shares8 + (blockIdx.x >> 3);
  const int64_t first = (int64_t)me * share, end = min(units, first + share);
  // records of unfinished tiles: one a tile where the batch has few (p.records of them at most; those
  // past the last tile say that there is none), one a share otherwise
  Unfinished* records = (Unfinished*)p.parts;
  if (p.records) {
    if (tid == 0 && me < p.records && me >= num_tiles * p.Hkv) records[me].parts = 0;
  } else if (first >= end && tid == 0) {
    records[me].parts = 0;
  }
  if (first >= end) return;
  bool off = false;
  int hk = uniform((int)div_units(first, per_head));
  int ti = uniform(find_tile(tile_before, num_tiles, cost, first - hk * per_head));
  bool left = false;

  // What each lane loads (the piece that belongs at its place in the block), and where that is from
  // the first row of the wave's part of a tile
  const int kr = lane / (D / 8), vr = (lane >> 2) % C::kLoadRows;
  const uint32_t piece_v = 16 * ((lane >> 2) / C::kLoadRows * 4 + (lane & 3));
  uint32_t piece_k[kLoads], off_k[kLoads], off_v[kLoads];
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int r = x * C::kLoadRows;
    piece_k[x] = 16 * ((lane % (D / 8)) ^ C::turn_k(wave * kRowsW + r + kr));
    off_k[x] = (uint32_t)(2 * (r + kr) * p.kv.ts) + piece_k[x];
    off_v[x] = (uint32_t)(2 * (r + vr) * p.kv.ts) + piece_v;
  }
  // and where its fragments start in a slot: of K's first steps, and of V (lane i of a 16-lane group
  // points at 4 values of key i / 4 and receives value i of four keys)
  uint32_t frag_k[C::kTurnsK];
#pragma unroll
  for (int t = 0; t < C::kTurnsK; ++t) frag_k[t] = C::k_at(col, 2 * t + half);
  const uint32_t frag_v = 8 * (lane & 1) +
                          C::v_at(4 * half + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1));

  const uint32_t token_bytes = (uint32_t)((Q8 ? 1 : 2) * p.kv.ts);
  // codes: this lane's piece of a load, this wave's codes (the keys' tiles, then the values'), and where this lane's
  // 16 values go in a slot: two pieces, side by side but for K's turn
  const uint32_t off_c = (uint32_t)(lane / C::kCodePieces * p.kv.ts) + 16 * (lane % C::kCodePieces);
  const uint32_t codes0 = lds_of(smem) + NSK * C::kSlotK + NSV * C::kSlotV + C::kPlaces * C::kPlaceBytes + C::kPlanLds +
                          wave * (2 * C::kCodeTiles * C::kCodes);
  const int row_c = wave * kRowsW + lane / C::kCodePieces, piece_c = 2 * (lane % C::kCodePieces);
  const uint32_t to_k = C::k_at(row_c, piece_c), to_v = C::v_at(row_c, piece_c);

  for (;;) {
    TileRec rec = tile_recs[ti];
    rec = TileRec{uniform(rec.row0), uniform(rec.key_begin), uniform(rec.key_end), uniform(rec.tok0),
                  uniform(rec.n), uniform(rec.len), uniform(rec.first_page), uniform(rec.gap)};
    const bool apart = SINKS && rec.gap != kNoGap;
    const int firsts = apart ? end_of_firsts(p, C::kKeys) : 0, gap = apart ? rec.gap : 0;
    // this share's part of the tile's key tiles: from `done` on (those before are the share before's)
    const int64_t start = hk * per_head + uniform64(tile_before[ti]) + (int64_t)ti * cost;
    const int tiles = uniform((int)(tile_before[ti + 1] - tile_before[ti]));
    const int done = (int)max((int64_t)0, first - start - cost);
    const int todo = (int)min((int64_t)tiles, end - start - cost) - done;
    if (todo > 0) {
      const int tok0 = rec.tok0, n = rec.n, first_page = rec.first_page, len = rec.len, past = len - n;

      // this lane's rows
      int lim[NQ], low[NQ];  // keys low .. lim (SINKS: of those from `firsts` on)
      u32x4 q[NQ][kSteps];
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        const int row = rec.row0 + wave * 32 * NQ + a * 32 + col;
        const int tok = (int)div_by(row, p.group), g = row - tok * G;
        const bool real = tok < n;
        lim[a] = real ? (p.causal ? min(past + tok, len - 1) : len - 1) : -1;
        low[a] = real && p.window > 0 ? max(0, past + tok - p.window + 1) : 0;
        if constexpr (SINKS) {
          low[a] = apart ? max(low[a], p.sinks) - gap : 0;  // (the sinks reach every row's window)
          lim[a] = lim[a] < 0 ? -1 : lim[a] - gap;
        }
        const u16* src = (const u16*)p.q.p + (int64_t)(tok0 + (real ? tok : 0)) * p.q.ts +
                         (int64_t)(hk * G + (real ? g : 0)) * p.q.hs + 8 * half;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[a][s] = *(const u32x4*)(src + 16 * s);
      }
      // keys all_low .. all_lim are seen by every row of the wave and need no mask
      int all_lim = 0x7fffffff, all_low = 0;
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        const int row = rec.row0 + wave * 32 * NQ + a * 32 + col;
        if ((int)div_by(row, p.group) < n) all_lim = min(all_lim, lim[a]);
        all_low = max(all_low, low[a]);
      }
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        all_lim = min(all_lim, __shfl_xor(all_lim, x, 64));
        all_low = max(all_low, __shfl_xor(all_low, x, 64));
      }
      all_lim = __builtin_amdgcn_readfirstlane(all_lim);
      all_low = __builtin_amdgcn_readfirstlane(all_low);

      const int key_a = rec.key_begin + done * C::kKeys;
      const int key_b = min(rec.key_end, key_a + todo * C::kKeys);
      const char* kbase = p.kv.k + (Q8 ? 1 : 2) * (int64_t)hk * p.kv.hs;
      const char* vbase = p.kv.v + (Q8 ? 1 : 2) * (int64_t)hk * p.kv.hs;

      f32x16 o[NQ][kBlocks];
      float m[NQ], l[NQ];
      constexpr int step = EVEN ? kRowsW : 1;

#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        m[a] = lim[a] < 0 ? 0.f : kNoScore;
        l[a] = 0.f;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[a][d][i] = 0.f;
      }

      // as many tiles at a time as the staged places reach, and the first tokens' by themselves
      for (int a0 = key_a; a0 < key_b;) {
        const bool few = SINKS && a0 < firsts;
        const int sinks = SINKS ? p.sinks : 0;
        const int a1 = (int)min((int64_t)(few ? min(sinks, key_b) : key_b), a0 + (int64_t)C::kPlaces * step);
        const int count = (a1 - a0 + C::kKeys - 1) / C::kKeys;
        __syncthreads();
        // (codes: a place for every wave's rows of the last tile, past the end with a scale of one for its zeros)
        const AttnParams& args = SINKS ? reloaded() : p;
        const int staged = Q8 ? a0 + count * C::kKeys : a1;
        for (int x = tid; a0 + x * step < staged; x += 64 * kWaves) {
          int key = a0 + x * step;
          if (Q8 && key >= a1) {
            places8[x] = Place8{0, 1.f, 1.f};
            continue;
          }
          if (SINKS && key >= firsts) key += gap;
          const int pg = (int)div_by(key, args.kv.page), off = key - pg * (int)args.kv.page.d;
          const int64_t id = args.kv.idx[first_page + pg];
          if constexpr (Q8) {
            const int64_t sc = id * args.scales.ps + (int64_t)div_by(off, args.scales.block) * args.scales.bs + hk * args.scales.hs;
            places8[x] = Place8{id * args.kv.ps + (int64_t)off * args.kv.ts, args.scales.k[sc], args.scales.v[sc]};
          } else {
            places[x] = 2 * (id * args.kv.ps + (int64_t)off * args.kv.ts);
          }
        }
        __syncthreads();

        // This wave's rows of a tile: one place when they lie in one page and are all there, otherwise
        // each lane's own (-1: past the end, zeros).  A tile's keys and, an iteration later, its values
        // go by the same places; `next` is read from LDS a tile ahead.
        const int last_place = EVEN ? (a1 - a0 - 1) / C::kKeys : 0;
        bool one;
        int64_t at, next = Q8 ? 0 : places[wave];
        int64_t lane_at[kLoads][2];
        auto advance = [&](int i) __attribute__((always_inline)) {
          at = uniform64(next);
          next = places[min(i + 1, last_place) * kWaves + wave];
        };
        auto place = [&](int i) __attribute__((always_inline)) {
          const int key0 = a0 + i * C::kKeys + wave * kRowsW;
          one = EVEN && key0 + kRowsW <= a1;
          advance(i);
          if (!one) {
#pragma unroll
            for (int x = 0; x < 2 * kLoads; ++x) {
              const int r = x / 2 * C::kLoadRows + (x & 1 ? vr : kr);
              const int64_t to = EVEN ? at + r * (int64_t)token_bytes : places[min(key0 + r, a1 - 1) - a0];
              lane_at[x / 2][x & 1] = key0 + r < a1 ? to : -1;
            }
          }
        };
        // load x of the placed tile's keys (or V: values) into a slot, from one place
        auto load_one = [&](uint32_t slot, bool V, int x) __attribute__((always_inline)) {
          const uint32_t dst = slot + (wave * kLoads + x) * (V ? C::kBlockV : C::kBlockK);
          dma16_at(dst, (V ? vbase : kbase) + at, V ? off_v[x] : off_k[x]);
        };
        auto load = [&](uint32_t slot, bool V) __attribute__((always_inline)) {
          if (one) {
#pragma unroll
            for (int x = 0; x < kLoads; ++x) load_one(slot, V, x);
          } else {
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
              const char* src = (V ? vbase : kbase) + lane_at[x][V] + (V ? piece_v : piece_k[x]);
              dma16<false>(slot + (wave * kLoads + x) * (V ? C::kBlockV : C::kBlockK),
                           lane_at[x][V] < 0 ? (const char*)&g_zero : src);
            }
          }
        };
        // The same inside the run, where pages end anywhere: every lane takes its row's place from LDS, a
        // part before its load.
        const int full = (a1 - a0) / C::kKeys;
        constexpr int kAhead = (2 * kLoads + 4 * KB - 1) / (4 * KB);
        int64_t ahead[kAhead];
        auto look = [&](int i, int part) __attribute__((always_inline)) {
#pragma unroll
          for (int y = part * 2 * kLoads / (4 * KB); y < (part + 1) * 2 * kLoads / (4 * KB); ++y) {
            const bool V = y < kLoads;
            const int x = V ? y : y - kLoads;
            ahead[y - part * 2 * kLoads / (4 * KB)] =
                places[min(i + (V ? 2 : 3), full - 1) * C::kKeys + wave * kRowsW + x * C::kLoadRows + (V ? vr : kr)];
          }
        };
        // Codes of this wave's rows of tile i, keys or values, on the way to its LDS (WHOLE: rows that are all there;
        // otherwise those past the end are zeros), and a piece of them written as values to a slot.  Tile i's keys go
        // by way of buffer i % 2, its values too.
        auto ask = [&](auto whole, bool V, int i, const char* from) __attribute__((always_inline)) {
          const uint32_t dst = codes0 + ((V ? C::kCodeTiles : 0) + (i & 1)) * C::kCodes;
          const char* base = (V ? vbase : kbase) + (int64_t)from;
#pragma unroll
          for (int x = 0; x < C::kCodeLoads; ++x) {
            if constexpr (decltype(whole)::value) {
              dma16_at(dst + x * 1024, base, off_c + x * C::kCodeRows * token_bytes);
            } else {
              const int key = a0 + i * C::kKeys + wave * kRowsW + x * C::kCodeRows + lane / C::kCodePieces;
              dma16<false>(dst + x * 1024,
                           key < a1 ? base + off_c + x * C::kCodeRows * token_bytes : (const char*)&g_zero);
            }
          }
        };
        const int last8 = (a1 - a0 - 1) / C::kKeys;  // (as last_place)
        auto place8 = [&](int i) __attribute__((always_inline)) { return places8[min(i, last8) * kWaves + wave]; };
        auto codes = [&](bool V, int i, int x) __attribute__((always_inline)) {
          return *(lds_u32x4)(codes0 + ((V ? C::kCodeTiles : 0) + (i & 1)) * C::kCodes + x * 1024 + lane * 16);
        };
        auto put = [&](bool V, uint32_t slot, int x, u32x4 w, float sc) __attribute__((always_inline)) {
          const uint32_t to = slot + (V ? to_v : to_k) + x * (C::kCodeRows / C::kLoadRows * (V ? C::kBlockV : C::kBlockK));
          typedef __attribute__((address_space(3))) u32x4* lds_out;
          *(lds_out)(to) = values8<E>(u32x2{w[0], w[1]}, sc, sc);
          *(lds_out)(V ? to + 16 : to ^ 16) = values8<E>(u32x2{w[2], w[3]}, sc, sc);
          asm volatile("" ::"v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]));  // (read, before the codes after them land)
        };
        // tile i's values and tile i + 1's keys are in LDS, and every wave is done with tile i - 1's values
        // and keys (codes: tile i + 1's values and tile i + 2's keys, of this wave, are there as well)
        auto arrive = [&]() __attribute__((always_inline)) {
          wait_vm<Q8 ? 2 * C::kCodeLoads : 2 * kLoads>();
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        };

        // The slots of tile i's keys and values, of tile i + 1's keys, and those that tile i - 1 leaves free,
        // as addresses in LDS.
        const uint32_t keys0 = lds_of(smem), values0 = keys0 + NSK * C::kSlotK;
        uint32_t k_now = keys0, k_next = keys0 + C::kSlotK, k_free = keys0 + (NSK - 1) * C::kSlotK;
        uint32_t v_now = values0, v_free = values0 + (NSV - 1) * C::kSlotV;
        auto turn = [&]() __attribute__((always_inline)) {
          k_free = k_now;
          k_now = k_next;
          k_next = k_next == keys0 + (NSK - 1) * C::kSlotK ? keys0 : k_next + C::kSlotK;
          v_free = v_now;
          v_now = v_now == values0 + (NSV - 1) * C::kSlotV ? values0 : v_now + C::kSlotV;
        };
        // (where the keys go that tile i asks for, three tiles ahead)
        auto k_ahead = [&]() __attribute__((always_inline)) { return NSK == 4 ? k_free : k_now; };

        // K fragments t0 .. t1 of block kb (32 keys) of the tile in a slot
        u32x4 kf[kSteps];
        auto read_k = [&](uint32_t slot, int kb, int t0, int t1) __attribute__((always_inline)) {
          uint32_t from[C::kTurnsK];
#pragma unroll
          for (int t = 0; t < C::kTurnsK; ++t) {
            from[t] = frag_k[t] + slot;
            asm("" : "+v"(from[t]));  // (so that the rest goes into the reads' immediates)
          }
#pragma unroll
          for (int t = 0; t < kSteps; ++t)
            if (t >= t0 && t < t1)
              kf[t] = *(lds_u32x4)(from[t % C::kTurnsK] + t / C::kTurnsK * (32 * C::kTurnsK) +
                                   kb * 32 / C::kLoadRows * C::kBlockK);
        };
        // V fragments of half t of block kb of tile i: keys 16 t + 4 half + 0..3, and 8 more
        u32x2 vf[2][kBlocks][2];
        auto read_v = [&](int kb, int t) __attribute__((always_inline)) {
          uint32_t from = frag_v + v_now;
          asm("" : "+v"(from));
#pragma unroll
          for (int d = 0; d < kBlocks; ++d)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              vf[t][d][x] = __builtin_bit_cast(
                  u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                             (lds_s16x4)(from + (kb * 32 + 16 * t + 8 * x) / C::kLoadRows * C::kBlockV +
                                         d * (64 * C::kLoadRows))));
        };
        f32x16 s[NQ];
        auto scores = [&](int t0, int t1) __attribute__((always_inline)) {
          if (t0 == 0) {
#pragma unroll
            for (int a = 0; a < NQ; ++a)
#pragma unroll
              for (int e = 0; e < 16; ++e) s[a][e] = 0.f;
          }
#pragma unroll
          for (int t = 0; t < kSteps; ++t)
            if (t >= t0 && t < t1) {
#pragma unroll
              for (int a = 0; a < NQ; ++a) s[a] = E::mfma(kf[t], q[a][t], s[a]);
            }
        };
        // whether row block a sees the key of value e in the block of keys from key0 (this lane's keys are
        // 4 half + 8 (e / 4) + e % 4): span[a] keys from begin[a] on
        int begin[NQ];
        uint32_t span[NQ];
#pragma unroll
        for (int a = 0; a < NQ; ++a) {
          begin[a] = few ? 0 : low[a];
          span[a] = (uint32_t)max(0, few ? (lim[a] < 0 ? 0 : min(sinks, lim[a] + gap + 1)) : min(lim[a], a1 - 1) + 1 - low[a]);
        }
        auto seen = [&](int a, int e, int key0) __attribute__((always_inline)) {
          return (uint32_t)(8 * (e >> 2) + (e & 3) + (key0 + 4 * half - begin[a])) < span[a];
        };
        u32x4 pt[NQ][2], pw[NQ][2];
        float sum[NQ];
        // weights of values v0 .. v1 of a lane's 16 NQ
        auto weights = [&](auto mask, const f32x16 (&x)[NQ], int v0, int v1, int key0) __attribute__((always_inline)) {
#pragma unroll
          for (int a = 0; a < NQ; ++a)
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              if (16 * a + e >= v0 && 16 * a + e < v1) {
                float w0, w1;
                if constexpr (CAP == kCapShort) {
                  w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(under_cap(p, x[a][e]), -2.f * p.cap, p.cap - m[a]));
                  w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(under_cap(p, x[a][e + 1]), -2.f * p.cap, p.cap - m[a]));
                } else if constexpr (CAP == kCap) {
                  w0 = __builtin_amdgcn_exp2f(score<CAP>(p, x[a][e]) - m[a]);
                  w1 = __builtin_amdgcn_exp2f(score<CAP>(p, x[a][e + 1]) - m[a]);
                } else {
                  w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[a][e], p.scale, -m[a]));
                  w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[a][e + 1], p.scale, -m[a]));
                }
                if constexpr (decltype(mask)::value) {
                  w0 = seen(a, e, key0) ? w0 : 0.f;
                  w1 = seen(a, e + 1, key0) ? w1 : 0.f;
                }
                sum[a] = e == 0 ? w0 + w1 : sum[a] + w0 + w1;
                pw[a][e >> 3][(e >> 1) & 3] = E::pack(w0, w1);
              }
        };
        auto product = [&](int t) __attribute__((always_inline)) {
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) {
            const u32x4 f{vf[t][d][0][0], vf[t][d][0][1], vf[t][d][1][0], vf[t][d][1][1]};
#pragma unroll
            for (int a = 0; a < NQ; ++a) o[a][d] = E::mfma(f, pt[a][t], o[a][d]);
          }
        };
        // References for the rows that have none yet: kBias below the highest score that the row sees in the
        // block of scores at hand.
        auto refer = [&](const f32x16 (&x)[NQ], int key0) __attribute__((always_inline)) {
          bool none = false;
#pragma unroll
          for (int a = 0; a < NQ; ++a) none = none || m[a] == kNoScore;
          if (__any(none)) {
#pragma unroll
            for (int a = 0; a < NQ; ++a) {
              float top = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; ++e) top = fmaxf(top, seen(a, e, key0) ? score<CAP>(p, x[a][e]) : -INFINITY);
              top = fmaxf(top, other_half(top));
              if (m[a] == kNoScore && top > kNoScore) m[a] = top - E::kBias;
            }
          }
        };

        // Weights that outgrew the element type's range: their rows' references move to kBias below the highest
        // score of the block at hand, whose weights are taken again.
        auto move = [&](auto mask, const f32x16 (&x)[NQ], int key0) __attribute__((always_inline)) {
#pragma unroll
          for (int a = 0; a < NQ; ++a) {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!decltype(mask)::value || seen(a, e, key0)) top = fmaxf(top, score<CAP>(p, x[a][e]));
            top = fmaxf(top, other_half(top));
            const float to = fmaxf(m[a], top - E::kBias), f = __builtin_amdgcn_exp2f(m[a] - to);
            m[a] = to;
            l[a] *= f;
#pragma unroll
            for (int d = 0; d < kBlocks; ++d)
#pragma unroll
              for (int e = 0; e < 16; ++e) o[a][d][e] *= f;
          }
          weights(mask, x, 0, 16 * NQ, key0);
        };

        // One tile, block by block: the weights of a block, and beside them the product of the block
        // before with V and the scores of the block after, in four parts that each take their share of
        // the products, of the fragment reads for the next ones, of the weights and of the loads.
        // `inner`: a tile that every row of the wave sees whole, as the next one, all there and from
        // one place, so that nothing is asked inside it.
        auto tile = [&](auto inner, int i) __attribute__((always_inline)) {
          constexpr bool kInner = decltype(inner)::value;
          // codes: the pieces written as values in this tile, the next tile but one's keys and then the next one's
          // values, are read a part before; the codes asked for then take their places
          constexpr int kUnits = 2 * C::kCodeLoads, kParts = 4 * KB;
          u32x4 held{};
          float scale = 1.f;
          int64_t from = 0;
          // (the queries stay in accumulation registers, which the products read directly)
#pragma unroll
          for (int a = 0; a < NQ; ++a)
#pragma unroll
            for (int t = 0; t < kSteps; ++t) asm volatile("" : "+a"(q[a][t]));
          arrive();
          if constexpr (Q8) {
            scale = place8(i + 2).k;
            from = place8(i + 4).at;
            held = codes(false, i + 2, 0);
          }
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            f32x16 x[NQ];
#pragma unroll
            for (int a = 0; a < NQ; ++a) x[a] = s[a];
            const int nkb = kb + 1 < KB ? kb + 1 : 0;
            if constexpr (!kInner) refer(x, a0 + i * C::kKeys + kb * 32);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (g < 2) {
                product(g);
                read_k(nkb ? k_now : k_next, nkb, g * kSteps / 2, (g + 1) * kSteps / 2);
              } else {
                scores((g - 2) * kSteps / 2, (g - 1) * kSteps / 2);
                read_v(kb, g - 2);
              }
              weights(std::bool_constant<!kInner>(), x, g * 4 * NQ, (g + 1) * 4 * NQ, a0 + i * C::kKeys + kb * 32);
              const int part = kb * 4 + g;
              if constexpr (Q8) {
                // unit u is written in part u kParts / kUnits
                if (part * kUnits % kParts == 0) {
                  const int u = part * kUnits / kParts;
                  const bool V = u >= C::kCodeLoads;
                  put(V, V ? v_free : k_free, V ? u - C::kCodeLoads : u, held, scale);
                }
                if ((part + 1) * kUnits % kParts == 0 && part + 1 < kParts) {
                  const int u = (part + 1) * kUnits / kParts;
                  const bool V = u >= C::kCodeLoads;
                  held = codes(V, V ? i + 1 : i + 2, V ? u - C::kCodeLoads : u);
                  if (u == C::kCodeLoads) scale = place8(i + 1).v;
                }
                constexpr int kAskK = kUnits == kParts ? kParts / 2 : kParts / 2 - 1;
                if (part == kAskK) {
                  ask(std::bool_constant<kInner>(), false, i + 4, (const char*)uniform64(from));
                  from = place8(i + 3).at;
                }
                if (part == kParts - 1) ask(std::bool_constant<kInner>(), true, i + 3, (const char*)uniform64(from));
                if constexpr (kInner) {
#pragma unroll
                  for (int y = 0; y < kSteps * NQ / 2; ++y) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (y > 3) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                  }
                  __builtin_amdgcn_sched_barrier(0);
                }
              } else if constexpr (kInner) {
                if (EVEN && part == 2 * KB) advance(i + 3);
#pragma unroll
                for (int y = part * 2 * kLoads / (4 * KB); y < (part + 1) * 2 * kLoads / (4 * KB); ++y) {
                  const bool V = y < kLoads;
                  const int x = V ? y : y - kLoads;
                  if constexpr (EVEN) {
                    load_one(V ? v_free : k_ahead(), V, x);
                  } else {
                    dma16<false>((V ? v_free : k_ahead()) + (wave * kLoads + x) * (V ? C::kBlockV : C::kBlockK),
                                 (V ? vbase : kbase) + ahead[y - part * 2 * kLoads / (4 * KB)] + (V ? piece_v : piece_k[x]));
                  }
                }
                if constexpr (!EVEN) look(part + 1 < 4 * KB ? i : i + 1, (part + 1) % (4 * KB));
                // one product, from the fifth on a fragment read, then up to four vector operations, in turn
                // (2,048 tokens over 32,768: 928 us; reads where the compiler puts them 950 to 975, with
                // every product 969, from the third on 972)
#pragma unroll
                for (int y = 0; y < kSteps * NQ / 2; ++y) {
                  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                  if (y > 3) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                  __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
              } else {
                if (part == 0) load(v_free, true);
                if (part == 2 * KB) {
                  place(i + 3);
                  load(k_ahead(), false);
                }
              }
            }
            if constexpr (E::kMoves) {
              float most = sum[0];
#pragma unroll
              for (int a = 1; a < NQ; ++a) most = fmaxf(most, sum[a]);
              // (D 64 and 128: the weights are packed beside the products, not behind the branch: 2,048 tokens
              // over 32,768 1,082 -> 1,062 us; at D 256 the compiler does better by itself, 254 against 260, and
              // with a cap it would spill)
              if constexpr (NQ == 2 && CAP == kNoCap) {
#pragma unroll
                for (int e = 0; e < 8 * NQ; ++e) asm volatile("" ::"v"(pw[e >> 3][(e >> 2) & 1][e & 3]));
              }
              if (__any(most > E::kMost)) move(std::bool_constant<!kInner>(), x, a0 + i * C::kKeys + kb * 32);
            }
#pragma unroll
            for (int a = 0; a < NQ; ++a) {
              l[a] += sum[a];
#pragma unroll
              for (int t = 0; t < 2; ++t) pt[a][t] = pw[a][t];
            }
          }
          turn();
        };
        if constexpr (Q8) {
          const std::false_type some;
          auto from = [&](int i) __attribute__((always_inline)) { return (const char*)uniform64(place8(i).at); };
          ask(some, false, 0, from(0));
          ask(some, false, 1, from(1));
          ask(some, true, 0, from(0));
          ask(some, true, 1, from(1));
          wait_vm<C::kCodeLoads>();
#pragma unroll
          for (int x = 0; x < C::kCodeLoads; ++x) {
            put(false, keys0, x, codes(false, 0, x), place8(0).k);
            put(false, keys0 + C::kSlotK, x, codes(false, 1, x), place8(1).k);
            put(true, values0, x, codes(true, 0, x), place8(0).v);
          }
          ask(some, false, 2, from(2));
          ask(some, false, 3, from(3));
          ask(some, true, 2, from(2));
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        } else {
#pragma unroll
          for (int x = 0; x < 3; ++x) {
            place(x);
            load(keys0 + x * C::kSlotK, false);
            if (x < 2) load(values0 + x * C::kSlotV, true);
          }
          wait_vm<4 * kLoads>();
          asm volatile("s_barrier" ::: "memory");
        }
        read_k(keys0, 0, 0, kSteps);
        scores(0, kSteps);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int a = 0; a < NQ; ++a) pt[a][t] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) vf[t][d][0] = vf[t][d][1] = u32x2{0u, 0u};
        }
        refer(s, a0);
        // Tiles inner0 .. inner1 are seen whole by every row of the wave, and every row has its reference
        // (those that see the first block have it now, the others from the tile that `all_low` lies in);
        // the loads they ask for are of whole tiles or of none.
        const int inner0 = few ? count : all_low <= a0 ? 0 : min(count, (all_low - a0) / C::kKeys + 1);
        const int inner1 = min(full < count ? full - (Q8 ? 4 : 3) : full, (min(all_lim, a1 - 1) - a0 + 1) / C::kKeys);
        int i = 0;
        for (; i < inner0; ++i) tile(std::false_type(), i);
        if (!EVEN && i < inner1) look(i, 0);
        for (; i < inner1; ++i) tile(std::true_type(), i);
        if (!EVEN && inner0 < inner1) place(i + 2);  // (what the next tile's values go by)
        // (the scores after the last block are of zeros, and nobody's)
        for (; i < count; ++i) tile(std::false_type(), i);
        product(0);
        product(1);
        wait_vm<0>();
        a0 = few && a1 == p.sinks ? firsts : a1;
      }

      const AttnParams& args = SINKS ? reloaded() : p;
      const bool whole = done == 0 && todo == tiles;
      const bool head = done > 0;  // a part that continues a run: slot 0, one that starts it: slot 1
      const int64_t part = whole ? -1 : 2 * (int64_t)me + (head ? 0 : 1);
      // a row whose weights overflowed, or whose outputs are not finite: the share is computed again
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        l[a] += other_half(l[a]);
        float z = 0.f;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) z = __builtin_fmaf(o[a][d][e], 0.f, z);
        if (lim[a] < 0)
          l[a] = -1.f;
        else
          off = off || !(l[a] <= E::kHigh) || z != 0.f;
      }
#pragma unroll
      for (int a = 0; a < NQ; ++a)
        store_rows<E, D>(args, rec, hk, wave * 32 * NQ + a * 32 + col, part, o[a], m[a], l[a]);
      if (!head && (!whole || args.records)) {
        left = true;
        const int parts = whole ? 0 : (int)div_units(start + cost + tiles - 1, share) - me + 1;
        if (tid == 0)
          records[args.records ? hk * num_tiles + ti : me] = Unfinished{parts, me, rec.row0, rec.tok0, rec.n, hk, {}};
      }
    }
    if (start + cost + tiles >= end) break;
    if (++ti == num_tiles) {
      ti = 0;
      ++hk;
    }
  }
  if (!left && !p.records && tid == 0) records[me].parts = 0;

  // The share again, with care, where its references did not hold: scores that outgrew them by more
  // than the weights can hold, or values that are not finite.  Here the reference follows the
  // maximum, and a value that is not finite enters only the rows that see it, as itself: its places
  // are taken out of the product with V and counted by products of zeros and ones.  Five times slower.
  if (!__syncthreads_or(off)) return;
  char *sk = smem, *sv = smem + 32 * D * 2;
  hk = uniform((int)div_units(first, per_head));
  ti = uniform(find_tile(tile_before, num_tiles, cost, first - hk * per_head));
#pragma unroll 1
  for (;;) {
    const TileRec rec = tile_recs[ti];
    const int64_t start = hk * per_head + uniform64(tile_before[ti]) + (int64_t)ti * cost;
    const int tiles = uniform((int)(tile_before[ti + 1] - tile_before[ti]));
    const int done = (int)max((int64_t)0, first - start - cost);
    const int todo = (int)min((int64_t)tiles, end - start - cost) - done;
    if (todo > 0) {
      const int tok0 = rec.tok0, n = rec.n, first_page = rec.first_page, len = rec.len, past = len - n;
      const int key_a = rec.key_begin + done * C::kKeys;
      const int key_b = min(rec.key_end, key_a + todo * C::kKeys);
      const int64_t part = done == 0 && todo == tiles ? -1 : 2 * (int64_t)me + (done > 0 ? 0 : 1);
#pragma unroll 1
      for (int rows = 0; rows < C::kRows; rows += 32 * kWaves) {
        const int row = rec.row0 + rows + wave * 32 + col;
        const int tok = (int)div_by(row, p.group), g = row - tok * G;
        const bool real = tok < n;
        const int lim = real ? (p.causal ? min(past + tok, len - 1) : len - 1) : -1;
        const int low = real && p.window > 0 ? max(0, past + tok - p.window + 1) : 0;
        const int64_t h = (int64_t)hk * G + (real ? g : 0);
        u32x4 q[kSteps];
#pragma unroll
        for (int t = 0; t < kSteps; ++t)
          q[t] = *(const u32x4*)((const u16*)p.q.p + (int64_t)(tok0 + (real ? tok : 0)) * p.q.ts + h * p.q.hs + 8 * half + 16 * t);
        f32x16 o[kBlocks];
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
        float m = kNoScore, l = 0.f;
#pragma unroll 1
        for (int key0 = key_a; key0 < key_b; key0 += 32) {
          __syncthreads();
          for (int x = tid; x < 32 * D / 8; x += 64 * kWaves) {
            const int r = x / (D / 8), c = x % (D / 8), key = key0 + r;
            u32x4 wk{0u, 0u, 0u, 0u}, wv = wk;
            const bool apart = SINKS && rec.gap != kNoGap, window = apart && key >= end_of_firsts(p, C::kKeys);
            if (key < key_b && (!apart || window || key < p.sinks)) {
              const int token = window ? key + rec.gap : key;
              const int pg = (int)div_by(token, p.kv.page), off = token - pg * (int)p.kv.page.d;
              const int64_t id = p.kv.idx[first_page + pg], at = id * p.kv.ps + (int64_t)off * p.kv.ts + hk * p.kv.hs + 8 * c;
              if constexpr (Q8) {
                const int64_t sc = id * p.scales.ps + (int64_t)div_by(off, p.scales.block) * p.scales.bs + hk * p.scales.hs;
                wk = values8<E>(*(const u32x2*)(p.kv.k + at), p.scales.k[sc], p.scales.k[sc]);
                wv = values8<E>(*(const u32x2*)(p.kv.v + at), p.scales.v[sc], p.scales.v[sc]);
              } else {
                wk = *(const u32x4*)((const u16*)p.kv.k + at);
                wv = *(const u32x4*)((const u16*)p.kv.v + at);
              }
            }
            *(u32x4*)(sk + k_at<D>(r, c)) = wk;
            *(u32x4*)(sv + v_at<D>(r, c)) = wv;
          }
          __syncthreads();
          f32x16 s;
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
          for (int t = 0; t < kSteps; ++t) s = E::mfma(*(const u32x4*)(sk + k_at<D>(col, 2 * t + half)), q[t], s);
          // value e is of key 4 half + 8 (e / 4) + e % 4
          auto seen = [&](int e) __attribute__((always_inline)) {
            const int key = key0 + 4 * half + 8 * (e >> 2) + (e & 3);
            if constexpr (!SINKS) return (key <= min(lim, key_b - 1)) & (key >= low);
            // before the window's tiles the sinks, or every key where those reach each row's window
            const bool apart = rec.gap != kNoGap, window = apart && key >= end_of_firsts(p, C::kKeys);
            const int token = window ? key + rec.gap : key;
            return (key < key_b) & (token <= lim) & (window ? token >= max(low, p.sinks) : !apart || token < p.sinks);
          };
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            s[e] = seen(e) ? score<CAP>(p, s[e]) : -INFINITY;
            top = fmaxf(top, s[e]);
          }
          const float to = fmaxf(m, fmaxf(top, other_half(top)) - E::kBias), f = __builtin_amdgcn_exp2f(m - to);
          m = to;
          l *= f;
#pragma unroll
          for (int d = 0; d < kBlocks; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = rescaled(o[d][e], f);
          u32x4 pt[2];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float a = __builtin_amdgcn_exp2f(s[e] - m), b = __builtin_amdgcn_exp2f(s[e + 1] - m);
            l += a + b;
            pt[e >> 3][(e >> 1) & 3] = E::pack(a, b);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int d = 0; d < kBlocks; ++d) {
              // keys 16 t + 4 half + 0..3, and 8 more
              const int key = 16 * t + 4 * half + ((lane & 15) >> 2);
              const int dim = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3), sub = (dim & 7) * 2;
              const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(key, dim >> 3) + sub));
              const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(key + 8, dim >> 3) + sub));
              const u32x2 wl = __builtin_bit_cast(u32x2, lo), wh = __builtin_bit_cast(u32x2, hi);
              u32x4 vf{wl[0], wl[1], wh[0], wh[1]};
              if (__any(has_odd<E>(vf))) {
                u32x4 ones, plus, minus;
                take_odd<E>(vf, plus, minus);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  ones[x] = (seen(8 * t + 2 * x) ? E::kOne : 0u) | (seen(8 * t + 2 * x + 1) ? E::kOne << 16 : 0u);
                f32x16 np, nm;
#pragma unroll
                for (int e = 0; e < 16; ++e) np[e] = nm[e] = 0.f;
                np = E::mfma(plus, ones, np);
                nm = E::mfma(minus, ones, nm);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  o[d][e] += np[e] > 0.f ? INFINITY : 0.f;
                  o[d][e] += nm[e] > 0.f ? -INFINITY : 0.f;
                }
              }
              o[d] = E::mfma(vf, pt[t], o[d]);
            }
        }
        store_rows<E, D>(p, rec, hk, rows + wave * 32 + col, part, o, m, lim < 0 ? -1.f : l + other_half(l));
      }
    }
    if (start + cost + tiles >= end) break;
    if (++ti == num_tiles) {
      ti = 0;
      ++hk;
    }
  }
}

// Joins the parts of the tiles that cross shares: workgroup (r, y) takes kGroups
// rows of the tile of record r; its parts are slot 1 of the share that starts it
// and slot 0 of the shares after that.
template <class E, int D>
__global__ __launch_bounds__(256) void chunk_join_kernel(AttnParams p) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  const int d = 4 * (threadIdx.x % kLanes), in_tile = blockIdx.y * kGroups + threadIdx.x / kLanes;
  const Unfinished u = ((const Unfinished*)p.parts)[blockIdx.x];
  const int w = u.share, row = u.row0 + in_tile, tok = (int)div_by(row, p.group), g = row - tok * (int)p.group.d;
  if (u.parts == 0 || tok >= u.n) return;
  float top = kNoScore, sum = 0.f;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  bool none = false;
  // four parts at a time, on the way together
  for (int i0 = 0; i0 < u.parts; i0 += 4) {
    float2 ml[4];
    f32x4 o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = min(i0 + x, u.parts - 1);
      const int64_t at = (int64_t)(i == 0 ? 2 * w + 1 : 2 * (w + i)) * p.part_rows + in_tile;
      ml[x] = *(const float2*)(p.part_ml + at * 2);
      o[x] = *(const f32x4*)(p.part_o + at * D + d);
      if (i0 + x >= u.parts) ml[x].y = 0.f;
    }
    none = ml[0].y < 0.f;  // (so in every part)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (!(ml[x].y <= 0.f)) {  // (a part without weights counts for nothing, whatever its reference)
        const float to = fmaxf(top, ml[x].x), f = __builtin_amdgcn_exp2f(top - to), h = __builtin_amdgcn_exp2f(ml[x].x - to);
        top = to;
        sum = sum * f + ml[x].y * h;
        acc = rescaled(acc, f) + rescaled(o[x], h);
      }
  }
  acc *= none ? 0.f : 1.f / sum;
  const int64_t h = (int64_t)u.hk * p.group.d + g;
  *(u32x2*)((u16*)p.o.p + (int64_t)(u.tok0 + tok) * p.o.ts + h * p.o.hs + d) =
      u32x2{E::pack(acc[0], acc[1]), E::pack(acc[2], acc[3])};
  if (p.lse && d == 0)
    p.lse[(int64_t)(u.tok0 + tok) * p.Hq + h] = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

// Workspace of a chunk call: the plan, and two parts a share.
struct ChunkWs {
  int64_t tiles, part_rows;
  size_t recs, before, seqs, count, parts, ml, o, total;
};
template <int D>
ChunkWs chunk_ws(int64_t T, int64_t B, int64_t G) {
  constexpr bool Q8 = false;  // (the same either way)
  ChunkWs w;
  const int64_t shares = device_cus();
  w.tiles = T * G / Chunk<D, Q8>::kRows + B;  // sum over the sequences of ceil(n G / kRows)
  w.part_rows = std::min<int64_t>(Chunk<D, Q8>::kRows, T * G);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align16(bytes);
    return x;
  };
  w.recs = take((w.tiles + 1) * sizeof(TileRec));
  w.before = take((w.tiles + 1) * sizeof(int64_t));
  w.seqs = take(B * sizeof(SeqRec));
  w.count = take(sizeof(PlanHead));
  w.parts = take(shares * sizeof(Unfinished));
  w.ml = take(2 * shares * w.part_rows * 2 * sizeof(float));
  w.o = take(2 * shares * w.part_rows * D * sizeof(float));
  w.total = at;
  return w;
}

template <class Kernel>
hipError_t allow_lds(Kernel* k, int bytes, std::atomic<bool> (&raised)[kMaxDevices]) {
  const int dev = current_device();
  if (dev >= 0 && dev < kMaxDevices && raised[dev].load(std::memory_order_acquire)) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && dev >= 0 && dev < kMaxDevices) raised[dev].store(true, std::memory_order_release);
  return e;
}

template <class E, int D, Cap CAP, bool EVEN, bool Q8, bool SINKS>
hipError_t launch_chunk_kernel(const AttnParams& p, hipStream_t s) {
  static std::atomic<bool> raised[kMaxDevices];
  hipError_t e = allow_lds(chunk_kernel<E, D, CAP, EVEN, Q8, SINKS>, Chunk<D, Q8>::kLds, raised);
  if (e != hipSuccess) return e;
  const int shares = device_cus();
  if (p.head) {
    plan_kernel<<<dim3(1), dim3(1024), 0, s>>>(p, Chunk<D, Q8>::kRows, Chunk<D, Q8>::kKeys, shares);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  chunk_kernel<E, D, CAP, EVEN, Q8, SINKS><<<dim3(shares), dim3(64 * kWaves), Chunk<D, Q8>::kLds, s>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int groups = 256 / (D / 4);
  chunk_join_kernel<E, D><<<dim3(p.records ? p.records : shares, (p.part_rows + groups - 1) / groups), dim3(256), 0,
                            s>>>(p);
  return hipGetLastError();
}

template <class E, int D, bool Q8, bool SINKS>
hipError_t launch_chunk(AttnParams p, void* workspace, hipStream_t s) {
  const ChunkWs w = chunk_ws<D>(p.T, p.kv.B, p.group.d);
  char* base = (char*)workspace;
  p.tiles = base + w.recs;
  p.before = (int64_t*)(base + w.before);
  p.seqs = base + w.seqs;
  p.head = w.tiles > Chunk<D, Q8>::kFewTiles ? base + w.count : nullptr;
  p.parts = (int*)(base + w.parts);
  p.part_ml = (float*)(base + w.ml);
  p.part_o = (float*)(base + w.o);
  p.part_rows = (int)w.part_rows;
  // Few tiles: a record each, and joins launched for those alone (17 tokens over 1,000: 8 of them instead
  // of 256 shares' take the join from 6.4 to 4.0 us).
  p.records = w.tiles * p.Hkv <= device_cus() ? (int)w.tiles * p.Hkv : 0;
  // A wave's rows of a tile start at a multiple of 16 (or 8) keys: pages of a multiple of 16 tokens hold
  // them whole, and a load goes by one place and 32-bit offsets; otherwise every row's place is staged
  // (1,024 tokens over 8,192, pages of 64 and of 100: 147 and 153 us at D 128; with its
  // tiles checked like the last ones, 232).
  const bool even = p.kv.page.d % 16 == 0 && p.kv.ts * p.kv.page.d < (int64_t(1) << 30);
  if constexpr (Q8) {
    // (blocks of a multiple of 16 tokens divide the pages)
    if (p.cap > kMostShort / kLn2) return launch_chunk_kernel<E, D, kCap, true, true, SINKS>(p, s);
    if (p.cap > 0.f) return launch_chunk_kernel<E, D, kCapShort, true, true, SINKS>(p, s);
    return launch_chunk_kernel<E, D, kNoCap, true, true, SINKS>(p, s);
  } else {
    if (p.cap > kMostShort / kLn2)
      return even ? launch_chunk_kernel<E, D, kCap, true, false, SINKS>(p, s) : launch_chunk_kernel<E, D, kCap, false, false, SINKS>(p, s);
    if (p.cap > 0.f)
      return even ? launch_chunk_kernel<E, D, kCapShort, true, false, SINKS>(p, s)
                  : launch_chunk_kernel<E, D, kCapShort, false, false, SINKS>(p, s);
    return even ? launch_chunk_kernel<E, D, kNoCap, true, false, SINKS>(p, s) : launch_chunk_kernel<E, D, kNoCap, false, false, SINKS>(p, s);
  }
}

// ------------------------------------------------------------------ decode
//
// One token per sequence: the G query rows of a kv-head against every key the
// sequence holds.  Bound by reading the cache once, so the work is cut by bytes:
// every (sequence, kv-head) is a run of 32-key tiles, the runs of the batch laid
// end to end are cut into equal shares, one a wave, and a run that crosses shares
// is joined afterwards from its parts' (m, l, o).
//
// A run whose outputs are not finite is computed again with care: a value that is
// not finite then enters as itself, however small its weight (its place is taken out
// of the product with V and counted by products of ones).
//
// No wave waits for another: it loads its keys and values straight into its own
// ring in LDS, and reads them once they have landed while the next are on the way.
// Products on 16x16x32 MFMAs in the same transposed form as above; P enters as the
// sum of two 16-bit parts (the matrix units idle anyway), so what it adds to the
// output's own rounding is invisible.
//
// Bound by memory: 512 sequences of up to 4,096 tokens (3.09 GB) 514 us, 6.0 TB/s, at
// D 64 270 us, 5.7 TB/s, at D 256 on 4 heads 523 us, 5.9 TB/s; 4 of 131,072 tokens
// 355 us, 6.0 TB/s (a copy reaches 5.7 to 6.0).  Where runs are short their start
// (page table, page ids, first keys) shows: 512 sequences of up to 150 tokens on 8
// heads 38 us, against 62 when four waves shared each run and waited for each other;
// long runs lose 1% to the parts they write.  Codes of a cache of 8 bits become values,
// times their scales, in the registers that feed a product (the values' out of a
// transposed read of 8-bit elements): 512 sequences of up to 4,096 tokens (1.55 GB) 291
// to 298 us, 5.2 to 5.3 TB/s, 4 of 131,072 tokens 187 us, 5.7 TB/s.  With first tokens
// beside a window of 2,048, 256 sequences of up to 16,384 tokens (1.38 GB) 257 to 260 us,
// 5.3 TB/s (the window alone 255).  A run holds 16 query rows: more q-heads
// on a kv-head read its keys and values again for every 16 (64 sequences of up to
// 8,192 tokens, 16 and 32 q-heads on one: 62 and 106 us).

constexpr int kDecTile = 32;   // keys of a tile
constexpr int kDecRows = 16;   // query rows of a run
template <bool Q8>
constexpr int kDecPages = Q8 ? 256 : 512;  // page ids a wave stages at a time
template <int D>
constexpr int kDecStages = D == 64 ? 2 : 1;  // tiles of keys (and of values) in a wave's ring
// Workgroups a compute unit holds.  A tile of codes takes as many instructions as one of 16-bit values and half the
// time on the way, so more waves carry them, with one tile each in place of two (4 of 131,072 tokens 212 -> 187 us,
// 512 of up to 300 50 -> 44 us, at D 256 299 -> 291 us; 512 of up to 4,096 alike; with 4 the registers do not suffice).
template <int D, bool Q8>
constexpr int kDecPerCu = Q8 ? (D == 256 ? 2 : 3) : D == 256 ? 1 : 2;
template <int D, bool Q8>
constexpr int kDecLds = kWaves * kDecStages<D> * 2 * kDecTile * D * (Q8 ? 1 : 2);
// Which 16-byte piece of row r of a tile lies in its place c: the turns are their own inverses.  Rows of codes are
// read 16 keys' piece at a time, and transposed 8 keys' of two groups (keys 4 g .. and 16 + 4 g ..), which the turns
// spread over the banks.
template <int D, bool Q8, bool V>
__device__ __forceinline__ int dec_turn(int r) {
  if constexpr (!Q8) return V ? (D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2) : (D == 64 ? (r >> 1) & 7 : r & 15);
  constexpr int kIn = 256 / D;  // rows of 256 bytes: 4, 2 or 1
  if constexpr (!V) return (r / kIn) & (D / 16 - 1);
  return ((r & 7) / kIn) | ((r >> 4) & 1) << (D == 64 ? 1 : D == 128 ? 2 : 3);
}

template <class E>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma16<Bf>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16<Hf>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                0);
}

// Two weights as hi + lo in the element type, hi cut off, not rounded.
template <class E>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo);
template <>
__device__ __forceinline__ void split2<Bf>(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t x = __float_as_uint(a) & 0xffff0000u, y = __float_as_uint(b) & 0xffff0000u;
  hi = (x >> 16) | y;
  lo = f2bf2(a - __uint_as_float(x), b - __uint_as_float(y));
}
template <>
__device__ __forceinline__ void split2<Hf>(float a, float b, uint32_t& hi, uint32_t& lo) {
  const f16x2 h = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a, b));
  hi = __builtin_bit_cast(uint32_t, h);
  lo = Hf::pack(a - (float)h[0], b - (float)h[1]);
}

// Tokens sequence b holds, and which its (only) query sees: those from begin on, and the first `firsts` (those of
// the sinks that lie before begin).
struct Span {
  int first_page, len, begin, firsts;
};
__device__ __forceinline__ Span dec_span(const AttnParams& p, int b) {
  const int f = p.kv.ptr[b], e = p.kv.ptr[b + 1], last = p.kv.lpl[b];
  const int len = e > f ? (e - f - 1) * (int)p.kv.page.d + last : 0;
  const int begin = p.window > 0 ? max(0, len - p.window) : 0;
  return Span{f, len, begin, min(p.sinks, begin)};
}
// its tiles: of the first tokens, then those from the one that holds `begin` on
__device__ __forceinline__ int dec_first_tiles(const Span& s) { return (s.firsts + kDecTile - 1) / kDecTile; }
__device__ __forceinline__ int dec_tiles(const Span& s) {
  return s.len <= s.begin ? 0 : dec_first_tiles(s) + (s.len + kDecTile - 1) / kDecTile - s.begin / kDecTile;
}
template <class E, int D, Cap CAP, bool Q8>
__global__ __launch_bounds__(64 * kWaves, (kDecPerCu<D, Q8>)) void decode_kernel(AttnParams p) {
  constexpr int NS = kDecStages<D>;
  constexpr int kBytes = Q8 ? 1 : 2;          // of a value in the cache
  constexpr int kRow = kBytes * D, kPieces = kRow / 16;
  constexpr int kSlot = kDecTile * kRow;      // bytes of a tile's keys
  constexpr int kLoads = kSlot / 1024;        // load instructions for them
  constexpr int kScales = Q8 ? 1 : 0;         // and for the scales of a tile, with its keys
  constexpr int kRowsPerLoad = 1024 / kRow;
  constexpr int kSteps = D / 32, kBlocks = D / 16;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int staged_ids[kWaves][kDecPages<Q8>];
  __shared__ __attribute__((aligned(16))) float staged_scales[Q8 ? kWaves * NS * 64 : 1];
  __shared__ int s_where[kWaves][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), grp = lane >> 4, col = lane & 15;
  const int G = (int)p.group.d, vh = (G + kDecRows - 1) / kDecRows;  // row blocks of a kv-head
  const int heads = p.Hkv * vh, B = p.kv.B;

  // this wave's share: units first .. end of the runs laid end to end
  int* page_ids = staged_ids[wave];
  const int me = blockIdx.x * kWaves + wave, shares = gridDim.x * kWaves;
  const int per = (B + 64 * kWaves - 1) / (64 * kWaves);
  const int b0 = tid * per, b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Span sp = dec_span(p, b);
    mine += dec_tiles(sp);
    if (sp.len <= 0 && b % gridDim.x == blockIdx.x) {  // a sequence without a token: zeros
      for (int h = 0; p.records && h < heads; ++h) p.parts[4 * (b * heads + h) + 2] = 0;
      for (int x = 0; x < p.Hq * (D / 8); ++x)
        *(u32x4*)((u16*)p.o.p + (int64_t)b * p.o.ts + (int64_t)(x / (D / 8)) * p.o.hs + 8 * (x % (D / 8))) =
            u32x4{0u, 0u, 0u, 0u};
      if (p.lse)
        for (int h = 0; h < p.Hq; ++h) p.lse[(int64_t)b * p.Hq + h] = -INFINITY;
    }
  }
  int total;
  const int before = block_exclusive_scan(mine, &total);
  const int64_t units = (int64_t)total * heads;
  const int64_t share = div_units(units + shares - 1, shares);
  // records {item, its first share, parts} of unfinished runs (parts 0: none): one an item, a sequence's
  // row block, where the batch has few, one a share otherwise
  if (blockIdx.x * kWaves * share < units)
    for (int w = 0; w < kWaves; ++w) {
      const int64_t first = (blockIdx.x * kWaves + w) * share;
      if (first >= (int64_t)before * heads && first < (int64_t)(before + mine) * heads) {
        int64_t at = (int64_t)before * heads;
        int b = b0, n = mine;
        if (per > 1)
          for (;; ++b) {
            n = dec_tiles(dec_span(p, b));
            if (first < at + (int64_t)n * heads) break;
            at += (int64_t)n * heads;
          }
        const int h = (int)div_units(first - at, n);
        s_where[w][0] = b;
        s_where[w][1] = h;
        s_where[w][2] = (int)(first - at - (int64_t)h * n);
      }
    }
  __syncthreads();
  const int64_t first = me * share, end = min(units, first + share);
  if (first >= end) {
    if (!p.records && lane == 0) p.parts[4 * me + 2] = 0;
    return;
  }
  int b = uniform(s_where[wave][0]), h = uniform(s_where[wave][1]), t = uniform(s_where[wave][2]);
  bool left = false;  // an unfinished run
  // the spans of 64 sequences from `base` on, one a lane
  int base = b;
  Span spans = dec_span(p, min(b + lane, B - 1));

  int staged_b = -1, staged_page = 0, staged_last = 0;  // the page ids at hand
  char* ring = smem + wave * (2 * NS * kSlot);
  bool care = false;  // this run is computed again
  for (int64_t u = first; u < end;) {
    if (b - base >= 64) {
      base = b;
      spans = dec_span(p, min(b + lane, B - 1));
    }
    const Span sp{uniform(__shfl(spans.first_page, b - base, 64)), uniform(__shfl(spans.len, b - base, 64)),
                  uniform(__shfl(spans.begin, b - base, 64)), uniform(__shfl(spans.firsts, b - base, 64))};
    const int tiles = dec_tiles(sp);
    if (tiles == 0) {
      ++b;
      continue;
    }
    const int todo = (int)min((int64_t)(tiles - t), end - u);  // tiles of this run taken here
    const int hk = h / vh, row0 = (h - hk * vh) * kDecRows, rows = min(kDecRows, G - row0);

    u32x4 q[kSteps];
    {
      const u16* src = (const u16*)p.q.p + (int64_t)b * p.q.ts + (int64_t)(hk * G + row0 + min(col, rows - 1)) * p.q.hs;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        // (a lane's 16 codes of a row are its part of two steps)
        q[s] = *(const u32x4*)(src + (Q8 ? 64 * (s >> 1) + 16 * grp + 8 * (s & 1) : 32 * s + 8 * grp));
    }
    static_assert(4 * kBlocks <= 64);
    f32x4 o[kBlocks];
    uint64_t above = 0, below = 0;  // with care: outputs 4 d + e that an infinity, or a NaN (both), belongs to
    float m = kNoScore, l = 0.f;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

    const char* kbase = p.kv.k + kBytes * (int64_t)hk * p.kv.hs;
    const char* vbase = p.kv.v + kBytes * (int64_t)hk * p.kv.hs;

    // the keys of this part: of the first tokens, then of those from `begin` on
#pragma unroll 1
    for (int part = sp.firsts ? 0 : 1; part < 2; ++part) {
    const int firsts = dec_first_tiles(sp);
    const int tile_a = part ? max(t, firsts) - firsts + sp.begin / kDecTile : t;
    const int tile_b = part ? t + todo - firsts + sp.begin / kDecTile : min(t + todo, firsts);
    const int key_b = min(part ? sp.len : sp.firsts, tile_b * kDecTile);

    // as many tiles at a time as the staged page ids reach
    for (int a0 = part ? max(tile_a * kDecTile, sp.begin) : tile_a * kDecTile; a0 < key_b;) {
      const int page0 = (int)div_by(a0, p.kv.page);
      const int64_t reach = (int64_t)(page0 + kDecPages<Q8>) * p.kv.page.d;  // first key past the staged pages
      // (whole tiles; kDecPages pages are more than a tile's keys)
      const int a1 = reach >= key_b ? key_b : (int)reach / kDecTile * kDecTile;
      const int last = (int)div_by(a1 - 1, p.kv.page);
      // (the heads of a sequence go by the same pages: 512 mixed sequences 517 -> 512 us)
      if (b != staged_b || page0 != staged_page || last > staged_last) {
        for (int i = lane; i <= last - page0; i += 64) page_ids[i] = p.kv.idx[sp.first_page + page0 + i];
        wait_lds();
        staged_b = b;
        staged_page = page0;
        staged_last = last;
      }
      const int start = a0 / kDecTile * kDecTile;
      const int n = (a1 - start + kDecTile - 1) / kDecTile;

      // Where the rows lie that this lane loads of a tile, in bytes from the start of the kv-head (-1:
      // not a key of this part, zeros): each lane of a half finds one row's place, and the others take
      // it from there.
      int64_t at[kLoads];
      auto place = [&](int i) __attribute__((always_inline)) {
        const int key = start + i * kDecTile + (lane & 31);
        int64_t mine = -1;
        if (key >= a0 && key < a1) {
          const int pg = (int)div_by(key, p.kv.page);
          mine = kBytes * ((int64_t)page_ids[pg - page0] * p.kv.ps + (int64_t)(key - pg * (int)p.kv.page.d) * p.kv.ts);
        }
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          const int r = x * kRowsPerLoad + lane / kPieces;
          const uint32_t lo = __shfl((int)(uint32_t)mine, r, 64), hi = __shfl((int)(mine >> 32), r, 64);
          at[x] = (int64_t)(((uint64_t)hi << 32) | lo);
        }
      };
      // the scales of a tile, of its first and last 16 keys (which share a block each): lanes 0 and 1 the keys', 2
      // and 3 the values'
      auto load_scales = [&](int i) __attribute__((always_inline)) {
        const int key = start + i * kDecTile + 16 * (lane & 1);
        const char* src = (const char*)&g_one;
        if (key + 15 >= a0 && key < a1) {
          const int pg = (int)div_by(key, p.kv.page), off = key - pg * (int)p.kv.page.d;
          src = (const char*)((lane & 2 ? p.scales.v : p.scales.k) + (int64_t)page_ids[pg - page0] * p.scales.ps +
                              (int64_t)div_by(off, p.scales.block) * p.scales.bs + hk * p.scales.hs);
        }
        dma4(lds_of(staged_scales + (wave * NS + i % NS) * 64), src);
      };
      // values (V) or keys of the placed tile into the slot of tile i
      auto load = [&](int i, bool V) __attribute__((always_inline)) {
        const uint32_t dst = lds_of(ring + (V ? NS * kSlot : 0) + (i % NS) * kSlot);
        if (Q8 && !V) load_scales(i);
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          const int r = x * kRowsPerLoad + lane / kPieces, slot = lane % kPieces;
          // the piece that belongs at this lane's place
          const int c = slot ^ (V ? dec_turn<D, Q8, true>(r) : dec_turn<D, Q8, false>(r));
          const char* src = (V ? vbase : kbase) + at[x] + 16 * c;
          dma16<true>(dst + x * 1024, at[x] < 0 ? (const char*)&g_zero : src);
        }
      };
      // V^T of 16 values: keys 4 grp + 0..3 and 16 more, in the order S leaves them
      auto read_v = [&](const char* sv, int d, f32x4 sc) __attribute__((always_inline)) {
        if constexpr (Q8) {
          // lane i of a 16-lane group points at 8 codes of the key i / 2 and receives code i of all 8 keys
          const int r = 4 * grp + (col >> 1 & 3) + 16 * (col >> 3);
          const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2)(sv + r * kRow + ((d ^ dec_turn<D, Q8, true>(r)) << 4) + 8 * (col & 1)));
          return values8<E>(__builtin_bit_cast(u32x2, w), sc[2], sc[3]);
        }
        const int kr = 4 * grp + (col >> 2), dim = 16 * d + 4 * (lane & 3), sub = (dim & 7) * 2;
        const s16x4 wl = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(kr, dim >> 3) + sub));
        const s16x4 wh = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(kr + 16, dim >> 3) + sub));
        const u32x2 a = __builtin_bit_cast(u32x2, wl), c = __builtin_bit_cast(u32x2, wh);
        return u32x4{a[0], a[1], c[0], c[1]};
      };
      // Takes what is not finite out of a tile of V, and notes the outputs it belongs to (keys outside the
      // part are zeros here).
      auto take_out = [&](char* sv) __attribute__((always_inline)) {
        constexpr uint32_t kOnes = E::kOne | E::kOne << 16;
        const u32x4 ones{kOnes, kOnes, kOnes, kOnes};
        const f32x4 none{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int d = 0; d < kBlocks; ++d) {
          u32x4 vf = read_v(sv, d, f32x4{}), plus, minus;
          take_odd<E>(vf, plus, minus);
          const f32x4 np = mfma16<E>(plus, ones, none), nm = mfma16<E>(minus, ones, none);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            above |= (uint64_t)(np[e] > 0.f) << (4 * d + e);
            below |= (uint64_t)(nm[e] > 0.f) << (4 * d + e);
          }
        }
        wait_lds();
        for (int x = lane; x < kSlot / 16; x += 64) {
          u32x4 w = *(const u32x4*)(sv + 16 * x), plus, minus;
          take_odd<E>(w, plus, minus);
          *(u32x4*)(sv + 16 * x) = w;
        }
        wait_lds();
      };
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        place(i);
        load(i, false);
        load(i, true);
      }
      for (int i = 0; i < n; ++i) {
        const char* sk = ring + (i % NS) * kSlot;
        char* sv = ring + NS * kSlot + (i % NS) * kSlot;
        // outstanding after the keys of tile i: its values and NS - 1 whole tiles
        wait_vm<(2 * NS - 1) * kLoads + (NS - 1) * kScales>();
        f32x4 sc{1.f, 1.f, 1.f, 1.f};
        if constexpr (Q8) sc = *(const f32x4*)(staged_scales + (wave * NS + i % NS) * 64);
        f32x4 s[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          s[kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < kSteps; ++x) {
            if constexpr (Q8) {
              const int r = kb * 16 + col;
              const u32x4 w = *(const u32x4*)(sk + r * kRow + (((4 * (x >> 1) + grp) ^ dec_turn<D, Q8, false>(r)) << 4));
              s[kb] = mfma16<E>(x & 1 ? values8<E>(u32x2{w[2], w[3]}, sc[kb], sc[kb]) : values8<E>(u32x2{w[0], w[1]}, sc[kb], sc[kb]),
                                q[x], s[kb]);
            } else {
              s[kb] = mfma16<E>(*(const u32x4*)(sk + k_at<D>(kb * 16 + col, 4 * x + grp)), q[x], s[kb]);
            }
          }
        }
        wait_lds();
        place(i + NS);
        load(i + NS, false);
        float x[8], top = -INFINITY;
        const int key = start + i * kDecTile + 4 * grp;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = key + 16 * (e >> 2) + (e & 3);
          x[e] = k >= a0 && k < a1 ? score<CAP>(p, s[e >> 2][e & 3]) : -INFINITY;
          top = fmaxf(top, x[e]);
        }
        if (__any(top > m + (E::kBias + E::kSlack))) {
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64)) - E::kBias;
          const float to = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - to);
          m = to;
          l *= f;
#pragma unroll
          for (int d = 0; d < kBlocks; ++d) o[d] *= f;
        }
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = __builtin_amdgcn_exp2f(x[e] - m), c = __builtin_amdgcn_exp2f(x[e + 1] - m);
          l += a + c;
          uint32_t wh, wl;
          split2<E>(a, c, wh, wl);
          hi[e >> 1] = wh;
          lo[e >> 1] = wl;
        }
        // outstanding after the values of tile i: NS - 1 tiles and the keys just asked for
        wait_vm<(2 * NS - 1) * kLoads + NS * kScales>();
        if constexpr (!Q8)
          if (care) take_out(sv);
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) {
          const u32x4 vf = read_v(sv, d, sc);
          o[d] = mfma16<E>(vf, lo, o[d]);
          o[d] = mfma16<E>(vf, hi, o[d]);
        }
        wait_lds();
        load(i + NS, true);
      }
      wait_vm<0>();
      a0 = a1;
    }
    }

    if (care) {
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[d][e] += above >> (4 * d + e) & 1 ? INFINITY : 0.f;
          o[d][e] += below >> (4 * d + e) & 1 ? -INFINITY : 0.f;
        }
    } else {
      float z = 0.f;
#pragma unroll
      for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) z = __builtin_fmaf(o[d][e], 0.f, z);
      // (codes have no infinity, and a NaN among the values makes an output NaN whatever its weight)
      care = !Q8 && __any(z != 0.f);
      if (care) continue;
    }
    care = false;
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const bool whole = t == 0 && todo == tiles;
    const bool head = t > 0;  // a part that continues a run: slot 0, one that starts it: slot 1
    if (col < rows) {
      if (whole) {
        const int64_t hq = (int64_t)hk * G + row0 + col;
        const float inv = 1.f / l;
        u16* dst = (u16*)p.o.p + (int64_t)b * p.o.ts + hq * p.o.hs + 4 * grp;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
          *(u32x2*)(dst + 16 * d) = u32x2{E::pack(o[d][0] * inv, o[d][1] * inv), E::pack(o[d][2] * inv, o[d][3] * inv)};
        if (p.lse && grp == 0) p.lse[(int64_t)b * p.Hq + hq] = (m + __builtin_amdgcn_logf(l)) * kLn2;
      } else {
        const int64_t row = (2 * (int64_t)me + (head ? 0 : 1)) * (Q8 ? p.part_rows : kDecRows) + col;
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) *(f32x4*)(p.part_o + row * D + 16 * d + 4 * grp) = o[d];
        if (grp == 0) *(float2*)(p.part_ml + row * 2) = float2{m, l};
      }
    }
    if (!head && (!whole || p.records)) {
      left = true;
      if (lane == 0) {
        int* rec = p.parts + 4 * (p.records ? b * heads + h : me);
        rec[0] = b * heads + h;
        rec[1] = me;
        rec[2] = whole ? 0 : (int)div_units(u + (tiles - t) - 1, share) - me + 1;
      }
    }
    u += todo;
    t += todo;
    if (t == tiles) {
      t = 0;
      if (++h == heads) {
        h = 0;
        ++b;
      }
    }
  }
  if (!left && !p.records && lane == 0) p.parts[4 * me + 2] = 0;
}

// The join of some parts of a row: their reference, sum and output.
struct Joined {
  float top = kNoScore, sum = 0.f;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float m, float l, f32x4 o) {
    if (l != 0.f) {  // (a part without weights counts for nothing, whatever its reference)
      const float to = fmaxf(top, m), f = __builtin_amdgcn_exp2f(top - to), h = __builtin_amdgcn_exp2f(m - to);
      top = to;
      sum = sum * f + l * h;
      acc = rescaled(acc, f) + rescaled(o, h);
    }
  }
};

// Joins the parts of the runs that cross shares, of the run of record x; they are
// slot 1 of the share that starts it and slot 0 of the shares after that.  Many
// runs have few parts each: a group of D / 4 threads takes a row, a part after the
// other.  FEW runs have up to hundreds: a workgroup takes 32 values of one row and
// reads 128 parts at once (16 runs of about 100: 6.2 us, 15.6 with 32 at once).
// Either way four parts of a thread are on the way together.
template <class E, int D, bool FEW>
__global__ __launch_bounds__(256) void decode_join_kernel(AttnParams p) {
  constexpr int kLanes = FEW ? 8 : D / 4, kGroups = 256 / kLanes, kStep = FEW ? kGroups : 1;
  const int tid = threadIdx.x, g = tid / kLanes, d = 4 * (blockIdx.z * kLanes + tid % kLanes);
  const int r = FEW ? blockIdx.y : blockIdx.y * kGroups + g;
  const int4 rec = ((const int4*)p.parts)[blockIdx.x];
  const int item = rec.x, w = rec.y, parts = rec.z;
  if (parts == 0) return;
  const int G = (int)p.group.d, vh = (G + kDecRows - 1) / kDecRows, heads = p.Hkv * vh;
  const int b = item / heads, h = item - b * heads, hk = h / vh, row0 = (h - hk * vh) * kDecRows;
  if (row0 + r >= G || r >= kDecRows) return;
  Joined a;
  for (int i0 = FEW ? g : 0; i0 < parts; i0 += 4 * kStep) {
    float2 ml[4];
    f32x4 o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = min(i0 + x * kStep, parts - 1);
      const int64_t row = (int64_t)(i == 0 ? 2 * w + 1 : 2 * (w + i)) * p.part_rows + r;
      ml[x] = *(const float2*)(p.part_ml + row * 2);
      o[x] = *(const f32x4*)(p.part_o + row * D + d);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i0 + x * kStep < parts) a.add(ml[x].x, ml[x].y, o[x]);
  }
  if constexpr (FEW) {
    __shared__ f32x4 acc_s[kWaves][kLanes];
    __shared__ float2 ml_s[kWaves][kLanes];
#pragma unroll
    for (int x = kLanes; x < 64; x <<= 1) {
      f32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __shfl_xor(a.acc[e], x, 64);
      a.add(__shfl_xor(a.top, x, 64), __shfl_xor(a.sum, x, 64), o);
    }
    if ((tid & 63) < kLanes) {
      acc_s[tid >> 6][tid & 63] = a.acc;
      ml_s[tid >> 6][tid & 63] = float2{a.top, a.sum};
    }
    __syncthreads();
    if (g) return;
    for (int i = 1; i < kWaves; ++i) a.add(ml_s[i][tid].x, ml_s[i][tid].y, acc_s[i][tid]);
  }
  const f32x4 acc = a.acc * (1.f / a.sum);
  const int64_t hq = (int64_t)hk * G + row0 + r;
  *(u32x2*)((u16*)p.o.p + (int64_t)b * p.o.ts + hq * p.o.hs + d) =
      u32x2{E::pack(acc[0], acc[1]), E::pack(acc[2], acc[3])};
  if (p.lse && d == 0) p.lse[(int64_t)b * p.Hq + hq] = (a.top + __builtin_amdgcn_logf(a.sum)) * kLn2;
}

// Waves of a decode: as many as the compute units hold at once.
template <int D, bool Q8>
int decode_shares() {
  return kWaves * device_cus() * kDecPerCu<D, Q8>;
}

// Rows of a part in the workspace.  Over codes as many as a run has: they have 1.5 to 2 times the waves, and need
// no more than 16-bit calls for groups of up to 7 q-heads (a caller's buffer serves both; 4 q-heads on one of 128
// 12.8 MB, over 16 bits 34.1).
template <bool Q8>
int dec_part_rows(int64_t group) {
  return Q8 ? (int)std::min<int64_t>(kDecRows, group) : kDecRows;
}

template <class E, int D, Cap CAP, bool Q8>
hipError_t launch_decode_cap(const AttnParams& p, hipStream_t s) {
  static std::atomic<bool> raised[kMaxDevices];
  hipError_t e = allow_lds(decode_kernel<E, D, CAP, Q8>, kDecLds<D, Q8>, raised);
  if (e != hipSuccess) return e;
  const int shares = decode_shares<D, Q8>();
  decode_kernel<E, D, CAP, Q8><<<dim3(shares / kWaves), dim3(64 * kWaves), kDecLds<D, Q8>, s>>>(p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int rows = std::min<int>(kDecRows, (int)p.group.d), groups = 1024 / D;
  // (runs of 4 parts and fewer by rows: 64 sequences of up to 2,000 tokens on 8 heads 40 us in all, 44 by
  // values; runs of 8 parts and more by values: 32 of up to 8,000 on 8 heads 48 us, 52 by rows)
  if (p.records && 8 * p.records <= shares)
    decode_join_kernel<E, D, true><<<dim3(p.records, rows, D / 32), dim3(256), 0, s>>>(p);
  else
    decode_join_kernel<E, D, false>
        <<<dim3(p.records ? p.records : shares, (rows + groups - 1) / groups), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

template <class E, int D, bool Q8>
hipError_t launch_dec(AttnParams p, void* workspace, hipStream_t s) {
  const int shares = decode_shares<D, Q8>();
  p.part_rows = dec_part_rows<Q8>(p.group.d);
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + (int64_t)2 * shares * p.part_rows * D;
  p.parts = (int*)(p.part_ml + (int64_t)2 * shares * p.part_rows * 2);
  const int64_t items = (int64_t)p.kv.B * p.Hkv * ((p.group.d + kDecRows - 1) / kDecRows);
  p.records = items <= shares ? (int)items : 0;
  return p.cap > 0.f ? launch_decode_cap<E, D, kCap, Q8>(p, s) : launch_decode_cap<E, D, kNoCap, Q8>(p, s);
}

template <int D, bool Q8>
size_t decode_bytes(int64_t group) {
  return (size_t)decode_shares<D, Q8>() * (2 * dec_part_rows<Q8>(group) * (D + 2) * sizeof(float) + 4 * sizeof(int));
}

// Chunks of one element type, over a cache of the same type or (Q8) of 8 bits; decode of it.
template <class E, bool Q8, bool SINKS>
hipError_t chunk_of_type(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  if (D == 64) return launch_chunk<E, 64, Q8, SINKS>(p, workspace, s);
  if (D == 128) return launch_chunk<E, 128, Q8, SINKS>(p, workspace, s);
  return launch_chunk<E, 256, Q8, SINKS>(p, workspace, s);
}
template <class E, bool Q8>
hipError_t decode_of_type(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  if (D == 64) return launch_dec<E, 64, Q8>(p, workspace, s);
  if (D == 128) return launch_dec<E, 128, Q8>(p, workspace, s);
  return launch_dec<E, 256, Q8>(p, workspace, s);
}

}  // namespace

}  // namespace gdn
