// The append that quantises a paged key/value cache to 8 bits as it writes, and the
// read back.
//
// A block of tokens of a page and head has one scale for its keys and one for its
// values, a power of two:
//   s = 2^ceil(log2(top / 448)),   code = e4m3(x / s),
// top the largest magnitude in the block, 448 the largest e4m3 value.  Scaling by a
// power of two is exact, so a code is one rounding of the (normed, rotated) value; a
// block that holds tokens already keeps its scale or takes the larger new one, and
// then its codes are rounded once more (exact but for those that become subnormal).
//
// A new token that opens a block, or is its sequence's first, leads the block's new
// tokens: its workgroup finds their largest value and writes them.  Blocks of few new
// tokens (decoded ones: one) are a row's lanes'; those of more one, two or all waves',
// which keep the rows in registers (four a lane; beyond 128 rows of 128 values they are
// read twice).  The queries of the workgroup's tokens are rotated beside them, a wave
// a head, four rows a lane on the way together.
//
// Bound by memory and by the waits of a workgroup's start (sequence, page, page id) and of
// each block (rows, largest value, scale): 32 ragged prompts (14,652 tokens, 32 q-heads
// on 8 of 128, 338 MB) 77 us, 4.4 TB/s, of which the queries alone take 45 in rope_kernel.
// Blocks of one wave dealt out one lead after another, two waves idle: 82 us, 492 sequences
// of up to 49 tokens 30 us against 19; every row read twice and half of a workgroup a block: 107.
#include <algorithm>
#include <type_traits>

#include "gdn_rows.h"

namespace gdn {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantTokens = 64;  // most tokens of a workgroup
// Loads and stores of calls that write more than this pass the caches, as in rope_kernel.
constexpr int64_t kQuantCacheBytes = 32 << 20;
constexpr int kShortBlock = 4;    // new tokens that a row's lanes take by themselves
constexpr int kKept = 4;          // rows of a block that a lane keeps in registers

// A token of the workgroup: its position, where its key and value go (-1: nowhere)
// and their scale, and, where it leads a block, the new tokens it leads (0 otherwise)
// and the block's rows before them.
struct Lead {
  int64_t pos, dst, scale;
  int rows, before;
  bool none;  // behind the last sequence
};

__device__ __forceinline__ void find_leads(const RopeParams& p, const ScalesDev& sc, int64_t t0, int tokens, Lead* leads) {
  const int lane = threadIdx.x;
  const int64_t t = t0 + lane;
  int b = (int)t;
  if (p.cu && p.kv.B <= 64) {
    // all ends in one load, a lane each: the sequence is how many are not after t
    const int end = lane < p.kv.B ? p.cu[lane + 1] : INT32_MAX;
    int lo = 0, hi = 64;
#pragma unroll
    for (int x = 0; x < 7; ++x) {
      const int mid = (lo + hi) >> 1;
      const int at = __shfl(end, mid & 63, 64);
      if (lo < hi) {
        if (at <= (int)t)
          lo = mid + 1;
        else
          hi = mid;
      }
    }
    b = min(lo, p.kv.B);
  } else if (p.cu) {
    int lo = wave_find_seq(p.cu, p.kv.B, (int)t0);
    int hi = tokens > 1 ? wave_find_seq(p.cu, p.kv.B, (int)(t0 + tokens - 1)) : lo;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= (int)t)
        lo = mid;
      else
        hi = mid - 1;
    }
    b = lo;
  }
  if (lane < tokens) {
    Lead l{-1, -1, 0, 0, 0, b >= p.kv.B};
    if (b < p.kv.B) {
      const int first = p.kv.ptr[b], pages = p.kv.ptr[b + 1] - first;
      const int64_t len = pages > 0 ? (int64_t)(pages - 1) * p.kv.page.d + p.kv.lpl[b] : 0;
      const int64_t left = p.cu ? p.cu[b + 1] - t : 1;  // new tokens of the sequence from this one on
      l.pos = len - left;
      if (l.pos >= 0) {
        const int pg = (int)div_by((uint32_t)l.pos, p.kv.page), off = (int)(l.pos - (int64_t)pg * p.kv.page.d);
        const int blk = (int)div_by((uint32_t)off, sc.block), in = off - blk * (int)sc.block.d;
        const int64_t id = p.kv.idx[first + pg];
        l.dst = id * p.kv.ps + (int64_t)off * p.kv.ts;
        l.scale = id * sc.ps + (int64_t)blk * sc.bs;
        if (in == 0 || !p.cu || t == p.cu[b]) {
          l.rows = (int)min(min((int64_t)sc.block.d - in, left), p.T - t);  // (no row past the call's)
          l.before = in;
        }
      }
    }
    leads[lane] = l;
  }
}

// The same for the whole wave, in scalar registers.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ Lead uniform_lead(const Lead& l) {
  return Lead{uniform64(l.pos), uniform64(l.dst), uniform64(l.scale), __builtin_amdgcn_readfirstlane(l.rows),
              __builtin_amdgcn_readfirstlane(l.before), l.none};
}

// The scale of a block whose largest magnitude is `top`: 448 is 7/8 of 2^9.  At least
// 2^-100, so that a scale and its inverse are ordinary numbers.
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t w = __float_as_uint(top);
  const int e = (int)(w >> 23) - 126 - 9 + ((w & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}
__device__ __forceinline__ float inverse(float scale) { return __uint_as_float(0x7f000000u - __float_as_uint(scale)); }

// What is stored of a value: NaN for those that are not finite, and no magnitude whose
// code would stand for more than the rows' type holds: 15/8 of its highest power of
// two (240 codes times 2^8 in fp16, 2^120 in bf16).
template <class Tag>
constexpr float kMostStored = Tag::kFp16 ? 0x1.ep15f : 0x1.ep127f;
template <class Tag>
__device__ __forceinline__ float storable(float x) {
  constexpr float most = kMostStored<Tag>;
  return __builtin_isfinite(x) ? fminf(fmaxf(x, -most), most) : __builtin_nanf("");
}
// The larger magnitude, NaN if either is.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(fabsf(a), fabsf(b)); }

// 4 values as codes
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// codes, taken to a larger scale
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return codes4(lo[0] * ratio, lo[1] * ratio, hi[0] * ratio, hi[1] * ratio);
}

template <int W>
__device__ __forceinline__ void store_codes(char* dst, const float (&x)[W], float inv) {
  if constexpr (W == 8)
    *(u32x2*)dst = u32x2{codes4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                         codes4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
  else
    *(u16*)dst = (u16)__builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
}
template <int W>
__device__ __forceinline__ void rescale_codes(char* dst, float ratio) {
  if constexpr (W == 8) {
    const u32x2 w = *(const u32x2*)dst;
    *(u32x2*)dst = u32x2{rescale4(w[0], ratio), rescale4(w[1], ratio)};
  } else {
    *(u16*)dst = (u16)rescale4(*(const u16*)dst, ratio);
  }
}

// Workgroup (x, y): tokens x * tokens_per_block .., kv-heads y * heads_per .., and the
// q-heads' share y.
// FEW: blocks of up to kShortBlock new tokens, and queries, are a row's lanes each; otherwise a wave's.
template <class Tag, bool NEAR, int W, bool NORM, bool NT, bool FEW>
__global__ __launch_bounds__(kQuantThreads, 3) void quant_append_kernel(RopeParams p, NormDev n, ScalesDev sc, int heads_per,
                                                                    int q_per) {
  typedef typename Tag::type E;
  __shared__ Lead leads[kQuantTokens];
  __shared__ int few[kQuantTokens], many[kQuantTokens], counts[3];  // many: first those that one wave takes
  __shared__ float tops[kQuantThreads / 64];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);
  if (threadIdx.x < 64) {
    find_leads(p, sc, t0, tokens, leads);
    const int rows = threadIdx.x < tokens ? leads[threadIdx.x].rows : 0;
    const int shortest = FEW ? kShortBlock : 0;  // (of those a wave takes, less one)
    const int longest = kKept * (64 >> n.shift);  // of one wave
    const uint64_t s = __ballot(rows > 0 && rows <= shortest), m = __ballot(rows > shortest && rows <= longest);
    const uint64_t l = __ballot(rows > shortest && rows > longest), below = (uint64_t(1) << threadIdx.x) - 1;
    if (rows > 0 && rows <= shortest)
      few[__popcll(s & below)] = threadIdx.x;
    else if (rows > 0)
      many[rows <= longest ? __popcll(m & below) : __popcll(m) + __popcll(l & below)] = threadIdx.x;
    if (threadIdx.x == 0) {
      counts[0] = __popcll(s);
      counts[1] = __popcll(m);
      counts[2] = __popcll(m) + __popcll(l);
    }
  }
  const int L = 1 << n.shift, sub = threadIdx.x & (L - 1);
  float wq[1][2][W], wk[1][2][W];
  if constexpr (NORM) {
    load_weights<Tag, NEAR, W, 1>(n, n.wq, p.D, p.rot, wq);
    load_weights<Tag, NEAR, W, 1>(n, n.wk, p.D, p.rot, wk);
  }
  __syncthreads();
  // (a row's lanes are as many as its units: D is a power of two)
  const Columns<NEAR, W> c(sub, p.D, p.rot);
  const int h0 = blockIdx.y * heads_per, hn = min(heads_per, p.Hk - h0);
  const int q0 = blockIdx.y * q_per, qn = max(0, min(q_per, p.Hq - q0));

  auto normed = [&](float (&x)[2][W], const float (&w)[2][W]) __attribute__((always_inline)) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) sum = __builtin_fmaf(x[0][i], x[0][i], __builtin_fmaf(x[1][i], x[1][i], sum));
    const float f = rsqrtf(__builtin_fmaf(row_sum(sum, L), n.inv_dim, n.eps));
#pragma unroll
    for (int i = 0; i < W; ++i) {
      x[0][i] *= f * w[0][i];
      x[1][i] *= f * w[1][i];
    }
  };
  auto row_at = [&](bool V, int h, int64_t t) __attribute__((always_inline)) {
    const RowsDev& r = V ? p.v : p.k;
    return (const E*)r.p + t * r.ts + h * r.hs;
  };
  // a key (or V: value) at position pos, normed and turned
  auto finish = [&](bool V, int64_t pos, float (&x)[2][W]) __attribute__((always_inline)) {
    if (V) return;
    if constexpr (NORM)
      if (n.wk) normed(x, wk[0]);
    if (c.turned) turn_unit<NEAR, W>(p, pos, c.a, c.b, p.sign, x);
  };
  auto fetch = [&](bool V, int h, int64_t t, int64_t pos, float (&x)[2][W]) __attribute__((always_inline)) {
    load_unit<W, false>(row_at(V, h, t), c.a, c.b, x);
    finish(V, pos, x);
  };
  auto top_of = [&](const float (&x)[2][W], float top) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W; ++i) top = larger(larger(x[0][i], x[1][i]), top);
    return top;
  };
  // Values that cannot be stored as they are (the largest is NaN, infinite or too large) are changed, and counted
  // anew: rare, so asked of a block's largest alone.
  auto odd = [&](float top) __attribute__((always_inline)) { return !(top <= kMostStored<Tag>); };
  auto store_able = [&](float (&x)[2][W]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < W; ++i) x[k][i] = storable<Tag>(x[k][i]);
  };
  auto top_of_stored = [&](const float (&x)[2][W], float top) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));  // (NaN counts for nothing)
    return top;
  };
  // A block's scale with the new tokens' largest value; codes that were there are taken to it.
  // (`old` is read as early as may be: it is a wait of its own)
  auto old_scale = [&](bool V, int h, const Lead& l) __attribute__((always_inline)) {
    return l.before ? ((V ? sc.v : sc.k) + l.scale)[h * sc.hs] : 0.f;
  };
  auto settle = [&](bool V, int h, const Lead& l, float old, float top, int row, int step) __attribute__((always_inline)) {
    const float scale = fmaxf(old, scale_for(top));
    if (l.before && scale > old) {
      char* base = (V ? p.kv.v : p.kv.k) + l.dst + h * p.kv.hs;
#pragma unroll 1
      for (int r = row; r < l.before; r += step) {
        char* dst = base + (int64_t)(r - l.before) * p.kv.ts;
        rescale_codes<W>(dst + c.a, old * inverse(scale));
        rescale_codes<W>(dst + c.b, old * inverse(scale));
      }
    }
    return scale;
  };
  auto put_row = [&](bool V, int h, const Lead& l, int r, const float (&x)[2][W], float inv) __attribute__((always_inline)) {
    char* dst = (V ? p.kv.v : p.kv.k) + l.dst + (int64_t)r * p.kv.ts + h * p.kv.hs;
    store_codes<W>(dst + c.a, x[0], inv);
    store_codes<W>(dst + c.b, x[1], inv);
  };

  // queries of many tokens: a wave takes a head's rows, as many as it keeps of a block, at a time
  const int at_once = 64 >> n.shift, lane_row = (threadIdx.x & 63) >> n.shift, kept = kKept * at_once;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q_parts = FEW ? 0 : (tokens + kept - 1) / kept;
#pragma unroll 1
  for (int i = wave; i < qn * q_parts; i += kQuantThreads / 64) {
    const int part = i / qn, h = q0 + i - part * qn;
    float x[kKept][2][W];
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
      const int64_t t = t0 + min(part * kept + j * at_once + lane_row, tokens - 1);  // (rows past the last take it again)
      load_unit<W, NT>((const E*)p.q.p + t * p.q.ts + h * p.q.hs, c.a, c.b, x[j]);
    }
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
      const int tok = part * kept + j * at_once + lane_row;
      if constexpr (NORM)
        if (n.wq) normed(x[j], wq[0]);
      if (tok < tokens && !leads[tok].none) {
        if (c.turned) turn_unit<NEAR, W>(p, leads[tok].pos, c.a, c.b, p.sign, x[j]);
        store_unit<W, NT>((E*)p.q_out.p + (t0 + tok) * p.q_out.ts + h * p.q_out.hs, c.a, c.b, x[j]);
      }
    }
  }

  // queries of few tokens, and blocks of few new tokens: one row of lanes each
  const int q_items = FEW ? tokens * qn : 0, items = FEW ? q_items + counts[0] * 2 * hn : 0;
#pragma unroll 1
  for (int i = threadIdx.x >> n.shift; i < items; i += kQuantThreads >> n.shift) {
    float x[2][W];
    if (i < q_items) {
      const int tok = i / qn, h = q0 + i - tok * qn;
      const int64_t t = t0 + tok;
      if (leads[tok].none) continue;
      load_unit<W, false>((const E*)p.q.p + t * p.q.ts + h * p.q.hs, c.a, c.b, x);
      if constexpr (NORM)
        if (n.wq) normed(x, wq[0]);
      if (c.turned) turn_unit<NEAR, W>(p, leads[tok].pos, c.a, c.b, p.sign, x);
      store_unit<W, false>((E*)p.q_out.p + t * p.q_out.ts + h * p.q_out.hs, c.a, c.b, x);
    } else {
      const int j = i - q_items, tok = few[j / (2 * hn)], k = j % (2 * hn), h = h0 + (k >> 1);
      const bool V = k & 1;
      const Lead l = leads[tok];
      const float old = old_scale(V, h, l);
      float top = 0.f;
#pragma unroll 1
      for (int r = 0; r < l.rows; ++r) {
        fetch(V, h, t0 + tok + r, l.pos + r, x);
        top = top_of(x, top);
      }
      for (int m = 1; m < L; m <<= 1) top = larger(top, __shfl_xor(top, m, 64));
      const bool change = odd(top);
      if (change) {
        top = 0.f;
#pragma unroll 1
        for (int r = 0; r < l.rows; ++r) {
          fetch(V, h, t0 + tok + r, l.pos + r, x);
          store_able(x);
          top = top_of_stored(x, top);
        }
        for (int m = 1; m < L; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
      }
      const float scale = settle(V, h, l, old, top, 0, 1);
      // (the row's lanes are of one wave: they have all read the old scale)
      if (sub == 0) ((V ? sc.v : sc.k) + l.scale)[h * sc.hs] = scale;
      const float inv = inverse(scale);
#pragma unroll 1
      for (int r = 0; r < l.rows; ++r) {
        if (l.rows > 1) {
          fetch(V, h, t0 + tok + r, l.pos + r, x);
          if (change) store_able(x);
        }
        put_row(V, h, l, r, x, inv);
      }
    }
  }

  // Blocks of more: one, two or all waves each, as many as keep its rows in registers (kKept a lane); beyond
  // that all, which read the rows twice (blocks of 256, 512 and 896 rows of 128 values 102, 118 and 151 us, with half of
  // the workgroup on the keys and half on the values 108, 127 and 163; of 256 values 122, 154 and 211, against 133, 175
  // and 250).  Those of one wave are dealt out together; where more than one wave has a part, all wait for each
  // other (every wave goes through the same turns).
  constexpr int kWaves = kQuantThreads / 64;
  const int alone = __builtin_amdgcn_readfirstlane(counts[1]), many_leads = __builtin_amdgcn_readfirstlane(counts[2]);
  int together = alone ? alone : 1;
#pragma unroll 1
  for (int j = 0; j < many_leads; j += together, together = 1) {
    const int rows = __builtin_amdgcn_readfirstlane(leads[many[j]].rows);
    const int team = j < alone ? 1 : rows > 2 * kept ? kWaves : 2;  // waves
    const int step = team * at_once, row = (wave & (team - 1)) * at_once + lane_row, most = kKept * step;
    const int teams = kWaves / team, work = 2 * hn * together, turns = (work + teams - 1) / teams;
#pragma unroll 1
    for (int i = 0; i < turns; ++i) {
      const int item = i * teams + wave / team, at = min(item, work - 1);  // (those past the last only wait)
      const int lead = at / (2 * hn), k2 = at - lead * 2 * hn, h = h0 + (k2 >> 1);
      const bool mine = item < work, V = k2 & 1;
      const int tok = __builtin_amdgcn_readfirstlane(many[j + lead]);
      const Lead l = uniform_lead(leads[tok]);
      const float old = mine ? old_scale(V, h, l) : 0.f;
      float x[kKept][2][W], top = 0.f, inv = 1.f;
      bool change = false;
      // first the largest value, once more where some cannot be stored as they are, then the codes
#pragma unroll 1
      for (int phase = 0; phase < 3; ++phase) {
        asm volatile("" : "+s"(phase));  // (one loop for all three: in copies of it the rows would not fit)
        if (mine) {
#pragma unroll 1
          for (int r0 = 0; r0 < l.rows; r0 += most) {
            if (phase == 0 || l.rows > most) {
#pragma unroll
              for (int k = 0; k < kKept; ++k)  // (rows past the last take it again)
                load_unit<W, NT>(row_at(V, h, t0 + tok + min(r0 + k * step + row, l.rows - 1)), c.a, c.b, x[k]);
#pragma unroll
              for (int k = 0; k < kKept; ++k) finish(V, l.pos + min(r0 + k * step + row, l.rows - 1), x[k]);
            }
            if (change) {
#pragma unroll
              for (int k = 0; k < kKept; ++k) {
                store_able(x[k]);
                top = top_of_stored(x[k], top);
              }
            }
            if (phase == 0) {
#pragma unroll
              for (int k = 0; k < kKept; ++k) top = top_of(x[k], top);
            }
            if (phase == 2) {
#pragma unroll
              for (int k = 0; k < kKept; ++k) {
                const int r = r0 + k * step + row;
                if (r < l.rows) put_row(V, h, l, r, x[k], inv);
              }
            }
          }
        }
        if (phase == 2) break;
        for (int m = 1; m < 64; m <<= 1) top = larger(top, __shfl_xor(top, m, 64));
        if (team > 1) {
          __syncthreads();  // (the last turn's have been read)
          if ((threadIdx.x & 63) == 0) tops[wave] = top;
          __syncthreads();
          const int first = wave & ~(team - 1);
          for (int w = 0; w < team; ++w) top = larger(top, tops[first + w]);
        }
        top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));  // (every lane's)
        if (phase == 0) {
          // (teams of several waves wait together: if one changes its values, all look again)
          change = odd(top);
          if (team > 1) change = __builtin_amdgcn_readfirstlane(__syncthreads_or(change)) != 0;
          if (change) {
            top = 0.f;
            continue;
          }
          phase = 1;
        }
        float scale = 1.f;
        if (mine) scale = settle(V, h, l, old, top, row, step);
        if (team > 1) __syncthreads();  // (everyone has read the old scale)
        if (mine && row == 0 && sub == 0) ((V ? sc.v : sc.k) + l.scale)[h * sc.hs] = scale;
        inv = inverse(scale);
      }
    }
  }
}

// ---------------------------------------------------------------- the read back
//
// A thread takes 8 codes of a key and of the value beside it: 16 bytes read, 32 (or 64)
// written.  Bound by memory: 95,773 tokens of 8 heads (588 MB) 107 us, 5.5 TB/s (keys and
// values in turns of their own 150 us).

constexpr int kReadTokens = 64;

template <class Tag, bool NT>
__device__ __forceinline__ void write_values(typename Tag::type* dst, u32x2 w, float s) {
  float x[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    x[i][0] = lo[0] * s;
    x[i][1] = lo[1] * s;
    x[i][2] = hi[0] * s;
    x[i][3] = hi[1] * s;
  }
  if constexpr (sizeof(typename Tag::type) == 2) {
    store<NT, 8>(dst, *(const float(*)[8])x);
  } else {
    store<NT, 4>(dst, x[0]);
    store<NT, 4>(dst + 4, x[1]);
  }
}

template <class Tag, bool NT>
__global__ __launch_bounds__(kQuantThreads) void quant_read_kernel(RopeParams p, ScalesDev sc) {
  typedef typename Tag::type E;
  __shared__ Lead places[kReadTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);
  if (threadIdx.x < 64) find_leads(p, sc, t0, tokens, places);
  __syncthreads();
  const uint32_t units = p.row_units.d, H = p.heads.d, total = (uint32_t)tokens * H * units;
  constexpr int U = 2;  // on the way together
  for (uint32_t u0 = threadIdx.x; u0 < total; u0 += U * kQuantThreads) {
    u32x2 w[U][2];
    float s[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = min(u0 + i * kQuantThreads, total - 1), row = div_by(u, p.row_units), tok = div_by(row, p.heads);
      const uint32_t at = 8 * (u - row * units), h = row - tok * H;
      const Lead l = places[tok];
      w[i][0] = w[i][1] = u32x2{0u, 0u};
      s[i][0] = s[i][1] = 0.f;
      if (l.dst >= 0) {
        w[i][0] = get<NT>((const u32x2*)(p.kv.k + l.dst + h * p.kv.hs + at));
        w[i][1] = get<NT>((const u32x2*)(p.kv.v + l.dst + h * p.kv.hs + at));
        s[i][0] = sc.k[l.scale + h * sc.hs];
        s[i][1] = sc.v[l.scale + h * sc.hs];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + i * kQuantThreads, row = div_by(u, p.row_units), tok = div_by(row, p.heads);
      const uint32_t at = 8 * (u - row * units), h = row - tok * H;
      if (u >= total || places[tok].none) continue;
      write_values<Tag, NT>((E*)p.k.p + (t0 + tok) * p.k.ts + h * p.k.hs + at, w[i][0], s[i][0]);
      write_values<Tag, NT>((E*)p.v.p + (t0 + tok) * p.v.ts + h * p.v.hs + at, w[i][1], s[i][1]);
    }
  }
}

template <class Tag, bool NEAR, int W>
hipError_t launch_append_width(RopeParams p, NormDev n, const ScalesDev& sc, hipStream_t s) {
  n.units = rope_units(p, W);
  n.shift = 0;
  while ((1 << n.shift) < n.units) ++n.shift;
  n.inv_dim = 1.f / (float)p.D;
  // one token per sequence: as many as keep the workgroup's threads busy; otherwise a workgroup a kv-head, of 64
  // tokens where that fills the chip (prompts of 14,652 tokens in blocks of 32, 64, 128: 77, 79, 78 us; of 32 tokens
  // 79, 86, 86) and no fewer than 4 (21 sequences of up to 11 tokens, 36 q-heads on 3: 12.7 us; with no fewer than 16,
  // which share the search for their sequence, 20.5)
  const int64_t per_token = (int64_t)(p.Hq + 2 * p.Hk) << n.shift;
  const bool decode = !p.cu;
  const int y = decode ? 1 : p.Hk;
  p.tokens_per_block = decode ? (int)std::max<int64_t>(1, std::min<int64_t>(kQuantTokens, kQuantThreads / per_token))
                              : (int)std::max<int64_t>(4, std::min<int64_t>(kQuantTokens, p.T * y / (2 * device_cus())));
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block), y);
  const int heads = decode ? p.Hk : 1, q_heads = (p.Hq + y - 1) / y;
  const bool norm = n.wq || n.wk, nt = W == 8 && p.T * (p.Hq + 2 * p.Hk) * p.D * 2 > kQuantCacheBytes;
  auto launch = [&](auto with_norm, auto past, auto few) {
    quant_append_kernel<Tag, NEAR, W, decltype(with_norm)::value, decltype(past)::value, decltype(few)::value>
        <<<grid, dim3(kQuantThreads), 0, s>>>(p, n, sc, heads, q_heads);
  };
  const std::true_type yes;
  const std::false_type no;
  if (p.T <= kShortBlock * (int64_t)p.kv.B) {
    norm ? launch(yes, no, yes) : launch(no, no, yes);
  } else {
    if constexpr (W == 8) {
      if (nt) norm ? launch(yes, yes, no) : launch(no, yes, no);
    }
    if (!nt) norm ? launch(yes, no, no) : launch(no, no, no);
  }
  return hipGetLastError();
}
template <class Tag>
hipError_t launch_append_type(const RopeParams& p, const NormDev& n, const ScalesDev& sc, bool near_, int width, hipStream_t s) {
  if (width == 8)
    return near_ ? launch_append_width<Tag, true, 8>(p, n, sc, s) : launch_append_width<Tag, false, 8>(p, n, sc, s);
  return near_ ? launch_append_width<Tag, true, 2>(p, n, sc, s) : launch_append_width<Tag, false, 2>(p, n, sc, s);
}

}  // namespace

hipError_t launch_quant_append(const RopeParams& p, const NormDev& n, const ScalesDev& sc, int dtype, bool interleaved, int width,
                               hipStream_t s) {
  return dtype == 0 ? launch_append_type<Bf16>(p, n, sc, interleaved, width, s)
                    : launch_append_type<Half>(p, n, sc, interleaved, width, s);
}

template <class Tag>
static void launch_read_type(const RopeParams& p, const ScalesDev& sc, hipStream_t s) {
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block)), blk(kQuantThreads);
  if (2 * p.T * p.Hk * p.D * (int64_t)sizeof(typename Tag::type) > kQuantCacheBytes)
    quant_read_kernel<Tag, true><<<grid, blk, 0, s>>>(p, sc);
  else
    quant_read_kernel<Tag, false><<<grid, blk, 0, s>>>(p, sc);
}

hipError_t launch_quant_read(RopeParams p, const ScalesDev& sc, int dtype, hipStream_t s) {
  const int units = p.D / 8;
  p.heads = fast_div(p.Hk);
  p.row_units = fast_div(units);
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(kReadTokens, 4 * kQuantThreads / ((int64_t)p.Hk * units)));
  if (dtype == 0)
    launch_read_type<Bf16>(p, sc, s);
  else if (dtype == 1)
    launch_read_type<Half>(p, sc, s);
  else
    launch_read_type<Single>(p, sc, s);
  return hipGetLastError();
}

}  // namespace gdn
