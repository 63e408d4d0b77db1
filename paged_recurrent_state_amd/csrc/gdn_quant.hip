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
// tokens (decoded ones: one) are a row's lanes', both passes in turn; longer ones the
// workgroup's, its first half the keys, its second half the values.  The queries of
// the workgroup's tokens are rotated beside them.  Bound by memory: values are read
// twice, the second time from the cache.
#include <algorithm>

#include "gdn_rows.h"

namespace gdn {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantTokens = 32;  // most tokens of a workgroup
constexpr int kShortBlock = 4;    // new tokens that a row's lanes take by themselves

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
  if (p.cu) {
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
          l.rows = (int)min((int64_t)sc.block.d - in, left);
          l.before = in;
        }
      }
    }
    leads[lane] = l;
  }
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
__device__ __forceinline__ float storable(float x) {
  constexpr float most = Tag::kFp16 ? 0x1.ep15f : 0x1.ep127f;
  return __builtin_isfinite(x) ? fminf(fmaxf(x, -most), most) : __builtin_nanf("");
}

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
template <class Tag, bool NEAR, int W>
__global__ __launch_bounds__(kQuantThreads) void quant_append_kernel(RopeParams p, NormDev n, ScalesDev sc, int heads_per,
                                                                    int q_per) {
  typedef typename Tag::type E;
  __shared__ Lead leads[kQuantTokens];
  __shared__ int few[kQuantTokens], many[kQuantTokens], counts[2];
  __shared__ float tops[kQuantThreads / 64];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);
  if (threadIdx.x < 64) {
    find_leads(p, sc, t0, tokens, leads);
    const int rows = threadIdx.x < tokens ? leads[threadIdx.x].rows : 0;
    const uint64_t s = __ballot(rows > 0 && rows <= kShortBlock), l = __ballot(rows > kShortBlock);
    const uint64_t below = (uint64_t(1) << threadIdx.x) - 1;
    if (rows > 0 && rows <= kShortBlock) few[__popcll(s & below)] = threadIdx.x;
    if (rows > kShortBlock) many[__popcll(l & below)] = threadIdx.x;
    if (threadIdx.x == 0) {
      counts[0] = __popcll(s);
      counts[1] = __popcll(l);
    }
  }
  const int L = 1 << n.shift, sub = threadIdx.x & (L - 1);
  float wq[1][2][W], wk[1][2][W];
  load_weights<Tag, NEAR, W, 1>(n, n.wq, p.D, p.rot, wq);
  load_weights<Tag, NEAR, W, 1>(n, n.wk, p.D, p.rot, wk);
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
  // the key (or V: value) of head h of new token t at position pos, as it is stored, but for the scale
  auto fetch = [&](bool V, int h, int64_t t, int64_t pos, float (&x)[2][W]) __attribute__((always_inline)) {
    const RowsDev& r = V ? p.v : p.k;
    load_unit<W, false>((const E*)r.p + t * r.ts + h * r.hs, c.a, c.b, x);
    if (!V) {
      if (n.wk) normed(x, wk[0]);
      if (c.turned) turn_unit<NEAR, W>(p, pos, c.a, c.b, p.sign, x);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < W; ++i) x[k][i] = storable<Tag>(x[k][i]);
  };
  auto top_of = [&](const float (&x)[2][W], float top) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));  // (NaN counts for nothing)
    return top;
  };
  // A block's scale with the new tokens' largest value; codes that were there are taken to it.
  auto settle = [&](bool V, int h, const Lead& l, float top, int row, int step) __attribute__((always_inline)) {
    float* at = (V ? sc.v : sc.k) + l.scale + h * sc.hs;
    const float old = l.before ? *at : 0.f, scale = fmaxf(old, scale_for(top));
    if (l.before && scale > old) {
      char* base = (V ? p.kv.v : p.kv.k) + l.dst + h * p.kv.hs;
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

  // queries, and blocks of few new tokens: one row of lanes each
  const int q_items = tokens * qn, items = q_items + counts[0] * 2 * hn;
  for (int i = threadIdx.x >> n.shift; i < items; i += kQuantThreads >> n.shift) {
    float x[2][W];
    if (i < q_items) {
      const int tok = i / qn, h = q0 + i - tok * qn;
      const int64_t t = t0 + tok;
      load_unit<W, false>((const E*)p.q.p + t * p.q.ts + h * p.q.hs, c.a, c.b, x);
      if (n.wq) normed(x, wq[0]);
      if (c.turned) turn_unit<NEAR, W>(p, leads[tok].pos, c.a, c.b, p.sign, x);
      store_unit<W, false>((E*)p.q_out.p + t * p.q_out.ts + h * p.q_out.hs, c.a, c.b, x);
    } else {
      const int j = i - q_items, tok = few[j / (2 * hn)], k = j % (2 * hn), h = h0 + (k >> 1);
      const bool V = k & 1;
      const Lead l = leads[tok];
      float top = 0.f;
      for (int r = 0; r < l.rows; ++r) {
        fetch(V, h, t0 + tok + r, l.pos + r, x);
        top = top_of(x, top);
      }
      for (int m = 1; m < L; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
      const float scale = settle(V, h, l, top, 0, 1);
      // (the row's lanes are of one wave: they have all read the old scale)
      if (sub == 0) ((V ? sc.v : sc.k) + l.scale)[h * sc.hs] = scale;
      const float inv = inverse(scale);
      for (int r = 0; r < l.rows; ++r) {
        if (l.rows > 1) fetch(V, h, t0 + tok + r, l.pos + r, x);
        put_row(V, h, l, r, x, inv);
      }
    }
  }

  // blocks of more: half of the workgroup each
  const bool V = threadIdx.x >= kQuantThreads / 2;
  const int row = (threadIdx.x % (kQuantThreads / 2)) >> n.shift, step = (kQuantThreads / 2) >> n.shift;
  for (int j = 0; j < counts[1] * hn; ++j) {
    const int tok = many[j / hn], h = h0 + j % hn;
    const Lead l = leads[tok];
    float x[2][W], top = 0.f;
    for (int r = row; r < l.rows; r += step) {
      fetch(V, h, t0 + tok + r, l.pos + r, x);
      top = top_of(x, top);
    }
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(tops[V ? 2 : 0], tops[V ? 3 : 1]);
    const float scale = settle(V, h, l, top, row, step);
    __syncthreads();  // (everyone has read the old scale, and the largest values)
    if (threadIdx.x % (kQuantThreads / 2) == 0) ((V ? sc.v : sc.k) + l.scale)[h * sc.hs] = scale;
    const float inv = inverse(scale);
    for (int r = row; r < l.rows; r += step) {
      fetch(V, h, t0 + tok + r, l.pos + r, x);
      put_row(V, h, l, r, x, inv);
    }
  }
}

// ---------------------------------------------------------------- the read back
//
// Every thread takes 8 codes of a row: 8 bytes read, 16 (or 32) written.

constexpr int kReadTokens = 64;

template <class Tag>
__global__ __launch_bounds__(kQuantThreads) void quant_read_kernel(RopeParams p, ScalesDev sc) {
  typedef typename Tag::type E;
  __shared__ Lead places[kReadTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);
  if (threadIdx.x < 64) find_leads(p, sc, t0, tokens, places);
  __syncthreads();
  const uint32_t units = p.row_units.d, H = p.heads.d, total = (uint32_t)tokens * H * units;
  for (uint32_t u = threadIdx.x; u < total; u += kQuantThreads) {
    const uint32_t row = div_by(u, p.row_units), at = 8 * (u - row * units), tok = div_by(row, p.heads);
    int h = (int)(row - tok * H);
    const bool V = h >= p.Hk;
    if (V) h -= p.Hk;
    const Lead l = places[tok];
    if (l.none) continue;
    const RowsDev& r = V ? p.v : p.k;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (l.dst >= 0) {
      const u32x2 w = *(const u32x2*)((V ? p.kv.v : p.kv.k) + l.dst + h * p.kv.hs + at);
      const float s = ((V ? sc.v : sc.k) + l.scale)[h * sc.hs];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        x[4 * i] = lo[0] * s;
        x[4 * i + 1] = lo[1] * s;
        x[4 * i + 2] = hi[0] * s;
        x[4 * i + 3] = hi[1] * s;
      }
    }
    E* dst = (E*)r.p + (t0 + tok) * r.ts + h * r.hs + at;
    if constexpr (sizeof(E) == 2) {
      store<false, 8>(dst, x);
    } else {
      store<false, 4>(dst, *(const float(*)[4])x);
      store<false, 4>(dst + 4, *(const float(*)[4])(x + 4));
    }
  }
}

template <class Tag, bool NEAR, int W>
hipError_t launch_append_width(RopeParams p, NormDev n, const ScalesDev& sc, hipStream_t s) {
  n.units = rope_units(p, W);
  n.shift = 0;
  while ((1 << n.shift) < n.units) ++n.shift;
  n.inv_dim = 1.f / (float)p.D;
  // one token per sequence: as many as keep the workgroup's threads busy; otherwise a workgroup a kv-head
  const int64_t per_token = (int64_t)(p.Hq + 2 * p.Hk) << n.shift;
  const bool decode = !p.cu;
  p.tokens_per_block = decode ? (int)std::max<int64_t>(1, std::min<int64_t>(kQuantTokens, kQuantThreads / per_token)) : kQuantTokens;
  const int y = decode ? 1 : p.Hk;
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block), y);
  quant_append_kernel<Tag, NEAR, W><<<grid, dim3(kQuantThreads), 0, s>>>(p, n, sc, decode ? p.Hk : 1, (p.Hq + y - 1) / y);
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

hipError_t launch_quant_read(RopeParams p, const ScalesDev& sc, int dtype, hipStream_t s) {
  const int units = p.D / 8;
  p.heads = fast_div(2 * p.Hk);
  p.row_units = fast_div(units);
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(kReadTokens, 4 * kQuantThreads / ((int64_t)2 * p.Hk * units)));
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block)), blk(kQuantThreads);
  if (dtype == 0)
    quant_read_kernel<Bf16><<<grid, blk, 0, s>>>(p, sc);
  else if (dtype == 1)
    quant_read_kernel<Half><<<grid, blk, 0, s>>>(p, sc);
  else
    quant_read_kernel<Single><<<grid, blk, 0, s>>>(p, sc);
  return hipGetLastError();
}

}  // namespace gdn
