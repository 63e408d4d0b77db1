// Rotary positions, and the append to a paged key/value cache that applies them
// on the way.
//
// Pair i of a row at position t is turned by the angle t f_i:
//   (a, b) -> (a c - b s, b c + a s),   c, s from the caller's table,
// or by the opposite angle (transposed: the gradient's map; the table's
// magnitude stays).  Every value is read once and written once, two products and
// a sum each, so the kernel is bound by memory.
//
// A thread takes 2 W values of a row, in two pieces: values W u .. and rot/2 + W u
// .., which hold W whole pairs in either layout (pairs across the two, or W / 2
// within each), so no value moves between lanes and neighbouring threads take
// neighbouring pieces.  A piece is 16 bytes, or less where the sizes, strides or
// addresses allow no more (heads of 80 values of which 20 turn: W = 2), or one pair
// a thread.
// A workgroup takes as many tokens as keep its threads busy; their places in the
// page table are looked up once per token, by one lane each.
#include <algorithm>

#include "gdn_internal.h"

namespace gdn {

namespace {

struct Bf16 {
  typedef u16 type;
};
struct Half {
  typedef _Float16 type;
};
struct Single {
  typedef float type;
};

__device__ __forceinline__ float to_f(u16 x) { return bf2f(x); }
__device__ __forceinline__ float to_f(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void from_f(float x, u16& y) { y = f2bf(x); }
__device__ __forceinline__ void from_f(float x, _Float16& y) { y = (_Float16)x; }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }

// W values at once, 16 bytes at most.
template <int W, typename E>
struct Piece {
  typedef E type __attribute__((ext_vector_type(W)));
};
template <bool NT, typename V>
__device__ __forceinline__ void put(V* p, V w) {
  if constexpr (NT)
    __builtin_nontemporal_store(w, p);
  else
    *p = w;
}
template <bool NT, typename V>
__device__ __forceinline__ V get(const V* p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}
template <int W, bool NT = false, typename E>
__device__ __forceinline__ void load(const E* p, float (&x)[W]) {
  const typename Piece<W, E>::type w = get<NT>((const typename Piece<W, E>::type*)p);
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = to_f(w[i]);
}
template <bool NT, int W, typename E>
__device__ __forceinline__ void store(E* p, const float (&x)[W]) {
  typename Piece<W, E>::type w;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    E y;
    from_f(x[i], y);
    w[i] = y;
  }
  put<NT>((typename Piece<W, E>::type*)p, w);
}

// (a c - b s, b c + a s), one product of each rounded and the other fused, the
// same in every path
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = a;
  a = __builtin_fmaf(x, c, -(b * s));
  b = __builtin_fmaf(b, c, x * s);
}

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 64;  // most tokens of a workgroup

// A token of the workgroup: its position, and where its key and value go in the
// cache (elements; -1: nowhere).
struct Place {
  int64_t pos, dst;
};

// Loads and stores pass the caches (NT) when the call writes more than the L2s hold
// together; below that the next kernel may find the rows there.  Other rows in every
// call: 368 MB of prompts 69 us (5.3 TB/s; 72 when the loads stay), 688 MB of
// gradients 115 us (6.0 TB/s; 117 when the loads stay, 128 when the stores do too; a
// copy reaches 5.7-6.0); the same prompts again and again, part of which the
// memory-side cache then holds, 56 us, 74 when the stores stay.
constexpr int64_t kCacheBytes = 32 << 20;

template <class Tag, bool NEAR, int W, bool NT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  typedef typename Tag::type E;
  __shared__ Place place[kRopeTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);

  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const int64_t t = t0 + lane;
    if (p.pos) {
      if (lane < tokens)
        place[lane] = Place{p.pos64 ? ((const int64_t*)p.pos)[t] : (int64_t)((const int32_t*)p.pos)[t], -1};
    } else {
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
        Place pl{-1, -1};
        if (b < p.kv.B) {
          const int first = p.kv.ptr[b], pages = p.kv.ptr[b + 1] - first;
          const int64_t len = pages > 0 ? (int64_t)(pages - 1) * p.kv.page.d + p.kv.lpl[b] : 0;
          const int64_t pos = p.cu ? t - p.cu[b + 1] + len : len - 1;
          pl.pos = pos;
          if (pos >= 0 && pos < len) {
            const int pg = (int)div_by((uint32_t)pos, p.kv.page);
            pl.dst = (int64_t)p.kv.idx[first + pg] * p.kv.ps + (pos - (int64_t)pg * p.kv.page.d) * p.kv.ts;
          }
        }
        place[lane] = pl;
      }
    }
  }
  __syncthreads();

  const int rot = p.rot, half = rot >> 1;
  const uint32_t H = p.heads.d, total = (uint32_t)tokens * H * p.row_units.d;
  for (uint32_t u = threadIdx.x; u < total; u += kRopeThreads) {
    const uint32_t row = div_by(u, p.row_units);
    const int w = (int)(u - row * p.row_units.d);
    const uint32_t tok = div_by(row, p.heads);
    int h = (int)(row - tok * H);
    const int64_t t = t0 + tok;
    const Place pl = place[tok];
    const E* src;
    E* dst;
    bool turn = rot > 0;
    if (h < p.Hq) {
      src = (const E*)p.q.p + t * p.q.ts + h * p.q.hs;
      dst = (E*)p.q_out.p + t * p.q_out.ts + h * p.q_out.hs;
    } else if ((h -= p.Hq) < p.Hk) {
      src = (const E*)p.k.p + t * p.k.ts + h * p.k.hs;
      dst = p.Hv ? (E*)p.kv.k + pl.dst + h * p.kv.hs : (E*)p.k_out.p + t * p.k_out.ts + h * p.k_out.hs;
      if (p.Hv && pl.dst < 0) continue;
    } else {
      h -= p.Hk;
      src = (const E*)p.v.p + t * p.v.ts + h * p.v.hs;
      dst = (E*)p.kv.v + pl.dst + h * p.kv.hs;
      if (pl.dst < 0) continue;
      turn = false;
    }
    const bool known = pl.pos >= 0 && pl.pos < p.table_rows;
    const float* tab = p.table + (known ? pl.pos : 0) * rot;
    if constexpr (W > 1) {
      // the turned part, or what passes: two halves either way
      const int turned = turn ? rot / (2 * W) : 0;
      turn = w < turned;
      const int a = W * (turn ? w : w + turned);
      const int b = a + (turn ? half : (p.D >> 1) - W * turned);
      float x[W], y[W];
      load<W, NT>(src + a, x);
      load<W, NT>(src + b, y);
      if (turn) {
        // cosines and sines: of the pairs across the pieces, or of each one's own
        constexpr int P = NEAR ? W / 2 : W;
        float c[2][P], s[2][P];
#pragma unroll
        for (int k = 0; k < (NEAR ? 2 : 1); ++k) {
          const float* t = tab + (NEAR ? (k ? b : a) / 2 : a);
          load<P>(t, c[k]);
          load<P>(t + half, s[k]);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (!known) c[k][i] = s[k][i] = __builtin_nanf("");
            s[k][i] *= p.sign;
          }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if constexpr (NEAR) {
            turn_pair(x[2 * i], x[2 * i + 1], c[0][i], s[0][i]);
            turn_pair(y[2 * i], y[2 * i + 1], c[1][i], s[1][i]);
          } else {
            turn_pair(x[i], y[i], c[0][i], s[0][i]);
          }
        }
      }
      store<NT, W>(dst + a, x);
      store<NT, W>(dst + b, y);
    } else if (turn && w < half) {
      const int a = NEAR ? 2 * w : w, b = NEAR ? a + 1 : a + half;
      const float c = known ? tab[w] : __builtin_nanf("");
      const float s = known ? tab[half + w] * p.sign : c;
      float x = to_f(src[a]), y = to_f(src[b]);
      turn_pair(x, y, c, s);
      from_f(x, dst[a]);
      from_f(y, dst[b]);
    } else {
      // row_units counts half + D - rot threads a row: value half + w, or, in
      // rows that are not turned, also the values the others' pairs would take
      if (turn) {
        dst[half + w] = src[half + w];
      } else {
        dst[w] = src[w];
        if (w + p.row_units.d < (uint32_t)p.D) dst[w + p.row_units.d] = src[w + p.row_units.d];
      }
    }
  }
}

// One thread per (position, pair): the angle and its cosine and sine in fp64.
// Run once per model; bound by the fp64 functions.
__global__ __launch_bounds__(256) void rope_table_kernel(float* table, int64_t rows, FastDiv half, double base,
                                                         double factor, int bands, double original, double low,
                                                         double high, double magnitude) {
  const int n = (int)half.d;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < rows * n; u += stride) {
    const int64_t t = u / n;
    const int i = (int)(u - t * n);
    double f = pow(base, -(double)i / n);
    if (bands) {
      const double turns = original * f / 6.283185307179586476925;
      const double w = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
      f *= (1.0 - w) / factor + w;
    } else {
      f /= factor;
    }
    double s, c;
    sincos((double)t * f, &s, &c);
    table[t * 2 * n + i] = (float)(magnitude * c);
    table[t * 2 * n + n + i] = (float)(magnitude * s);
  }
}

template <class Tag, bool NEAR>
void launch_rope_type(const RopeParams& p, int width, bool nt, dim3 grid, hipStream_t s) {
  const dim3 blk(kRopeThreads);
  constexpr int kMost = 16 / sizeof(typename Tag::type);  // 8, or 4 of fp32
  if (width == kMost && nt)
    rope_kernel<Tag, NEAR, kMost, true><<<grid, blk, 0, s>>>(p);
  else if (width == kMost)
    rope_kernel<Tag, NEAR, kMost, false><<<grid, blk, 0, s>>>(p);
  else if (width == 4)
    rope_kernel<Tag, NEAR, 4, false><<<grid, blk, 0, s>>>(p);
  else if (width == 2)
    rope_kernel<Tag, NEAR, 2, false><<<grid, blk, 0, s>>>(p);
  else
    rope_kernel<Tag, NEAR, 1, false><<<grid, blk, 0, s>>>(p);
}
template <class Tag>
void launch_rope_type(const RopeParams& p, bool near_, int width, dim3 grid, hipStream_t s) {
  const bool nt = p.T * (p.Hq + p.Hk + p.Hv) * p.D * (int64_t)sizeof(typename Tag::type) > kCacheBytes;
  if (near_)
    launch_rope_type<Tag, true>(p, width, nt, grid, s);
  else
    launch_rope_type<Tag, false>(p, width, nt, grid, s);
}

}  // namespace

hipError_t launch_rope(RopeParams p, int dtype, bool interleaved, int width, hipStream_t s) {
  const int H = p.Hq + p.Hk + p.Hv;
  if (p.T == 0 || H == 0) return hipSuccess;
  const int units = rope_units(p, width);
  p.heads = fast_div(H);
  p.row_units = fast_div(units);
  // two rounds of the workgroup's threads (one 72, two 72, four 74, eight 82 us for the prompts)
  const int64_t per_token = (int64_t)H * units;
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(kRopeTokens, 2 * kRopeThreads / per_token));
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block));
  if (dtype == 0)
    launch_rope_type<Bf16>(p, interleaved, width, grid, s);
  else if (dtype == 1)
    launch_rope_type<Half>(p, interleaved, width, grid, s);
  else
    launch_rope_type<Single>(p, interleaved, width, grid, s);
  return hipGetLastError();
}

hipError_t launch_rope_table(float* table, int64_t rows, int rot, double base, double factor, int bands,
                             double original, double low, double high, double magnitude, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int64_t n = rows * (rot / 2);
  const dim3 grid((uint32_t)std::min<int64_t>((n + 255) / 256, 65536));
  rope_table_kernel<<<grid, dim3(256), 0, s>>>(table, rows, fast_div(rot / 2), base, factor, bands, original, low,
                                               high, magnitude);
  return hipGetLastError();
}

}  // namespace gdn
