// Rotary positions, and the append to a paged key/value cache that applies them
// on the way.
//
// Pair i of a row at position t is turned by the angle t f_i:
//   (a, b) -> (a c - b s, b c + a s),   c, s from the caller's table,
// or by the opposite angle (transposed: the gradient's map; the table's
// magnitude stays).  Every value is read once and written once, two products and
// a sum each, so the kernel is bound by memory.
//
// A thread takes 16 values of a row, in two 16-byte (fp32: 32-byte) pieces that
// hold eight whole pairs: values 8u .. and rot/2 + 8u .. of the half layout, 16
// neighbours otherwise, so no value moves between lanes.  Rows whose sizes,
// strides or addresses do not allow 16-byte accesses take one pair a thread.
// A workgroup takes as many tokens as keep its threads busy; their places in the
// page table are looked up once per token, by one lane each.
#include <algorithm>

#include "gdn_internal.h"

namespace gdn {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

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

__device__ __forceinline__ void load8(const u16* p, float (&x)[8]) {
  const u32x4 w = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const _Float16* p, float (&x)[8]) {
  const f16x8 w = *(const f16x8*)p;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)w[i];
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = a[i];
    x[4 + i] = b[i];
  }
}
template <bool NT, typename V>
__device__ __forceinline__ void put(V* p, V w) {
  if constexpr (NT)
    __builtin_nontemporal_store(w, p);
  else
    *p = w;
}
template <bool NT>
__device__ __forceinline__ void store8(u16* p, const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f2bf2(x[2 * i], x[2 * i + 1]);
  put<NT>((u32x4*)p, w);
}
template <bool NT>
__device__ __forceinline__ void store8(_Float16* p, const float (&x)[8]) {
  f16x8 w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (_Float16)x[i];
  put<NT>((f16x8*)p, w);
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  put<NT>((f32x4*)p, f32x4{x[0], x[1], x[2], x[3]});
  put<NT>((f32x4*)(p + 4), f32x4{x[4], x[5], x[6], x[7]});
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

// Stores pass the caches (NT) when the call writes more than the L2s hold together:
// 369 MB of prompts 74.4 -> 63.4 us, 688 MB of gradients 127.7 -> 123.8 us (5.6-5.8
// TB/s, the rate of a copy); below that the next kernel may find them there.
constexpr int64_t kCacheBytes = 32 << 20;

template <class Tag, bool NEAR, bool VEC, bool NT>
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
    if constexpr (VEC) {
      int a = 16 * w, b = a + 8;
      turn = turn && a < rot;
      if (!NEAR && turn) {
        a = 8 * w;
        b = half + a;
      }
      float x[8], y[8];
      load8(src + a, x);
      load8(src + b, y);
      if (turn) {
        float c[8], s[8];
        load8(tab + 8 * w, c);
        load8(tab + half + 8 * w, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!known) c[i] = s[i] = __builtin_nanf("");
          s[i] *= p.sign;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!NEAR)
            turn_pair(x[i], y[i], c[i], s[i]);
          else if (i < 4)
            turn_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
          else
            turn_pair(y[2 * i - 8], y[2 * i - 7], c[i], s[i]);
        }
      }
      store8<NT>(dst + a, x);
      store8<NT>(dst + b, y);
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
void launch_rope_type(const RopeParams& p, bool vec, bool nt, dim3 grid, hipStream_t s) {
  const dim3 blk(kRopeThreads);
  if (!vec)
    rope_kernel<Tag, NEAR, false, false><<<grid, blk, 0, s>>>(p);
  else if (nt)
    rope_kernel<Tag, NEAR, true, true><<<grid, blk, 0, s>>>(p);
  else
    rope_kernel<Tag, NEAR, true, false><<<grid, blk, 0, s>>>(p);
}
template <class Tag>
void launch_rope_type(const RopeParams& p, bool near_, bool vec, dim3 grid, hipStream_t s) {
  const bool nt = p.T * (p.Hq + p.Hk + p.Hv) * p.D * (int64_t)sizeof(typename Tag::type) > kCacheBytes;
  if (near_)
    launch_rope_type<Tag, true>(p, vec, nt, grid, s);
  else
    launch_rope_type<Tag, false>(p, vec, nt, grid, s);
}

}  // namespace

hipError_t launch_rope(RopeParams p, int dtype, bool interleaved, bool vec, hipStream_t s) {
  const int H = p.Hq + p.Hk + p.Hv;
  if (p.T == 0 || H == 0) return hipSuccess;
  const int units = vec ? p.D / 16 : p.D - p.rot / 2;
  p.heads = fast_div(H);
  p.row_units = fast_div(units);
  // two rounds of the workgroup's threads
  const int64_t per_token = (int64_t)H * units;
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(kRopeTokens, 2 * kRopeThreads / per_token));
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block));
  if (dtype == 0)
    launch_rope_type<Bf16>(p, interleaved, vec, grid, s);
  else if (dtype == 1)
    launch_rope_type<Half>(p, interleaved, vec, grid, s);
  else
    launch_rope_type<Single>(p, interleaved, vec, grid, s);
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
