// Device helpers of the kernels that work on rows of heads: pieces of values in any
// element type, the turn of a pair, and the places of a batch's tokens.
#pragma once

#include "gdn_internal.h"

namespace gdn {

namespace {

struct Bf16 {
  typedef u16 type;
  static constexpr bool kFp16 = false;
};
struct Half {
  typedef _Float16 type;
  static constexpr bool kFp16 = true;
};
struct Single {
  typedef float type;
  static constexpr bool kFp16 = false;
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

// A token of the workgroup: its position, and where its key and value go in the
// cache (elements; -1: nowhere).
struct Place {
  int64_t pos, dst;
};
constexpr int64_t kBehind = INT64_MIN;  // the position of a row behind the last sequence

// Finds the places of tokens t0 .. t0 + tokens (64 at most), one a lane; the whole first wave calls it.
__device__ __forceinline__ void find_places(const RopeParams& p, int64_t t0, int tokens, Place* place) {
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
      Place pl{kBehind, -1};
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

// The columns of unit w: two pieces of W from a and b; W = 1: one pair, or a alone (b = -1).
template <bool NEAR, int W>
struct Columns {
  int a, b;
  bool turned;
  __device__ __forceinline__ Columns(int w, int D, int rot) {
    const int half = rot >> 1;
    if constexpr (W > 1) {
      const int units = rot / (2 * W);
      turned = w < units;
      a = W * (turned ? w : w + units);
      b = a + (turned ? half : (D >> 1) - W * units);
    } else {
      turned = w < half;
      a = !turned ? w + half : NEAR ? 2 * w : w;
      b = !turned ? -1 : NEAR ? a + 1 : a + half;
    }
  }
};

template <int W, bool NT, typename E>
__device__ __forceinline__ void load_unit(const E* row, int a, int b, float (&x)[2][W]) {
  if constexpr (W > 1) {
    load<W, NT>(row + a, x[0]);
    load<W, NT>(row + b, x[1]);
  } else {
    x[0][0] = to_f(row[a]);
    x[1][0] = b < 0 ? 0.f : to_f(row[b]);
  }
}
template <int W, bool NT, typename E>
__device__ __forceinline__ void store_unit(E* row, int a, int b, const float (&x)[2][W]) {
  if constexpr (W > 1) {
    store<NT, W>(row + a, x[0]);
    store<NT, W>(row + b, x[1]);
  } else {
    from_f(x[0][0], row[a]);
    if (b >= 0) from_f(x[1][0], row[b]);
  }
}

// The unit turned by its position's angles (sign -1: the opposite ones).
template <bool NEAR, int W>
__device__ __forceinline__ void turn_unit(const RopeParams& p, int64_t pos, int a, int b, float sign, float (&x)[2][W]) {
  const bool known = pos >= 0 && pos < p.table_rows;
  const int half = p.rot >> 1;
  const float* tab = p.table + (known ? pos : 0) * p.rot;
  if constexpr (W > 1) {
    constexpr int P = NEAR ? W / 2 : W;
    float c[2][P], s[2][P];
#pragma unroll
    for (int k = 0; k < (NEAR ? 2 : 1); ++k) {
      const float* t = tab + (NEAR ? (k ? b : a) / 2 : a);
      if (known) {
        load<P>(t, c[k]);
        load<P>(t + half, s[k]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!known) c[k][i] = s[k][i] = __builtin_nanf("");
        s[k][i] *= sign;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (NEAR) {
        turn_pair(x[0][2 * i], x[0][2 * i + 1], c[0][i], s[0][i]);
        turn_pair(x[1][2 * i], x[1][2 * i + 1], c[1][i], s[1][i]);
      } else {
        turn_pair(x[0][i], x[1][i], c[0][i], s[0][i]);
      }
    }
  } else {
    const int i = NEAR ? a / 2 : a;
    const float c = known ? tab[i] : __builtin_nanf(""), s = known ? tab[half + i] * sign : c;
    turn_pair(x[0][0], x[1][0], c, s);
  }
}

// A lane's weights, offset added (0 in units past the row's).
template <class Tag, bool NEAR, int W, int R>
__device__ __forceinline__ void load_weights(const NormDev& n, const void* w, int D, int rot, float (&x)[R][2][W]) {
  const int L = 1 << n.shift, sub = threadIdx.x & (L - 1);
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[r][0][i] = x[r][1][i] = 0.f;
    if (w && sub + r * L < n.units) {
      const Columns<NEAR, W> c(sub + r * L, D, rot);
      if (W > 1 && n.vector) {
        if (n.wide) {
#pragma unroll
          for (int i = 0; i < W; i += W < 4 ? W : 4) {
            load<(W < 4 ? W : 4)>((const float*)w + c.a + i, *(float(*)[W < 4 ? W : 4])(x[r][0] + i));
            load<(W < 4 ? W : 4)>((const float*)w + c.b + i, *(float(*)[W < 4 ? W : 4])(x[r][1] + i));
          }
        } else {
          load<W>((const typename Tag::type*)w + c.a, x[r][0]);
          load<W>((const typename Tag::type*)w + c.b, x[r][1]);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          x[r][0][i] += n.offset;
          x[r][1][i] += n.offset;
        }
        continue;
      }
      // (one by one: the weights may start anywhere)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float u = n.wide ? ((const float*)w)[c.a + i] : to_f(((const typename Tag::type*)w)[c.a + i]);
        x[r][0][i] = n.offset + u;
        if (W > 1 || c.b >= 0) {
          const float v = n.wide ? ((const float*)w)[c.b + i] : to_f(((const typename Tag::type*)w)[c.b + i]);
          x[r][1][i] = n.offset + v;
        }
      }
    }
  }
}

// x of the lane that a DPP control names (quad_perm, half_mirror, mirror: within 16 lanes).
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
// The sum over a row's lanes, a power of two of neighbours (up to 16 of them without LDS: the
// sums of pairs, quads and eights are all their lanes', so any lane of the other one will do).
__device__ __forceinline__ float row_sum(float x, int lanes) {
  if (lanes > 1) x += dpp<0xb1>(x);   // quad_perm 1 0 3 2
  if (lanes > 2) x += dpp<0x4e>(x);   // quad_perm 2 3 0 1
  if (lanes > 4) x += dpp<0x141>(x);  // row_half_mirror
  if (lanes > 8) x += dpp<0x140>(x);  // row_mirror
  for (int m = 16; m < lanes; m <<= 1) x += __shfl_xor(x, m, 64);
  return x;
}

}  // namespace

}  // namespace gdn
