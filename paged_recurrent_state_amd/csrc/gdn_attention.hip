// Attention of a batch's new tokens over a paged key/value cache.
//
// For a query row q and the keys j it sees, with x_j = scale q . k_j (bounded by
// softcap * tanh(x / softcap) when asked for):
//   o = sum_j e^{x_j} v_j / sum_j e^{x_j},   lse = log sum_j e^{x_j},
// in one pass over the keys: a running reference m, the sum l of 2^{x - m} and
// the unnormalised output, all in fp32 and in log2 units; when a score exceeds
// the reference by more than kSlack the row's l and o are multiplied by
// 2^{m - m'}.  (Any reference gives the same quotient; one that lags behind the
// maximum by up to 2^kSlack costs no accuracy in floating point and makes the
// multiplication rare.)
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
#include <algorithm>
#include <atomic>

#include "gdn_internal.h"

namespace gdn {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kKeys = 64;        // keys of a tile
constexpr int kWaves = 4;
constexpr float kNoScore = -3.0e38f;  // reference before the first score
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Element types.  kBias: a new reference lies this far under the row's maximum,
// which puts 2^{x - m} where a half still holds small weights to full precision;
// kSlack more and the reference moves (2^(kBias + kSlack) stays in range).
struct Bf {
  static constexpr float kBias = 0.f, kSlack = 8.f;
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return f2bf2(a, b); }
};
struct Hf {
  static constexpr float kBias = 7.f, kSlack = 8.f;
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  }
};

// The value the other half of the wave (lane ^ 32) holds.
__device__ __forceinline__ float other_half(float x) {
  return __shfl_xor(x, 32, 64);
}

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

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

template <class E, int D, int NQ, bool CAP>
__global__ __launch_bounds__(64 * kWaves, 1) void chunk_kernel(AttnParams p) {
  constexpr int kRows = 32 * NQ * kWaves;  // query rows of a tile
  constexpr int kPieces = D / 8;           // 16-byte pieces of a row
  constexpr int kSteps = D / 16;           // MFMA steps over D
  constexpr int kBlocks = D / 32;          // 32-wide blocks of the output
  __shared__ __attribute__((aligned(16))) char sk[kKeys * D * 2];
  __shared__ __attribute__((aligned(16))) char sv[kKeys * D * 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, col = lane & 31;
  const int G = (int)p.group.d;
  const int hk = blockIdx.y;

  // which sequence and which of its tiles
  int b = -1, tile = 0, tok0 = 0, n = 0;
  {
    int before = 0;
    for (int b0 = 0; b0 < p.kv.B && b < 0; b0 += 64) {
      const int i = b0 + lane;
      int c0 = 0, c1 = 0;
      if (i < p.kv.B) {
        c0 = p.cu ? p.cu[i] : i;
        c1 = p.cu ? p.cu[i + 1] : i + 1;
      }
      const int t = (int)(((int64_t)(c1 - c0) * G + kRows - 1) / kRows);
      int incl = t;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(incl, off, 64);
        if (lane >= off) incl += y;
      }
      const uint64_t hit = __ballot(before + incl > (int)blockIdx.x);
      if (hit) {
        const int src = __ffsll((unsigned long long)hit) - 1;
        b = b0 + src;
        tile = (int)blockIdx.x - before - __shfl(incl - t, src, 64);
        tok0 = __shfl(c0, src, 64);
        n = __shfl(c1 - c0, src, 64);
      }
      before += __shfl(incl, 63, 64);
    }
    if (b < 0) return;
  }
  const int first_page = p.kv.ptr[b], pages = p.kv.ptr[b + 1] - first_page;
  const int len = pages > 0 ? (pages - 1) * (int)p.kv.page.d + p.kv.lpl[b] : 0;
  const int past = len - n;

  // this lane's rows
  int lim[NQ], low[NQ];  // keys low .. lim
  u32x4 q[NQ][kSteps];
#pragma unroll
  for (int a = 0; a < NQ; ++a) {
    const int row = tile * kRows + wave * 32 * NQ + a * 32 + col;
    const int tok = (int)div_by(row, p.group), g = row - tok * G;
    const bool real = tok < n;
    lim[a] = real ? (p.causal ? min(past + tok, len - 1) : len - 1) : -1;
    low[a] = real && p.window > 0 ? max(0, past + tok - p.window + 1) : 0;
    const u16* src = (const u16*)p.q.p + (int64_t)(tok0 + (real ? tok : 0)) * p.q.ts +
                     (int64_t)(hk * G + (real ? g : 0)) * p.q.hs + 8 * half;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[a][s] = *(const u32x4*)(src + 16 * s);
  }
  // the tile's keys
  const int last_tok = min(n - 1, (int)div_by(tile * kRows + kRows - 1, p.group));
  const int first_tok = (int)div_by(tile * kRows, p.group);
  const int key_end = p.causal ? min(past + last_tok + 1, len) : len;
  const int key_begin = p.window > 0 ? max(0, past + first_tok - p.window + 1) : 0;

  f32x16 o[NQ][kBlocks];
  float m[NQ], l[NQ];
#pragma unroll
  for (int a = 0; a < NQ; ++a) {
    m[a] = kNoScore;
    l[a] = 0.f;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[a][d][i] = 0.f;
  }

  const u32x4 zero{0u, 0u, 0u, 0u};
  for (int key0 = key_begin & ~(kKeys - 1); key0 < key_end; key0 += kKeys) {
    __syncthreads();
    constexpr int kLoads = kKeys * kPieces / (64 * kWaves);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int x = i * 64 * kWaves + threadIdx.x, r = x / kPieces, c = x % kPieces;
      const int key = key0 + r;
      u32x4 wk = zero, wv = zero;
      if (key < len) {
        const int pg = (int)div_by(key, p.kv.page);
        const int64_t at = (int64_t)p.kv.idx[first_page + pg] * p.kv.ps +
                           (int64_t)(key - pg * (int)p.kv.page.d) * p.kv.ts + hk * p.kv.hs + 8 * c;
        wk = *(const u32x4*)((const u16*)p.kv.k + at);
        wv = *(const u32x4*)((const u16*)p.kv.v + at);
      }
      *(u32x4*)(sk + k_at<D>(r, c)) = wk;
      *(u32x4*)(sv + v_at<D>(r, c)) = wv;
    }
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < kKeys / 32; ++kb) {
      f32x16 s[NQ];
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[a][i] = 0.f;
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        const u32x4 kf = *(const u32x4*)(sk + k_at<D>(kb * 32 + col, 2 * t + half));
#pragma unroll
        for (int a = 0; a < NQ; ++a) s[a] = E::mfma(kf, q[a][t], s[a]);
      }
      u32x4 pt[NQ][2];
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        // this lane's keys: base + 8 (i / 4) + i % 4
        const int base = key0 + kb * 32 + 4 * half;
        float x[16], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = base + 8 * (i >> 2) + (i & 3);
          x[i] = s[a][i] * p.scale;
          if constexpr (CAP) x[i] = p.cap * tanhf(x[i]);
          if (key > lim[a] || key < low[a]) x[i] = -INFINITY;
          top = fmaxf(top, x[i]);
        }
        if (__any(top > m[a] + (E::kBias + E::kSlack))) {
          top = fmaxf(top, other_half(top)) - E::kBias;
          const float to = fmaxf(m[a], top), f = __builtin_amdgcn_exp2f(m[a] - to);
          m[a] = to;
          l[a] *= f;
#pragma unroll
          for (int d = 0; d < kBlocks; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[a][d][i] *= f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = __builtin_amdgcn_exp2f(x[i] - m[a]);
          l[a] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) pt[a][i >> 2][i & 3] = E::pack(x[2 * i], x[2 * i + 1]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int d = 0; d < kBlocks; ++d) {
          // keys 16 t + 4 half + 0..3 and 8 more; lane i of a 16-lane group points
          // at 4 values of key i / 4 and receives value i of the four keys
          const int key = kb * 32 + 16 * t + 4 * half + ((lane & 15) >> 2);
          const int dim = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
          const int sub = (dim & 7) * 2;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(key, dim >> 3) + sub));
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(sv + v_at<D>(key + 8, dim >> 3) + sub));
          const u32x2 wl = __builtin_bit_cast(u32x2, lo), wh = __builtin_bit_cast(u32x2, hi);
          const u32x4 vf{wl[0], wl[1], wh[0], wh[1]};
#pragma unroll
          for (int a = 0; a < NQ; ++a) o[a][d] = E::mfma(vf, pt[a][t], o[a][d]);
        }
    }
  }

#pragma unroll
  for (int a = 0; a < NQ; ++a) {
    const float sum = l[a] + other_half(l[a]);
    const int row = tile * kRows + wave * 32 * NQ + a * 32 + col;
    const int tok = (int)div_by(row, p.group), g = row - tok * G;
    if (tok >= n) continue;
    const float inv = lim[a] < low[a] ? 0.f : 1.f / sum;
    const int64_t h = (int64_t)hk * G + g;
    u16* dst = (u16*)p.o.p + (int64_t)(tok0 + tok) * p.o.ts + h * p.o.hs;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x16& x = o[a][d];
        *(u32x2*)(dst + 32 * d + 8 * i + 4 * half) = u32x2{E::pack(x[4 * i] * inv, x[4 * i + 1] * inv),
                                                           E::pack(x[4 * i + 2] * inv, x[4 * i + 3] * inv)};
      }
    if (p.lse && half == 0)
      p.lse[(int64_t)(tok0 + tok) * p.Hq + h] =
          lim[a] < low[a] ? -INFINITY : (m[a] + __builtin_amdgcn_logf(sum)) * kLn2;
  }
}

template <class E, int D, int NQ>
hipError_t launch_chunk(const AttnParams& p, hipStream_t s) {
  constexpr int kRows = 32 * NQ * kWaves;
  const int64_t tiles = p.cu ? p.T * (int64_t)p.group.d / kRows + p.kv.B : p.kv.B * (int64_t)((p.group.d + kRows - 1) / kRows);
  const dim3 grid((uint32_t)tiles, (uint32_t)p.Hkv), blk(64 * kWaves);
  if (p.cap > 0.f)
    chunk_kernel<E, D, NQ, true><<<grid, blk, 0, s>>>(p);
  else
    chunk_kernel<E, D, NQ, false><<<grid, blk, 0, s>>>(p);
  return hipGetLastError();
}

template <class E>
hipError_t launch_type(const AttnParams& p, int D, hipStream_t s) {
  if (D == 64) return launch_chunk<E, 64, 2>(p, s);
  if (D == 128) return launch_chunk<E, 128, 2>(p, s);
  return launch_chunk<E, 256, 1>(p, s);
}

}  // namespace

hipError_t launch_attention(const AttnParams& p, int D, int dtype, hipStream_t s) {
  if (p.T == 0 || p.kv.B == 0) return hipSuccess;
  return dtype == 0 ? launch_type<Bf>(p, D, s) : launch_type<Hf>(p, D, s);
}

}  // namespace gdn
