// The norm of query and key heads with the rotation in the same pass, the append
// that does both on the way, and their gradient.
//
// For a row x of D values, with w' = offset + w and R the rotation of its position:
//   r = (sum x^2 / D + eps)^(-1/2),   out = R (x r w').
// For the gradient g of out, with y = R^T g (the opposite angles) and n = y w':
//   dx = r (n - x r^2 (sum n x) / D),   dw = sum over the rows of y x r.
// Every value is read once and written once, so both are bound by memory: the gradient
// of 32,768 tokens (40 heads of 128, bf16, 1.02 GB) 187 to 190 us, 5.4 TB/s, 6 of them
// the sum over the workgroups (an elementwise sum of two tensors into a third: 5.9).  The
// norm of as many in bf16 (688 MB) 165 us, 4.2 TB/s, in fp32 (1.36 GB) 229 us, 5.9 TB/s;
// on the way of a 16-bit append, 14,652 tokens of 48 heads (368 MB) 98 us, 67 without it.
//
// A row is a power of two of neighbouring lanes', each with the two pieces of W
// values that the rotation pairs (as in rope_kernel), so the row's sums are
// exchanges among them and a lane keeps its columns: it reads its weights once, and
// in the gradient adds up its columns' dw in registers over all the rows it takes.
// A workgroup's sums go to the workspace, and a second kernel adds them in a fixed
// order: the same inputs give the same dw.
#include <algorithm>

#include "gdn_rows.h"

namespace gdn {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormTokens = 64;  // most tokens of a workgroup at a time

// Units a lane takes: 2 W values each, D <= kNormMaxDim over 64 lanes (W = 1: a pair or one value).
template <int W>
constexpr int kNormUnits = W >= 4 ? 1 : W == 2 ? 2 : 8;

template <class Tag, bool NEAR, int W, bool NT>
__global__ __launch_bounds__(kNormThreads) void norm_rope_kernel(RopeParams p, NormDev n) {
  typedef typename Tag::type E;
  constexpr int R = kNormUnits<W>;
  __shared__ Place place[kNormTokens];
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.T - t0);
  if (threadIdx.x < 64) find_places(p, t0, tokens, place);
  const int L = 1 << n.shift, sub = threadIdx.x & (L - 1);
  float wq[R][2][W], wk[R][2][W];
  load_weights<Tag, NEAR, W, R>(n, n.wq, p.D, p.rot, wq);
  load_weights<Tag, NEAR, W, R>(n, n.wk, p.D, p.rot, wk);
  __syncthreads();

  const uint32_t H = p.heads.d, rows = (uint32_t)tokens * H;
  for (uint32_t row = threadIdx.x >> n.shift; row < rows; row += kNormThreads >> n.shift) {
    const uint32_t tok = div_by(row, p.heads);
    int h = (int)(row - tok * H);
    const int64_t t = t0 + tok;
    const Place pl = place[tok];
    const E* src;
    E* dst;
    bool is_q = false, is_v = false;
    if (h < p.Hq) {
      is_q = true;
      if (p.cu && pl.pos == kBehind) continue;
      src = (const E*)p.q.p + t * p.q.ts + h * p.q.hs;
      dst = (E*)p.q_out.p + t * p.q_out.ts + h * p.q_out.hs;
    } else if ((h -= p.Hq) < p.Hk) {
      src = (const E*)p.k.p + t * p.k.ts + h * p.k.hs;
      dst = p.Hv ? (E*)p.kv.k + pl.dst + h * p.kv.hs : (E*)p.k_out.p + t * p.k_out.ts + h * p.k_out.hs;
      if (p.Hv && pl.dst < 0) continue;
    } else {
      h -= p.Hk;
      is_v = true;
      src = (const E*)p.v.p + t * p.v.ts + h * p.v.hs;
      dst = (E*)p.kv.v + pl.dst + h * p.kv.hs;
      if (pl.dst < 0) continue;
    }
    const bool normed = !is_v && (is_q ? n.wq : n.wk) != nullptr;
    float x[R][2][W], sum = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int w = sub + r * L;
      if (w >= n.units) continue;
      const Columns<NEAR, W> c(w, p.D, p.rot);
      load_unit<W, NT>(src, c.a, c.b, x[r]);
#pragma unroll
      for (int i = 0; i < W; ++i) sum = __builtin_fmaf(x[r][0][i], x[r][0][i], __builtin_fmaf(x[r][1][i], x[r][1][i], sum));
    }
    const float f = normed ? rsqrtf(__builtin_fmaf(row_sum(sum, L), n.inv_dim, n.eps)) : 1.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int w = sub + r * L;
      if (w >= n.units) continue;
      const Columns<NEAR, W> c(w, p.D, p.rot);
      if (normed) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          x[r][0][i] *= f * (is_q ? wq[r][0][i] : wk[r][0][i]);
          x[r][1][i] *= f * (is_q ? wq[r][1][i] : wk[r][1][i]);
        }
      }
      if (c.turned && !is_v) turn_unit<NEAR, W>(p, pl.pos, c.a, c.b, p.sign, x[r]);
      store_unit<W, NT>(dst, c.a, c.b, x[r]);
    }
  }
}

// The gradient: the first workgroups take the queries' rows, the others the keys'.
template <class Tag, bool NEAR, int W, bool NT>
__global__ __launch_bounds__(kNormThreads) void norm_rope_grad_kernel(RopeParams p, NormDev n, NormGradDev g,
                                                                     float* partial) {
  typedef typename Tag::type E;
  constexpr int R = kNormUnits<W>;
  extern __shared__ float sums[];  // [rows at a time][D]
  const int which = (int)blockIdx.x < g.kind[0].blocks ? 0 : 1;
  const NormGradDev::Kind& kind = g.kind[which];
  const int me = blockIdx.x - (which ? g.kind[0].blocks : 0), per = kind.tokens;
  const int L = 1 << n.shift, sub = threadIdx.x & (L - 1);
  float wt[R][2][W], dw[R][2][W];
  load_weights<Tag, NEAR, W, R>(n, kind.w, p.D, p.rot, wt);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < W; ++i) dw[r][0][i] = dw[r][1][i] = 0.f;

  for (int64_t t0 = (int64_t)me * per; t0 < p.T; t0 += (int64_t)kind.blocks * per) {
    const int tokens = (int)min((int64_t)per, p.T - t0);
    const uint32_t rows = (uint32_t)tokens * kind.heads.d, groups = kNormThreads >> n.shift;
    for (uint32_t row = threadIdx.x >> n.shift; row < rows; row += groups) {
      const uint32_t tok = div_by(row, kind.heads);
      const int h = (int)(row - tok * kind.heads.d);
      const int64_t t = t0 + tok;
      // (32 rows of a position and more: from the cache, sooner than by way of LDS and a barrier)
      const int64_t pos = p.pos64 ? ((const int64_t*)p.pos)[t] : (int64_t)((const int32_t*)p.pos)[t];
      const E* src = (const E*)kind.x.p + t * kind.x.ts + h * kind.x.hs;
      const E* grad = (const E*)kind.g.p + t * kind.g.ts + h * kind.g.hs;
      float x[R][2][W], y[R][2][W], square = 0.f, along = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int w = sub + r * L;
        if (w >= n.units) continue;
        const Columns<NEAR, W> c(w, p.D, p.rot);
        load_unit<W, NT>(src, c.a, c.b, x[r]);
        load_unit<W, NT>(grad, c.a, c.b, y[r]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int w = sub + r * L;
        if (w >= n.units) continue;
        const Columns<NEAR, W> c(w, p.D, p.rot);
        if (c.turned) turn_unit<NEAR, W>(p, pos, c.a, c.b, -p.sign, y[r]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            square = __builtin_fmaf(x[r][k][i], x[r][k][i], square);
            along = __builtin_fmaf(y[r][k][i] * wt[r][k][i], x[r][k][i], along);
          }
      }
      const float f = rsqrtf(__builtin_fmaf(row_sum(square, L), n.inv_dim, n.eps));
      const float back = f * f * row_sum(along, L) * n.inv_dim;
      E* dst = (E*)kind.dx.p + t * kind.dx.ts + h * kind.dx.hs;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int w = sub + r * L;
        if (w >= n.units) continue;
        const Columns<NEAR, W> c(w, p.D, p.rot);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float xr = x[r][k][i];
            dw[r][k][i] = __builtin_fmaf(y[r][k][i], xr * f, dw[r][k][i]);
            x[r][k][i] = f * __builtin_fmaf(xr, -back, y[r][k][i] * wt[r][k][i]);
          }
        store_unit<W, NT>(dst, c.a, c.b, x[r]);
      }
    }
  }
  // the workgroup's sums, column by column
  const int group = threadIdx.x >> n.shift, groups = kNormThreads >> n.shift;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int w = sub + r * L;
    if (w >= n.units) continue;
    const Columns<NEAR, W> c(w, p.D, p.rot);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sums[group * p.D + c.a + i] = dw[r][0][i];
      if (W > 1 || c.b >= 0) sums[group * p.D + c.b + i] = dw[r][1][i];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.D; c += kNormThreads) {
    float s = 0.f;
    for (int g = 0; g < groups; ++g) s += sums[g * p.D + c];
    partial[(int64_t)blockIdx.x * p.D + c] = s;
  }
}

// dw from the workgroups' sums: 16 columns a workgroup, 64 of the sums at once.
template <class Tag>
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* partial, int D, int q_blocks, int blocks, int wide,
                                                           void* dwq, void* dwk) {
  __shared__ float s[64][17];
  const int col = threadIdx.x & 15, part = threadIdx.x >> 4, c = blockIdx.x * 16 + col;
  const int b0 = blockIdx.y ? q_blocks : 0, b1 = blockIdx.y ? blocks : q_blocks;
  float sum = 0.f;
  if (c < D)
    for (int b = b0 + part; b < b1; b += 64) sum += partial[(int64_t)b * D + c];
  s[part][col] = sum;
  __syncthreads();
  for (int m = 32; m > 0; m >>= 1) {
    if (part < m) s[part][col] += s[part + m][col];
    __syncthreads();
  }
  void* out = blockIdx.y ? dwk : dwq;
  if (part == 0 && c < D && out) {
    if (wide)
      ((float*)out)[c] = s[0][col];
    else
      from_f(s[0][col], ((typename Tag::type*)out)[c]);
  }
}

// Calls that write more than this pass the caches, as in rope_kernel.
constexpr int64_t kNormCacheBytes = 32 << 20;

// How rows are dealt: units of 2 W values, and lanes of a row.
template <int W>
void set_units(const RopeParams& p, NormDev& n) {
  n.units = rope_units(p, W);
  n.shift = 0;
  while ((1 << n.shift) < std::min(n.units, 64)) ++n.shift;
  n.inv_dim = 1.f / (float)p.D;
}

template <class Tag, bool NEAR, int W>
hipError_t launch_norm_width(RopeParams p, NormDev n, hipStream_t s) {
  constexpr int kMost = 16 / sizeof(typename Tag::type);
  set_units<W>(p, n);
  const int H = p.Hq + p.Hk + p.Hv;
  p.heads = fast_div(H);
  const int64_t per_token = (int64_t)H << n.shift;
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(kNormTokens, 2 * kNormThreads / per_token));
  const dim3 grid((uint32_t)((p.T + p.tokens_per_block - 1) / p.tokens_per_block)), blk(kNormThreads);
  if constexpr (W == kMost) {
    if (p.T * H * p.D * (int64_t)sizeof(typename Tag::type) > kNormCacheBytes) {
      norm_rope_kernel<Tag, NEAR, W, true><<<grid, blk, 0, s>>>(p, n);
      return hipGetLastError();
    }
  }
  norm_rope_kernel<Tag, NEAR, W, false><<<grid, blk, 0, s>>>(p, n);
  return hipGetLastError();
}

// Workgroups of the gradient: what the compute units hold at once, fewer for few rows; the keys' share
// of them by heads.  They take turns of two rows a thread (32,768 tokens: 190 us; four rows 197, sixteen 215:
// neighbours in memory are best read at once); two rows on the way in a thread leave room for fewer waves (203).
struct GradGrid {
  int q_blocks, k_blocks;
};
GradGrid grad_grid(int64_t T, int Hq, int Hk, int rows_at_once) {
  const int64_t all = 4 * (int64_t)device_cus();
  auto blocks = [&](int H) {
    const int64_t rows = T * H, most = (rows + rows_at_once - 1) / rows_at_once;
    return (int)(H ? std::max<int64_t>(1, std::min(most, all * H / (Hq + Hk))) : 0);
  };
  return GradGrid{blocks(Hq), blocks(Hk)};
}

template <class Tag, bool NEAR, int W>
hipError_t launch_grad_width(RopeParams p, NormDev n, NormGradDev g, void* dwq, void* dwk, float* partial, hipStream_t s) {
  constexpr int kMost = 16 / sizeof(typename Tag::type);
  set_units<W>(p, n);
  const int groups = kNormThreads >> n.shift;
  const GradGrid grid = grad_grid(p.T, p.Hq, p.Hk, groups);
  auto deal = [&](NormGradDev::Kind& k, int H, int blocks) {
    const int64_t share = blocks ? (p.T + blocks - 1) / blocks : 1, few = std::max(1, 2 * groups / std::max(1, H));
    k.blocks = blocks;
    k.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({share, kNormTokens, few}));
  };
  deal(g.kind[0], p.Hq, grid.q_blocks);
  deal(g.kind[1], p.Hk, grid.k_blocks);
  const int blocks = grid.q_blocks + grid.k_blocks;
  const size_t lds = (size_t)groups * p.D * sizeof(float);
  bool nt = false;
  if constexpr (W == kMost) {
    nt = p.T * (p.Hq + p.Hk) * p.D * (int64_t)sizeof(typename Tag::type) > kNormCacheBytes;
    if (nt) norm_rope_grad_kernel<Tag, NEAR, W, true><<<dim3(blocks), dim3(kNormThreads), lds, s>>>(p, n, g, partial);
  }
  if (!nt) norm_rope_grad_kernel<Tag, NEAR, W, false><<<dim3(blocks), dim3(kNormThreads), lds, s>>>(p, n, g, partial);
  if (hipError_t e = hipGetLastError()) return e;
  norm_weight_kernel<Tag><<<dim3((p.D + 15) / 16, p.Hk ? 2 : 1), dim3(1024), 0, s>>>(partial, p.D, grid.q_blocks, blocks, n.wide,
                                                                                    dwq, dwk);
  return hipGetLastError();
}

// f(Tag, NEAR, W) for a type, layout and piece width
template <class Tag, bool NEAR, class F>
hipError_t by_width(int width, F f) {
  if constexpr (sizeof(typename Tag::type) == 2)
    if (width == 8) return f.template operator()<Tag, NEAR, 8>();
  if (width == 4) return f.template operator()<Tag, NEAR, 4>();
  if (width == 2) return f.template operator()<Tag, NEAR, 2>();
  return f.template operator()<Tag, NEAR, 1>();
}
template <class F>
hipError_t by_type(int dtype, bool near_, int width, F f) {
  if (dtype == 0) return near_ ? by_width<Bf16, true>(width, f) : by_width<Bf16, false>(width, f);
  if (dtype == 1) return near_ ? by_width<Half, true>(width, f) : by_width<Half, false>(width, f);
  return near_ ? by_width<Single, true>(width, f) : by_width<Single, false>(width, f);
}

struct Forward {
  const RopeParams& p;
  const NormDev& n;
  hipStream_t s;
  template <class Tag, bool NEAR, int W>
  hipError_t operator()() const {
    return launch_norm_width<Tag, NEAR, W>(p, n, s);
  }
};
struct Backward {
  const RopeParams& p;
  const NormDev& n;
  const NormGradDev& g;
  void *dwq, *dwk;
  float* partial;
  hipStream_t s;
  template <class Tag, bool NEAR, int W>
  hipError_t operator()() const {
    return launch_grad_width<Tag, NEAR, W>(p, n, g, dwq, dwk, partial, s);
  }
};

}  // namespace

hipError_t launch_norm_rope(const RopeParams& p, const NormDev& n, int dtype, bool interleaved, int width, hipStream_t s) {
  if (p.T == 0 || p.Hq + p.Hk + p.Hv == 0) return hipSuccess;
  return by_type(dtype, interleaved, width, Forward{p, n, s});
}

hipError_t launch_norm_rope_grad(const RopeParams& p, const NormDev& n, const NormGradDev& g, int dtype, bool interleaved,
                                 int width, void* dwq, void* dwk, float* partial, hipStream_t s) {
  return by_type(dtype, interleaved, width, Backward{p, n, g, dwq, dwk, partial, s});
}

size_t norm_rope_grad_bytes(int D, int64_t T, int Hq, int Hk) {
  // (most workgroups where a row takes most lanes: 4 rows at once)
  const GradGrid g = grad_grid(T, Hq, Hk, kNormThreads / 64);
  return (size_t)(g.q_blocks + g.k_blocks) * D * sizeof(float);
}

}  // namespace gdn
