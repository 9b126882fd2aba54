// Tree attention: dispatch, and the kernels before and after the attention proper
// (tq_tree_impl.cuh), which rotate the queries and merge the partials.
#include "tq_tree_plan.cuh"

#include <algorithm>

namespace tq {
namespace {

// ---- queries: rotated, scaled by a power of two, rounded to fp16, in the layout
// of the product's B operand (128-byte rows of 64 channels, swizzled; blocks of
// `rows` rows; parts hi, lo of an fp16 call, sketch).  Grid: (units, shares of the
// rows); every block reads all of the unit's rows for the scale (few units would
// leave most SMs idle: one block per unit took 13 us for 8 units of 252 rows).  It
// is common to its rows: |u| <= d max|q| is brought to 2^14, or 2^10 before the
// second rotation, which can add sqrt(d).  Rows that are not finite do not count, nor
// do rows of zeros.  A unit's rows are wild
//   where they differ by more than 2^16 (a padded draft with what its memory held): the
//     small ones would lose bits under a common scale;
//   where a score may pass 2^26 (the longest row with a key of the largest fp16 norm):
//     score * norm - maximum, rounded once, and the maximum, rounded before, would differ
//     by more than the weights have room for.
// Then each row has a scale of its own, the unit's is 0, and the attention finishes every
// score before it uses it (63 drafts at 32k: 138 us if wild, 79 if not).
constexpr int kPrepThreads = 1024;
constexpr int kWildLog2 = 16;
constexpr float kWildScore = 0x1p26f;

template <int D>
__global__ void __launch_bounds__(kPrepThreads)
    tree_query_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                      const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl, uint8_t* __restrict__ ws) {
  constexpr int E = D / 32, kLogD = D == 64 ? 6 : D == 128 ? 7 : 8;
  __shared__ uint32_t red[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c0 = lane * E;
  const int unit = blockIdx.x, units = cv.kv_heads * pl.blocks, b = unit / units, u0 = unit - b * units;
  const int kvh = u0 / pl.blocks, rb = u0 - kvh * pl.blocks, group = ta.q_heads / cv.kv_heads;
  const int rows = min(pl.rows, ta.n_q * group - rb * pl.rows);
  pdl_wait();
  pdl_trigger();  // the attention may start: it waits for this grid where it needs the queries
  auto load = [&](int rr, float (&x)[E]) {
    const int r = rb * pl.rows + rr, i = r / group, h = kvh * group + (r - i * group);
    const uint16_t* src = static_cast<const uint16_t*>(ta.q) + (((long)b * ta.n_q + i) * ta.q_heads + h) * D + c0;
    uint32_t w[E / 2];
    if constexpr (E == 2) w[0] = *reinterpret_cast<const uint32_t*>(src);
    else if constexpr (E == 4) {
      const uint2 y = *reinterpret_cast<const uint2*>(src);
      w[0] = y.x;
      w[1] = y.y;
    } else {
      const uint4 y = *reinterpret_cast<const uint4*>(src);
      w[0] = y.x;
      w[1] = y.y;
      w[2] = y.z;
      w[3] = y.w;
    }
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 f = ta.dtype == kBF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]))
                                         : __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  };
  // max|x| of a row, as bits (whose order is that of floats that are not negative, then
  // infinity, then NaN); 0 for one that does not count
  auto size = [&](const float (&x)[E]) {
    uint32_t t = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e) t = max(t, __float_as_uint(x[e]) & 0x7fffffffu);
    t = __reduce_max_sync(0xffffffffu, t);
    return t < 0x7f800000u ? t : 0u;
  };
  auto exponent = [&](uint32_t bits) {  // of d max|x|
    int ex = 0;
    frexpf(__uint_as_float(bits), &ex);
    return bits ? ex + kLogD : 1;
  };
  auto scale_of = [&](int ex) { return ldexpf(1.f, max(min((tb.qjl ? 10 : 14) - ex, 100), -126)); };
  uint32_t most = 0u, least = 0xffffffffu;
#pragma unroll 4
  for (int rr = warp; rr < rows; rr += 32) {
    float x[E];
    load(rr, x);
    const uint32_t t = size(x);
    most = max(most, t);
    least = min(least, t - 1u);  // (0 becomes the largest)
  }
  if (lane == 0) {
    red[0][warp] = most;
    red[1][warp] = least;
  }
  __syncthreads();
  most = __reduce_max_sync(0xffffffffu, red[0][lane]);
  least = __reduce_min_sync(0xffffffffu, red[1][lane]);
  const float root = sqrtf((float)D), longest = __uint_as_float(most) * root;
  const float key = 65504.f * (tb.affine ? root : 1.f) * (tb.qjl ? 1.f + sqrtf(3.14159265358979f / 2.f) : 1.f);
  const bool wild = (least < most && exponent(most) - exponent(least + 1u) > kWildLog2) ||
                    longest * key * ta.scale * 1.4426950408889634f > kWildScore;
  const float unit_scale = scale_of(exponent(most));
  if (tid == 0 && blockIdx.y == 0) reinterpret_cast<float*>(ws + pl.ws_scale)[unit] = wild ? 0.f : unit_scale;
  uint8_t* table = ws + pl.ws_q + (long)unit * pl.q_bytes;
  const int blk = pl.rows * 128, part = pl.rows * D * 2;
#pragma unroll 1
  for (int rr = 32 * blockIdx.y + warp; rr < pl.rows; rr += 32 * gridDim.y) {
    float u[E];
    if (rr < rows) {
      load(rr, u);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = 0.f;
    }
    float scale = unit_scale;
    if (wild) {
      scale = scale_of(exponent(size(u)));
      if (lane == 0) reinterpret_cast<float*>(ws + pl.ws_rows)[(long)unit * pl.rows + rr] = score_factor(tb, ta.scale) / scale;
    }
    auto signs = [&](const uint32_t* s, float by) {
      const uint32_t w = s[c0 >> 5] >> (c0 & 31);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] *= (w >> e) & 1u ? -by : by;
    };
    signs(tb.s1, scale);
    warp_fwht<E>(u, lane);
    uint8_t* dst = table + (c0 >> 6) * blk + rr * 128 + ((((c0 >> 3) & 7) ^ (rr & 7)) << 4) + (c0 & 7) * 2;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      uint32_t hi, lo;
      split_pair(u[2 * e], u[2 * e + 1], hi, lo);
      reinterpret_cast<uint32_t*>(dst)[e] = hi;
      if (ta.dtype == kF16) reinterpret_cast<uint32_t*>(dst + part)[e] = lo;
    }
    if (tb.qjl) {
      // channels j and j + 16 of a 32-channel word are neighbours in the reduction
      signs(tb.s2, 1.f / sqrtf((float)D));
      warp_fwht<E>(u, lane);
      uint8_t* row = table + (pl.parts - 1) * part + rr * 128;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = c0 + e, j = c & 31, pos = (c & ~31) + (j < 16 ? 2 * j : 2 * (j - 16) + 1);
        *reinterpret_cast<uint16_t*>(row + (pos >> 6) * blk + ((((pos >> 3) & 7) ^ (rr & 7)) << 4) + (pos & 7) * 2) =
            __half_as_ushort(__float2half_rn(u[e]));
      }
    }
  }
}

constexpr int kMergeWarps = 4;
constexpr int kMergeMax = kTreeMaxCtas;  // partials of one row

// Merges the partials of one (batch row, draft, query head), in a fixed order,
// and rotates back.  The partition is worked out again from the lengths.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                      const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl,
                      const uint8_t* __restrict__ ws) {
  constexpr int E = D / 32, NT = 32 * kMergeWarps;
  __shared__ float wgt[kMergeMax];
  __shared__ float part[kMergeWarps][D];
  __shared__ float red[kMergeWarps];
  __shared__ long long tiles[2][kMergeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int i = blockIdx.x / ta.q_heads, h = blockIdx.x - i * ta.q_heads, H = cv.kv_heads, group = ta.q_heads / H;
  const int kvh = h / group, r = i * group + (h - kvh * group), rb = r / pl.rows, col = r - rb * pl.rows;
  const int units = H * pl.blocks, nctas = pl.ctas;
  long long before = 0, all = 0;
  for (int k = tid; k < cv.batch; k += NT) {
    const long long x = tree_span(cv, k, ta.n_q, ta.max_ctx);
    all += x;
    before += k < b ? x : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    tiles[0][warp] = all;
    tiles[1][warp] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    all += tiles[0][w];
    before += tiles[1][w];
  }
  const int n = tree_span(cv, b, ta.n_q, ta.max_ctx);
  const long out_at = (((long)b * ta.n_q + i) * ta.q_heads + h) * D;
  // the unit's tiles are [su, eu) of the T places
  const long long T = all * units, unit = (long long)kvh * pl.blocks + rb, eu = before * units + (unit + 1) * n,
                  su = eu - max(n - kUnitCost, 0);
  const int c_lo = n > 0 ? (int)(((su + 1) * nctas + T - 1) / T - 1) : 0;
  const int c_hi = n > 0 ? (int)((eu * nctas + T - 1) / T - 1) : -1;
  const int S = c_hi - c_lo + 1;
  const long slot0 = c_lo + (long)b * units + unit;
  pdl_wait();
  float m = kNoMax;
  for (int s = tid; s < S; s += NT) {
    const long long c = c_lo + s, f0 = tile_bound(c, T, nctas), f1 = tile_bound(c + 1, T, nctas);
    float ms = -INFINITY;
    if (max(f0, su) < min(f1, eu)) {  // a block with an empty range left no partial
      const float2 x = reinterpret_cast<const float2*>(ws + pl.ws_ml)[(slot0 + s) * pl.rows + col];
      if (x.y != 0.f) ms = x.x;
    }
    wgt[s] = ms;
    m = fmaxf(m, ms);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float o[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int s = warp; s < S; s += kMergeWarps) {
    const float ms = wgt[s];
    if (ms == -INFINITY) continue;
    const float x = fast_exp2(ms - m);
    const long at = (slot0 + s) * pl.rows + col;
    float v[E];
    if constexpr (E == 2) {
      const float2 y = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(ws) + at * D + lane * E);
      v[0] = y.x;
      v[1] = y.y;
    } else {
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        const float4 y = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ws) + at * D + lane * E)[e];
        v[4 * e] = y.x;
        v[4 * e + 1] = y.y;
        v[4 * e + 2] = y.z;
        v[4 * e + 3] = y.w;
      }
    }
    l = fmaf(reinterpret_cast<const float2*>(ws + pl.ws_ml)[at].y, x, l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(v[e], x, o[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = o[e];
  __syncthreads();  // every warp has read red
  if (lane == 0) red[warp] = l;
  __syncthreads();
  pdl_trigger();
  if (warp != 0) return;
  l = (red[0] + red[1]) + (red[2] + red[3]);
  const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing attended: zeros
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane * E + e;
    o[e] = ((part[0][c] + part[1][c]) + (part[2][c] + part[3][c])) * inv;
  }
  if (!tb.affine) {
    warp_fwht<E>(o, lane);
    const float f = 1.f / ((float)D * tb.v_lam);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane * E + e;
      o[e] *= ((tb.s1[c >> 5] >> (c & 31)) & 1u) ? -f : f;
    }
  }
  uint32_t y[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    if (ta.dtype == kBF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
      y[e] = *reinterpret_cast<const uint32_t*>(&x);
    } else {
      const __half2 x = __floats2half2_rn(o[2 * e], o[2 * e + 1]);
      y[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(ta.out) + out_at) + lane * (E / 2);
  if constexpr (E == 2) dst[0] = y[0];
  else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
}

}  // namespace

size_t tree_workspace_bytes(const Tables& tb, int batch, int q_heads, int kv_heads, int n_q, int max_ctx) {
  TreePlan a, b;  // of either type, so that the size does not depend on it
  if (!plan_tree(tb, kBF16, batch, q_heads, kv_heads, n_q, max_ctx, &a) ||
      !plan_tree(tb, kF16, batch, q_heads, kv_heads, n_q, max_ctx, &b))
    return 0;
  return std::max(plan_bytes(a), plan_bytes(b));
}

namespace {

template <int D>
cudaError_t launch_dim(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  // shares of 32 rows, until there is a block for each SM
  const long units = pl.slots - pl.ctas;
  if (units > 0x7fffffffL || (long)ta.n_q * ta.q_heads > 0x7fffffffL) return cudaErrorInvalidConfiguration;
  auto tree = [&](cudaLaunchConfig_t* c) {
    return tb.affine ? (tb.qjl ? launch_tree_dim<D, true, true>(tb, cv, ta, pl, ws, c)
                               : launch_tree_dim<D, true, false>(tb, cv, ta, pl, ws, c))
                     : (tb.qjl ? launch_tree_dim<D, false, true>(tb, cv, ta, pl, ws, c)
                               : launch_tree_dim<D, false, false>(tb, cv, ta, pl, ws, c));
  };
  cudaError_t e = tree(nullptr);  // nothing is launched unless all can be
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)units, (unsigned)std::max(1L, std::min((pl.rows + 31) / 32L, kTreeMaxCtas / units)));
  cfg.blockDim = dim3(kPrepThreads);
  e = cudaLaunchKernelEx(&cfg, tree_query_kernel<D>, tb, cv, ta, pl, ws);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(pl.ctas);
  cfg.dynamicSmemBytes = pl.smem;
  e = tree(&cfg);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(ta.n_q * ta.q_heads), (unsigned)cv.batch);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, tb, cv, ta, pl, (const uint8_t*)ws);
}

}  // namespace

cudaError_t launch_tree(const Tables& tb, const CacheView& cv, const TreeArgs& ta, float* workspace,
                        cudaStream_t stream) {
  TreePlan pl;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  if (!plan_tree(tb, ta.dtype, cv.batch, ta.q_heads, cv.kv_heads, ta.n_q, ta.max_ctx, &pl)) return cudaErrorNotSupported;
  switch (tb.d) {
    case 64: return launch_dim<64>(tb, cv, ta, pl, ws, stream);
    case 128: return launch_dim<128>(tb, cv, ta, pl, ws, stream);
    case 256: return launch_dim<256>(tb, cv, ta, pl, ws, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace tq
