// Attention of drafted tokens over the packed cache: out_i = R^T sum_t p_t v_t,
// p the softmax of scale * <R q_i, k_t> over the context and the drafts that the
// mask lets draft i see.  Simplest form: one warp per (batch row, draft, query
// head); a lane scores one of 32 tokens, then holds d/32 channels of the sum.
#include "tq_decode_impl.cuh"

namespace tq {
namespace {

constexpr int kTreeWarps = 4;

__device__ __forceinline__ int code_at(const uint8_t* row, int bits, int i) {
  const int bit = bits * i, by = bit >> 3;
  const uint32_t w = row[by] | (((bit & 7) + bits > 8 ? (uint32_t)row[by + 1] : 0u) << 8);
  return (int)((w >> (bit & 7)) & ((1u << bits) - 1u));
}

template <int D>
__global__ void __launch_bounds__(32 * kTreeWarps)
    tree_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                const __grid_constant__ TreeArgs ta) {
  constexpr int E = D / 32;
  __shared__ float s_q[kTreeWarps][2][D];
  __shared__ float s_cent[2][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  if (tid < 16) {
    s_cent[0][tid] = tb.k_cent[tid];
    s_cent[1][tid] = tb.v_cent[tid];
  }
  pdl_wait();
  const int row = blockIdx.x * kTreeWarps + warp;  // draft * q_heads + head
  const int i = row / ta.q_heads, h = row % ta.q_heads;
  const int stored = min(max(cv.seq_lens[b], 0), cv.capacity);
  if (tid == 0 && blockIdx.x == 0 && stored > ta.max_ctx) atomicOr(cv.status, (int)kFlagMaxCtx);
  const bool live = i < ta.n_q;
  const long at = (((long)b * ta.n_q + i) * ta.q_heads + h) * D;
  const float root = sqrtf((float)D);
  if (live) {
    float u[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = lane * E + e;
      const float x = load_any(ta.q, at + ch, ta.dtype);
      u[e] = ((tb.s1[ch >> 5] >> (ch & 31)) & 1u) ? -x : x;
    }
    warp_fwht<E>(u, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = lane * E + e;
      s_q[warp][0][ch] = u[e] / root;
      u[e] = ((tb.s2[ch >> 5] >> (ch & 31)) & 1u) ? -u[e] / root : u[e] / root;
    }
    warp_fwht<E>(u, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) s_q[warp][1][lane * E + e] = u[e] / root;
  }
  __syncthreads();
  if (!live) return;
  const int ctx = stored - ta.n_q, len = ctx < 0 ? 0 : min(stored, ta.max_ctx);
  const int words = (ta.n_q + 31) / 32;
  const uint32_t* mask = ta.mask ? ta.mask + b * ta.mask_stride + (long)i * words : nullptr;
  const int kvh = h / (ta.q_heads / cv.kv_heads);
  const long slot0 = ((long)b * cv.kv_heads + kvh) * cv.capacity;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int t0 = 0; t0 < len; t0 += 32) {
    const int t = t0 + lane, j = t - ctx;
    bool sees = t < len;
    if (sees && j >= 0) sees = mask ? (mask[j >> 5] >> (j & 31)) & 1u : j <= i;
    float s = -INFINITY;
    if (sees) {
      const long slot = slot0 + t;
      const uint8_t* codes = cv.k_codes + slot * (tb.k_bits * D / 8);
      float dot = 0.f;
      if (tb.affine) {
        const __half* meta = reinterpret_cast<const __half*>(cv.k_norm) + slot * (2 * D / kAffineGroup);
        for (int c = 0; c < D; ++c) {
          const __half* p = meta + 2 * (c / kAffineGroup);
          dot = fmaf(s_q[warp][0][c], fmaf(__half2float(p[0]), (float)code_at(codes, tb.k_bits, c), __half2float(p[1])), dot);
        }
      } else {
        for (int c = 0; c < D; ++c) dot = fmaf(s_q[warp][0][c], s_cent[0][code_at(codes, tb.k_bits, c)], dot);
        dot *= __half2float(__ushort_as_half(cv.k_norm[slot])) / root;
      }
      if (tb.qjl) {
        const uint8_t* sg = cv.k_signs + slot * (D / 8);
        float x = 0.f;
        for (int c = 0; c < D; ++c) x += (sg[c >> 3] >> (c & 7)) & 1 ? s_q[warp][1][c] : -s_q[warp][1][c];
        dot = fmaf(sqrtf(3.14159265358979f / (2.0f * D)) * __half2float(__ushort_as_half(cv.k_rnorm[slot])), x, dot);
      }
      s = dot * ta.scale;
    }
    float mx = s;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const unsigned seen = __ballot_sync(0xffffffffu, sees);
    if (seen == 0) continue;
    const float mn = fmaxf(m, mx), alpha = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = sees ? expf(s - mn) : 0.f;
    m = mn;
    l = l * alpha;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
    for (int k = 0; k < 32; ++k) {
      if (!((seen >> k) & 1u)) continue;
      const float pk = __shfl_sync(0xffffffffu, p, k);
      l += pk;
      const long slot = slot0 + t0 + k;
      const uint8_t* codes = cv.v_codes + slot * (tb.v_bits * D / 8);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int ch = lane * E + e, c = code_at(codes, tb.v_bits, ch);
        float v;
        if (tb.affine) {
          const __half* q = reinterpret_cast<const __half*>(cv.v_norm) + slot * (2 * D / kAffineGroup) + 2 * (ch / kAffineGroup);
          v = fmaf(__half2float(q[0]), (float)c, __half2float(q[1]));
        } else {
          v = s_cent[1][c] * __half2float(__ushort_as_half(cv.v_norm[slot])) / root;
        }
        o[e] = fmaf(pk, v, o[e]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= inv;
  if (!tb.affine) {
    warp_fwht<E>(o, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = lane * E + e;
      o[e] = (((tb.s1[ch >> 5] >> (ch & 31)) & 1u) ? -o[e] : o[e]) / root;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (ta.dtype == kBF16) static_cast<__nv_bfloat16*>(ta.out)[at + lane * E + e] = __float2bfloat16_rn(o[e]);
    else static_cast<__half*>(ta.out)[at + lane * E + e] = __float2half_rn(o[e]);
  }
  pdl_trigger();
}

}  // namespace

size_t tree_workspace_bytes(int batch, int q_heads, int kv_heads, int n_q, int max_ctx, int head_dim) {
  (void)batch; (void)q_heads; (void)kv_heads; (void)n_q; (void)max_ctx; (void)head_dim;
  return 0;
}

cudaError_t launch_tree(const Tables& tb, const CacheView& cv, const TreeArgs& ta, float* workspace,
                        cudaStream_t stream) {
  (void)workspace;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((ta.n_q * ta.q_heads + kTreeWarps - 1) / kTreeWarps), (unsigned)cv.batch);
  cfg.blockDim = dim3(32 * kTreeWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (tb.d) {
    case 64: return cudaLaunchKernelEx(&cfg, tree_kernel<64>, tb, cv, ta);
    case 128: return cudaLaunchKernelEx(&cfg, tree_kernel<128>, tb, cv, ta);
    case 256: return cudaLaunchKernelEx(&cfg, tree_kernel<256>, tb, cv, ta);
  }
  return cudaErrorNotSupported;
}

}  // namespace tq
