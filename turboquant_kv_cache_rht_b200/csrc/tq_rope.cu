// Rotary positions fused with quantize-and-append.
//
// Pair i of a head's first rot_dim channels, (a, b), becomes
//   (a cos - b sin, b cos + a sin),  cos and sin of position * f_i
// read from a table of the program's (every product and sum rounded to fp32 on
// its own, so codes are reproducible bit for bit).  Keys go on to the codec of
// tq_codec.cuh without being rounded in between, values go there as they are,
// queries are written out.  A separate rotation would write and re-read the
// keys and cost a launch; here a decode step's queries, keys and values are one
// grid.
#include "tq_codec.cuh"

#include <algorithm>

namespace tq {
namespace {

using namespace codec;

constexpr int kRopeThreads = 256;

__global__ void __launch_bounds__(256)
    rope_table_kernel(const __grid_constant__ RopeFrequencies rf, int pairs, long entries, float2* table) {
  pdl_wait();
  const long e = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (e < entries) {
    double s, c;
    sincos((double)(e / pairs) * rf.freq[e % pairs], &s, &c);
    table[e] = make_float2((float)(c * rf.factor), (float)(s * rf.factor));
  }
  pdl_trigger();
}

template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
  if constexpr (sizeof(T) == 4) return __ldg(p);
  else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(*p);
  else return __half2float(*p);
}

template <typename T>
__device__ __forceinline__ T round_to(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}

// E consecutive elements, rounded to T, as 16-, 8- or 4-byte words.
template <int E, typename T>
__device__ __forceinline__ void store_elems(T* p, const float (&x)[E]) {
  constexpr int NB = E * (int)sizeof(T), NW = NB / 4, PW = 4 / (int)sizeof(T);
  uint32_t w[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    T t[PW];
#pragma unroll
    for (int j = 0; j < PW; ++j) t[j] = round_to<T>(x[PW * i + j]);
    memcpy(&w[i], t, 4);
  }
  if constexpr (NB % 16 == 0) {
#pragma unroll
    for (int i = 0; i < NB / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else if constexpr (NB == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    static_assert(NB == 4, "4, 8 or a multiple of 16 bytes per lane");
    *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// Rotates the lane's channels c0 .. c0 + E - 1 of the vector at `vec` (held in
// x) by the table row `cs`.  Pairs half a rotation apart lie in another lane:
// the partner channels are read again (from L1), as one block where rot_dim
// keeps the lanes' blocks aligned.
template <int E, typename T>
__device__ __forceinline__ void rotate(float (&x)[E], const T* vec, const float2* __restrict__ cs, int c0,
                                       int rot, bool interleaved) {
  if (c0 >= rot) return;
  if (interleaved) {
    if constexpr (E >= 4) {
      if (c0 + E <= rot && (rot & 3) == 0) {  // whole block, 16-byte aligned entries: two at a time
        const float4* t4 = reinterpret_cast<const float4*>(cs + c0 / 2);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 t = __ldg(t4 + e / 4);
          const float a = x[e], b = x[e + 1], c = x[e + 2], d = x[e + 3];
          x[e] = __fsub_rn(__fmul_rn(a, t.x), __fmul_rn(b, t.y));
          x[e + 1] = __fadd_rn(__fmul_rn(b, t.x), __fmul_rn(a, t.y));
          x[e + 2] = __fsub_rn(__fmul_rn(c, t.z), __fmul_rn(d, t.w));
          x[e + 3] = __fadd_rn(__fmul_rn(d, t.z), __fmul_rn(c, t.w));
        }
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < E; e += 2)
      if (c0 + e < rot) {
        const float2 t = __ldg(cs + (c0 + e) / 2);
        const float a = x[e], b = x[e + 1];
        x[e] = __fsub_rn(__fmul_rn(a, t.x), __fmul_rn(b, t.y));
        x[e + 1] = __fadd_rn(__fmul_rn(b, t.x), __fmul_rn(a, t.y));
      }
    return;
  }
  const int half = rot >> 1;
  if (half % E == 0) {
    const bool first = c0 < half;
    const float2* t = cs + (first ? c0 : c0 - half);
    float p[E];
    load_elems<E>(vec + (first ? c0 + half : c0 - half), p);
#pragma unroll
    for (int e = 0; e < E; e += 2) {  // (half is even here, so pairs of entries are 16-byte aligned)
      const float4 f = __ldg(reinterpret_cast<const float4*>(t + e));
      const float own0 = __fmul_rn(x[e], f.x), other0 = __fmul_rn(p[e], f.y);
      const float own1 = __fmul_rn(x[e + 1], f.z), other1 = __fmul_rn(p[e + 1], f.w);
      x[e] = first ? __fsub_rn(own0, other0) : __fadd_rn(own0, other0);
      x[e + 1] = first ? __fsub_rn(own1, other1) : __fadd_rn(own1, other1);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = c0 + e;
      if (c < rot) {
        const bool first = c < half;
        const float2 f = __ldg(cs + (first ? c : c - half));
        const float own = __fmul_rn(x[e], f.x);
        const float other = __fmul_rn(load_one(vec + (first ? c + half : c - half)), f.y);
        x[e] = first ? __fsub_rn(own, other) : __fadd_rn(own, other);
      }
    }
  }
}

// What a grid encodes: bits of `kinds` and, per kind, its blocks, in the order
// keys, values, queries.
constexpr int kKeys = 1, kValues = 2, kQueries = 4;

// Grid: (blocks of the kinds present, batch).  A group of D / E lanes takes one
// vector.  `publish`: the last block of a row to finish sets its length.
template <int D, typename T, int E, bool AFF, int KINDS, int BITS, bool BULK>
__global__ void __launch_bounds__(kRopeThreads)
    rope_append_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                       const __grid_constant__ RopeAppend ra, int kv_blocks, int publish) {
  constexpr int GL = D / E, VPB = kRopeThreads / GL;
  __shared__ float s_kcent[16];
  const int tid = threadIdx.x, lane = tid & 31, g = lane & (GL - 1);
  if (tid < 16) s_kcent[tid] = tb.k_cent[tid];
  const int b = blockIdx.y;
  int kind = KINDS, block = blockIdx.x;
  if constexpr ((KINDS & (KINDS - 1)) != 0) {
    kind = block < kv_blocks ? kKeys : block < 2 * kv_blocks ? kValues : kQueries;
    block -= kind == kKeys ? 0 : kind == kValues ? kv_blocks : 2 * kv_blocks;
  }
  const Heads& in = kind == kKeys ? ra.k : kind == kValues ? ra.v : ra.q;
  const int heads = kind == kQueries ? ra.q_heads : cv.kv_heads;
  const long r = (long)block * VPB + tid / GL;
  const bool valid = r < (long)heads * ra.n_new;
  // consecutive lanes read consecutive memory whichever of heads and tokens is inner
  const bool inner = in.sh < in.st;
  const int h = !valid ? 0 : inner ? (int)(r % heads) : (int)(r / ra.n_new);
  const int j = !valid ? 0 : inner ? (int)(r / heads) : (int)(r % ra.n_new);

  pdl_wait();
  if constexpr (!BULK) pdl_trigger();  // this grid is resident at once: the next may set up
  const int stored = cv.seq_lens[b];
  const int base = ra.start ? ra.start[b] : stored;
  const bool in_row = base >= 0 && base <= stored;
  const bool fits = in_row && base <= cv.capacity - ra.n_new;
  if (!fits && tid == 0 && blockIdx.x == 0) atomicOr(cv.status, (int)(in_row ? kFlagCapacity : kFlagIndex));
  __syncthreads();  // s_kcent

  const bool writes = kind == kQueries || (kind == kKeys && ra.k_out != nullptr);
  if ((fits || writes) && __any_sync(kFull, valid)) {
    const T* vec = static_cast<const T*>(in.data) + b * in.sb + h * in.sh + j * in.st;
    float u[E];
    if (valid) {
      load_elems<E>(vec + g * E, u);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = 0.f;
    }
    if ((KINDS & (kKeys | kQueries)) != 0 && kind != kValues && valid) {
      long pos = ra.positions ? ra.positions[(long)b * ra.n_new + j] : j;
      if (!ra.positions || ra.relative) pos += base;
      const long at = min(max(pos, 0l), (long)ra.max_pos - 1);
      if (at != pos && g == 0) atomicOr(cv.status, (int)kFlagIndex);
      const int half = ra.rot_dim >> 1;
      rotate<E>(u, vec, reinterpret_cast<const float2*>(ra.table) + at * half, g * E, ra.rot_dim,
                ra.interleaved != 0);
      if (writes) {
        T* out = static_cast<T*>(kind == kQueries ? ra.q_out : ra.k_out);
        store_elems<E>(out + (((long)b * ra.n_new + j) * heads + h) * D + g * E, u);
      }
    }
    if constexpr ((KINDS & (kKeys | kValues)) != 0) {
      if (fits && kind != kQueries) {
        const bool is_v = kind == kValues;
        const long slot = ((long)b * cv.kv_heads + h) * cv.capacity + base + j;
        const int bits = is_v ? tb.v_bits : tb.k_bits;
        uint8_t* codes = (is_v ? cv.v_codes : cv.k_codes) + slot * (long)(bits * D / 8);
        constexpr int NH = AFF ? 2 * D / kAffineGroup : 1;
        uint16_t* norm = (is_v ? cv.v_norm : cv.k_norm) + slot * NH;
        uint8_t* signs = (!is_v && tb.qjl) ? cv.k_signs + slot * (long)(D / 8) : nullptr;
        uint16_t* rnorm = (!is_v && tb.qjl) ? cv.k_rnorm + slot : nullptr;
        encode_vector<D, E, AFF, BITS>(bits, u, tb, is_v, g, lane, valid, codes, norm, signs, rnorm, s_kcent);
      }
    }
  }
  if (publish) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const int ticket = atomicAdd(&cv.append_sync[b], 1);
      if (ticket == (int)gridDim.x - 1) {
        if (fits) cv.seq_lens[b] = base + ra.n_new;
        cv.append_sync[b] = 0;
      }
    }
  }
  if constexpr (BULK) pdl_trigger();
}

// Bulk queries, rot_dim a multiple of 16: a thread turns 8 pairs, both channels of
// each, for every hs-th head of a token, so that a table entry is read once for all of
// them: 8192 tokens of 32 heads in 29 us (4.6 TB/s), 55 us with one read per channel
// and head.  Lanes past the rotated channels copy 16 channels.  Grid: (blocks of
// tokens, batch).
template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads)
    rope_query_kernel(const __grid_constant__ CacheView cv, const __grid_constant__ RopeAppend ra, int hs) {
  constexpr int GL = D / 16, SLOTS = kRopeThreads / GL;
  const int g = threadIdx.x % GL, slot = threadIdx.x / GL, b = blockIdx.y;
  const int j = blockIdx.x * (SLOTS / hs) + slot / hs;
  pdl_wait();
  const int base = ra.start ? ra.start[b] : cv.seq_lens[b];
  if (j < ra.n_new) {
    const int half = ra.rot_dim >> 1;
    const bool turns = 8 * g < half;
    // channels of the thread's first and second eight
    const int c0 = !turns ? ra.rot_dim + 16 * (g - half / 8) : ra.interleaved ? 16 * g : 8 * g;
    const int c1 = turns && !ra.interleaved ? c0 + half : c0 + 8;
    float4 t[4];
    if (turns) {
      long pos = ra.positions ? ra.positions[(long)b * ra.n_new + j] : j;
      if (!ra.positions || ra.relative) pos += base;
      const long at = min(max(pos, 0l), (long)ra.max_pos - 1);
      if (at != pos && g == 0) atomicOr(cv.status, (int)kFlagIndex);
      const float4* cs = reinterpret_cast<const float4*>(reinterpret_cast<const float2*>(ra.table) + at * half + 8 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = __ldg(cs + i);
    }
    const T* src = static_cast<const T*>(ra.q.data) + b * ra.q.sb + j * ra.q.st;
    T* dst = static_cast<T*>(ra.q_out) + ((long)b * ra.n_new + j) * ra.q_heads * D;
#pragma unroll 4
    for (int h = slot % hs; h < ra.q_heads; h += hs) {
      float x[8], y[8];
      load_elems<8>(src + h * ra.q.sh + c0, x);
      load_elems<8>(src + h * ra.q.sh + c1, y);
      if (turns) {
        auto turn = [](float& a, float& b, float c, float s) {
          const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
          b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
          a = u;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (ra.interleaved) {
            float(&z)[8] = i < 2 ? x : y;
            turn(z[4 * (i & 1)], z[4 * (i & 1) + 1], t[i].x, t[i].y);
            turn(z[4 * (i & 1) + 2], z[4 * (i & 1) + 3], t[i].z, t[i].w);
          } else {
            turn(x[2 * i], y[2 * i], t[i].x, t[i].y);
            turn(x[2 * i + 1], y[2 * i + 1], t[i].z, t[i].w);
          }
        }
      }
      store_elems<8>(dst + h * D + c0, x);
      store_elems<8>(dst + h * D + c1, y);
    }
  }
  pdl_trigger();
}

// At most this many vectors in all take the layout of one vector per warp, as
// the append does: too few to fill the GPU, so latency rules.
constexpr long kRopeLatencyVectors = 4096;

template <typename Kernel>
cudaError_t launch(Kernel kern, long blocks, int batch, cudaStream_t stream, const Tables& tb,
                   const CacheView& cv, const RopeAppend& ra, long kv_blocks, int publish) {
  if (blocks > 0x7fffffffL || batch > 65535) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)batch);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tb, cv, ra, (int)kv_blocks, publish);
}

template <int D, typename T, bool AFF>
cudaError_t launch_typed(const Tables& tb, const CacheView& cv, const RopeAppend& ra, cudaStream_t stream) {
  auto blocks = [&](int lanes, int heads) {
    const int vpb = kRopeThreads / lanes;
    return ((long)heads * ra.n_new + vpb - 1) / vpb;
  };
  const long vectors = (long)cv.batch * ra.n_new * (2L * cv.kv_heads + ra.q_heads);
  if (vectors <= kRopeLatencyVectors) {
    constexpr int E = D / 32;
    const long kvb = blocks(32, cv.kv_heads), qb = ra.q.data ? blocks(32, ra.q_heads) : 0;
    return launch(rope_append_kernel<D, T, E, AFF, kKeys | kValues | kQueries, 0, false>, 2 * kvb + qb,
                  cv.batch, stream, tb, cv, ra, kvb, 1);
  }
  // bulk: a grid per kind, each of one code width (its unrolled encoder stays in
  // the instruction cache); the last one publishes the lengths
  cudaError_t e = cudaSuccess;
  if (ra.q.data && ra.rot_dim % 16 == 0) {
    const int hs = ra.q_heads >= 8 ? 8 : ra.q_heads >= 4 ? 4 : ra.q_heads >= 2 ? 2 : 1;
    const int tokens = kRopeThreads / (D / 16) / hs;
    const long nb = ((long)ra.n_new + tokens - 1) / tokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nb, (unsigned)cv.batch);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, rope_query_kernel<D, T>, cv, ra, hs);
    if (e != cudaSuccess) return e;
  } else if (ra.q.data) {
    constexpr int E = 8;
    e = launch(rope_append_kernel<D, T, E, false, kQueries, 2, true>, blocks(D / E, ra.q_heads), cv.batch,
               stream, tb, cv, ra, 0, 0);
    if (e != cudaSuccess) return e;
  }
  constexpr int E = 32;
  const long kvb = blocks(D / E, cv.kv_heads);
  auto keys = tb.k_bits == 2   ? rope_append_kernel<D, T, E, AFF, kKeys, 2, true>
              : tb.k_bits == 3 ? rope_append_kernel<D, T, E, AFF, kKeys, 3, true>
                               : rope_append_kernel<D, T, E, AFF, kKeys, 4, true>;
  e = launch(keys, kvb, cv.batch, stream, tb, cv, ra, 0, 0);
  if (e != cudaSuccess) return e;
  auto values = tb.v_bits == 2   ? rope_append_kernel<D, T, E, AFF, kValues, 2, true>
                : tb.v_bits == 3 ? rope_append_kernel<D, T, E, AFF, kValues, 3, true>
                                 : rope_append_kernel<D, T, E, AFF, kValues, 4, true>;
  return launch(values, kvb, cv.batch, stream, tb, cv, ra, 0, 1);
}

template <int D, typename T>
cudaError_t launch_codec(const Tables& tb, const CacheView& cv, const RopeAppend& ra, cudaStream_t stream) {
  return tb.affine ? launch_typed<D, T, true>(tb, cv, ra, stream) : launch_typed<D, T, false>(tb, cv, ra, stream);
}

template <int D>
cudaError_t launch_dim(const Tables& tb, const CacheView& cv, const RopeAppend& ra, int dtype,
                       cudaStream_t stream) {
  switch (dtype) {
    case kF32: return launch_codec<D, float>(tb, cv, ra, stream);
    case kBF16: return launch_codec<D, __nv_bfloat16>(tb, cv, ra, stream);
    case kF16: return launch_codec<D, __half>(tb, cv, ra, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_append(const Tables& tb, const CacheView& cv, const RopeAppend& ra, int dtype,
                               cudaStream_t stream) {
  switch (tb.d) {
    case 64: return launch_dim<64>(tb, cv, ra, dtype, stream);
    case 128: return launch_dim<128>(tb, cv, ra, dtype, stream);
    case 256: return launch_dim<256>(tb, cv, ra, dtype, stream);
  }
  return cudaErrorNotSupported;
}

cudaError_t launch_rope_table(const RopeFrequencies& rf, int pairs, int max_pos, float* table,
                              cudaStream_t stream) {
  const long entries = (long)max_pos * pairs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((entries + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, rf, pairs, entries, reinterpret_cast<float2*>(table));
}

}  // namespace tq
