// Attention of drafted tokens over the packed cache.
//
//   out_i = R^T sum_t p_it v_t,   p_i = softmax over t of scale <R q_i, k_t>
//
// over the tokens t of the row's context and the drafts that the mask lets draft
// i attend.  The R = n_q * (q_heads / kv_heads) query rows of a KV head share its
// packed keys and values, so the work is two matrix products per tile of 128
// tokens with the softmax between them, both on the tensor cores:
//   S [token][row]    = K_hat [token][ch] . Q^T [ch][row]
//   O^T [ch][row]    += V_hat^T [ch][token] . P [token][row]
// Tokens (then channels) are the instruction's 128 rows, so a tile fills it
// whatever the number of drafts; the query rows are its columns, 16 to 256.
//
// One block per SM, split by role:
//   warps 0-7   two softmax warpgroups.  Each takes the score columns of its own
//               chunks (or every other tile, when one chunk holds all rows),
//               keeps their maxima and sums and writes P to shared memory;
//   warps 8-15  keys: a thread unpacks half of a token's codes through a table of
//               code pairs into the token's lane of tensor memory, the product's A
//               operand (no shared-memory round trip, no swizzle);
//   warps 16-23 values: the same into shared memory, token rows of 64 channels;
//   warps 24, 25 issue the matrix instructions of scores and of outputs (one
//               thread's instructions would bound the kernel);
//   warp 26     works out the block's share, announces its segments to the others
//               and copies the packed tiles in, a few stages ahead;
//   warp 27     copies a segment's query table in.
// Twenty-eight warps in seven roles share the instruction caches, and what bounds this
// kernel first is fetching instructions: loops stay rolled where registers allow
// it, and nothing that runs once per segment is unrolled.
// A key's norm multiplies its scores, a value's norm its weights, both fp32, in
// the softmax; so the fp16 operands hold centroids (scaled by k_lam / v_lam, at
// which they are nearly exact) and lose nothing.  The sketch's signs follow the
// key's channels in the reduction, as +- rnorm / norm, against a second table of
// rotated queries; an fp16 call holds its queries in two fp16 parts (hi + lo).
// The affine codec's operands are scale * level + bias, rounded to fp16.
//
// The token tiles of all (batch row, KV head, block of query rows) units are laid
// end to end and each block takes an equal share, as in the decode; a unit that
// a block meets leaves a partial (O, maximum, sum) in the workspace.  A kernel
// before it rotates the queries and lays them out as the product's B operand, once
// for all blocks; a kernel after it merges the partials and rotates back.
#include "tq_decode_impl.cuh"
#include "tq_tmem.cuh"

#include <algorithm>
#include <vector>

namespace tq {
namespace {

constexpr int kTile = 128;          // tokens per tile: the matrix instruction's rows
constexpr int kTreeThreads = 896;   // 28 warps, 72 registers each at launch
constexpr int kTreeMaxCtas = 148;   // one block per SM; the workspace is sized for it
constexpr int kMetaSlots = 4;       // tiles whose norms are in flight
constexpr int kMaxStages = 4;
// Slack of the running maximum (log2): weights stay below 2^14, fp16 holds 2^16,
// and 2^-14 of the largest is still a normal number.  A key that resembles the
// query outscores the others by about 2^13 at head_dim 128, so that a slack of 8
// raised the maximum of some column in most tiles (4x the time of the softmax).
constexpr float kTreeLazyLog2 = 14.0f;
constexpr float kNoMax = -1e30f;    // running maximum before any score (finite: no inf - inf)

// Bytes of the tables: 2-bit codes four at a time (8 bytes, 16 copies), 3-bit
// pairs (32 copies), 4-bit pairs (16 copies: 32 would cost a stage).  A lane
// reads its own copy, so lookups meet in a bank at most twice.
constexpr int lut_bytes(int bits) { return bits == 2 ? 32768 : bits == 3 ? 8192 : 16384; }

// What the host settles about one call.
struct TreePlan {
  int cn, chunks;          // score columns per chunk, chunks (1: tiles alternate between the warpgroups)
  int rows, blocks;        // query rows per unit, blocks of them per KV head
  int cols;                // columns of a partial: rows, or 2 rows when tiles alternate
  int parts;               // query tables: 1, + 1 (fp16 low parts), + 1 (sketch)
  int nkb, nvb, nst;       // key, value and packed buffers
  int tm_k, tm_s, kcols;   // tensor memory columns: keys, scores; columns of one key buffer
  int lut_k, lut_v, sm_q, sm_v, sm_p, sm_st, sm_meta, sm_misc, smem;  // shared addresses
  int st_v, st_s, st_kn, st_vn, st_rn, st_bytes;                      // inside a stage
  int ctas, q_bytes;       // q_bytes: one unit's query table
  long slots, ws_ml, ws_q, ws_scale;  // workspace: bytes to the maxima and sums, query tables, their scales
};

// Shared misc area: barriers, segments, then floats.
constexpr int kSegs = 4;  // segments announced ahead
constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarStFull = 2, kBarStEmpty = kBarStFull + kMaxStages,
              kBarKFull = kBarStEmpty + kMaxStages, kBarKEmpty = kBarKFull + 2, kBarVFull = kBarKEmpty + 2,
              kBarVEmpty = kBarVFull + 2, kBarSFull = kBarVEmpty + 2, kBarSEmpty = kBarSFull + 2,
              kBarPFull = kBarSEmpty + 2, kBarPEmpty = kBarPFull + 2, kBarMetaFull = kBarPEmpty + 2,
              kBarMetaEmpty = kBarMetaFull + kMetaSlots, kBarSegFull = kBarMetaEmpty + kMetaSlots,
              kBarSegEmpty = kBarSegFull + kSegs, kBarDone = kBarSegEmpty + kSegs, kBars = kBarDone + 2;
constexpr int kSegReaders = 27;  // warps that read a segment
constexpr int kMiscTmem = kBars * 8, kMiscDead = kMiscTmem + 4,
              kMiscSeg = (kMiscTmem + 8 + 31) / 32 * 32,  // [kSegs][8] ints
              kMiscM = kMiscSeg + kSegs * 32,             // running maxima [256]
              kMiscAlpha = kMiscM + 1024,                 // rescale factors [4][32]
              kMiscRed = kMiscAlpha + 512,                // [4 warpgroups][4 warps][64]
              kMiscBytes = kMiscRed + 4096;

// Arrivals that complete barrier i's phase.
__device__ __forceinline__ int bar_count(int i, bool split, int softmax_warps, int unpack_warps) {
  if (i >= kBarStEmpty && i < kBarKFull) return 2 * unpack_warps;
  if ((i >= kBarKFull && i < kBarKEmpty) || (i >= kBarVFull && i < kBarVEmpty)) return unpack_warps;
  if ((i >= kBarSEmpty && i < kBarPFull) || (i >= kBarPFull && i < kBarPEmpty)) return softmax_warps / 2;
  if (i >= kBarMetaFull && i < kBarMetaEmpty) return 4;
  if (i >= kBarMetaEmpty && i < kBarSegFull) return split ? softmax_warps / 2 : softmax_warps;  // a tile's norms
  if (i >= kBarSegEmpty && i < kBarDone) return kSegReaders;
  return 1;
}

struct Segment {
  int b, unit, t0, tiles, len;  // row, unit of the row, first token, tiles (0: no more), tokens of the row
};

// Tokens of a row that a call attends: none if it holds fewer than n_q.
__device__ __forceinline__ int tree_len(const CacheView& cv, int b, int n_q, int max_ctx) {
  const int stored = min(max(cv.seq_lens[b], 0), cv.capacity);
  return stored < n_q ? 0 : min(stored, max_ctx);
}
__device__ __forceinline__ int tree_tiles(const CacheView& cv, int b, int n_q, int max_ctx) {
  return (tree_len(cv, b, n_q, max_ctx) + kTile - 1) / kTile;
}

// The next announced segment; false at the end or when a wait gave up.
__device__ __forceinline__ bool next_segment(uint32_t misc, uint32_t& n, Segment& s, bool& fail, volatile int* dead) {
  const uint32_t slot = n % kSegs;
  fail = !tm::mbar_wait(misc + 8 * (kBarSegFull + slot), (n / kSegs) & 1, dead) || fail;
  const uint4 x = tm::lds128(misc + kMiscSeg + 32 * slot);
  s = Segment{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)tm::lds32(misc + kMiscSeg + 32 * slot + 16)};
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tm::mbar_arrive(misc + 8 * (kBarSegEmpty + slot));
  ++n;
  return __all_sync(0xffffffffu, s.tiles > 0 && !fail);
}

// 32 channels of a packed row at shared address `row` -> 16 fp16 pairs.
template <int BITS>
__device__ __forceinline__ void unpack32(uint32_t row, uint32_t lut, uint32_t (&r)[16]) {
  if constexpr (BITS == 2) {
    const uint2 w = tm::lds64(row);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // a byte of four codes, entries 128 bytes apart
      const uint2 x = tm::lut64(bits_at(i < 4 ? w.x : w.y, 8 * (i & 3), 8, 7) | lut);
      r[2 * i] = x.x;
      r[2 * i + 1] = x.y;
    }
  } else if constexpr (BITS == 3) {
    const uint32_t w[3] = {tm::lds32(row), tm::lds32(row + 4), tm::lds32(row + 8)};
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = tm::lut32(field_scaled(w, 3, 6 * i, 6, 7) | lut);
  } else {
    const uint4 w = tm::lds128(row);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = i < 4 ? w.x : i < 8 ? w.y : i < 12 ? w.z : w.w;
      r[i] = tm::lut32(bits_at(x, 8 * (i & 3), 8, 6) | lut);
    }
  }
}

// f(block, pairs) for every 32 channels of a row, or of half of it.  The loop stays rolled: the
// roles share the instruction caches, and unrolled roles starved
// each other (two thirds of the stalls were for instructions).
template <int N, int BITS, typename F>
__device__ __forceinline__ void unpack_row(uint32_t row, uint32_t lut, int half, F f) {
#pragma unroll 1
  for (int c = half * N; c < (half + 1) * N; ++c) {
    uint32_t r[16];
    unpack32<BITS>(row + 4 * BITS * c, lut, r);
    f(c, r);
  }
}
template <int N, typename F>
__device__ __forceinline__ void unpack_row(int bits, uint32_t row, uint32_t lut, int half, F f) {
  if (bits == 2) unpack_row<N, 2>(row, lut, half, f);
  else if (bits == 3) unpack_row<N, 3>(row, lut, half, f);
  else unpack_row<N, 4>(row, lut, half, f);
}

// Fills a table with every lane's copy of every entry.
__device__ __forceinline__ void fill_lut(uint32_t lut, int bits, const float* cent, float lam) {
  const uint32_t mask = (1u << bits) - 1u;
  // 16-byte pieces: a quad's two pairs twice, or a pair four times
  const int shift = bits == 4 ? 2 : 3, pieces = (bits == 2 ? 256 : 1 << (2 * bits)) << shift;
#pragma unroll 1
  for (int i = threadIdx.x; i < pieces; i += kTreeThreads) {
    const uint32_t p = (uint32_t)i >> shift, q = bits == 2 ? p >> 4 : p;
    auto pair = [&](uint32_t c) {
      return pack_half2(__float2half_rn(cent[c & mask] * lam), __float2half_rn(cent[(c >> bits) & mask] * lam));
    };
    const uint32_t x = pair(p), y = pair(q);
    tm::sts128(lut + 16 * i, x, y, x, y);
  }
}

// ---- the softmax's parts ---------------------------------------------------
// A thread's scores: tokens g + 8 k (k < 4) of its warp's 32, columns 8 j + 2 q + c
// (j < NJ, c < 2), in register y_at(k, j) + c.
template <int NJ>
__device__ __forceinline__ constexpr int y_at(int k, int j) {
  return (k >> 1) * 4 * NJ + 4 * j + 2 * (k & 1);
}

// Which of them count, bit 8 j + 4 c + k: tokens of the row, drafts that the mask
// lets the column's draft attend, live columns.  Tokens of the context are like
// mask words of ones before the first.
template <int NJ>
__device__ __forceinline__ uint32_t visible(int tok, int len, int ctx, int row, int live_rows, int log_group,
                                            const uint32_t* mask, int words) {
  const int d0 = tok - ctx, idx = d0 >> 5;
  uint32_t in = 0;  // bit 8 k: token k is one of the row's
#pragma unroll
  for (int k = 0; k < 4; ++k) in |= (tok + 8 * k < len ? 1u : 0u) << (8 * k);
  uint32_t vis = 0;
#pragma unroll 1
  for (int n = 0; n < 2 * NJ; ++n) {
    const int r = row + 8 * (n >> 1) + (n & 1), i = r >> log_group;
    auto word = [&](int x) -> uint32_t {
      if (x < 0) return 0xffffffffu;
      if (mask) return x < words ? mask[i * words + x] : 0u;
      const int bits = i + 1 - 32 * x;  // of a chain
      return bits >= 32 ? 0xffffffffu : bits > 0 ? (1u << bits) - 1u : 0u;
    };
    const uint32_t f = r < live_rows ? __funnelshift_r(word(idx), word(idx + 1), d0 & 31) & in : 0u;
    const uint32_t four = (f & 1u) | ((f >> 7) & 2u) | ((f >> 14) & 4u) | ((f >> 21) & 8u);
    vis |= four << (4 * n);
  }
  return vis;
}

struct Raise {
  uint32_t t_s, t_o;                   // tensor memory: the scores, the outputs (lanes of this warp)
  uint32_t a_m, sm_al, sm_red, bar_p;  // maxima of this lane's columns; factors; scratch; the products' barrier
  uint32_t vis, parity;
  int wg, cols, blocks;                // blocks: 128-channel blocks of the output to rescale
};

// Raises the running maxima of NJ x 8 columns to the scores in tensor memory,
// leaves the factors 2^(old - new) in sm_al and scales the outputs by them.
// All four warps of the group call.  False: a wait gave up.
template <int NJ>
__device__ __forceinline__ bool raise_max(const Raise& a, const float (&kn)[4], const float (&ev)[4], volatile int* dead) {
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, qd = lane & 3;
  const bool ok = tm::mbar_wait(a.bar_p, a.parity, dead);  // the products so far are done
#pragma unroll 1
  for (int j2 = 0; j2 < NJ / 2; ++j2) {  // 16 columns at a time
    float y[16];
    tm::ld_16x256b(a.t_s + 16 * j2, y);
    tm::wait_ld(y);
    float v[4];  // columns 8 j + 2 q + c of the two j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = fmaf(y[y_at<2>(k, i >> 1) + (i & 1)], kn[k], ev[k]);
        if ((a.vis >> (16 * j2 + 4 * i + k)) & 1u) v[i] = fmaxf(v[i], x);
      }
    }
    // over the eight lanes of a column: halves of the columns change sides twice
    const bool up = (lane & 16) != 0, up2 = (lane & 8) != 0;
    float p = fmaxf(up ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16));
    float q = fmaxf(up ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16));
    p = fmaxf(up2 ? q : p, __shfl_xor_sync(0xffffffffu, up2 ? p : q, 8));
    p = fmaxf(p, __shfl_xor_sync(0xffffffffu, p, 4));
    if ((lane & 4) == 0) tm::stsf(a.sm_red + 256 * w + 4 * (16 * j2 + (up ? 8 : 0) + 2 * qd + (up2 ? 1 : 0)), p);
  }
  tm::bar_sync(1 + a.wg, 128);
  if (w == 0 && lane < 8 * NJ) {
    const uint32_t at = a.a_m + 4 * lane, red = a.sm_red + 4 * lane;
    const float old = tm::ldsf(at);
    const float mn = fmaxf(fmaxf(fmaxf(old, tm::ldsf(red)), tm::ldsf(red + 256)),
                           fmaxf(tm::ldsf(red + 512), tm::ldsf(red + 768)));
    tm::stsf(at, mn);
    tm::stsf(a.sm_al + 4 * lane, fast_exp2(old - mn));
  }
  tm::bar_sync(1 + a.wg, 128);
  if (a.blocks > 0) {
    tm::fence_after();
#pragma unroll 1
    for (int i = 0; i < a.blocks * (NJ / 2); ++i) {
      const int h = i % (NJ / 2);
      const uint32_t at = a.t_o + (i / (NJ / 2)) * a.cols + 16 * h;
      uint32_t o[16];
      tm::ld_32x32b(at, o);
      tm::wait_ld(o);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        o[e] = __float_as_uint(__uint_as_float(o[e]) * tm::ldsf(a.sm_al + 4 * (16 * h + e)));
      tm::st_32x32b(at, o);
    }
    tm::wait_st();
  }
  return ok;
}

// ---- queries: rotated, scaled by a power of two, rounded to fp16, in the layout
// of the product's B operand (128-byte rows of 64 channels, swizzled; blocks of
// `rows` rows; parts hi, lo of an fp16 call, sketch).  One block per unit; the scale
// is common to its rows: |u| <= d max|q| is brought to 2^14, or 2^10 before the
// second rotation, which can add sqrt(d).  Rows that are not finite do not count.
constexpr int kPrepThreads = 1024;

template <int D>
__global__ void __launch_bounds__(kPrepThreads)
    tree_query_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                      const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl, uint8_t* __restrict__ ws) {
  constexpr int E = D / 32;
  __shared__ float red[32];
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
  float amax = 0.f;
#pragma unroll 4
  for (int rr = warp; rr < rows; rr += 32) {
    float x[E], t = 0.f;
    load(rr, x);
    bool finite = true;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      t = fmaxf(t, fabsf(x[e]));
      finite = finite && fabsf(x[e]) < INFINITY;
    }
    if (__all_sync(0xffffffffu, finite)) amax = fmaxf(amax, t);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = red[lane];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  int ex = 0;
  frexpf(amax > 0.f ? amax * D : 1.f, &ex);
  const float scale = ldexpf(1.f, max(min((tb.qjl ? 10 : 14) - ex, 100), -100));
  if (tid == 0) reinterpret_cast<float*>(ws + pl.ws_scale)[unit] = scale;
  uint8_t* table = ws + pl.ws_q + (long)unit * pl.q_bytes;
  const int blk = pl.rows * 128, part = pl.rows * D * 2;
#pragma unroll 1
  for (int rr = warp; rr < pl.rows; rr += 32) {
    float u[E];
    if (rr < rows) {
      load(rr, u);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = 0.f;
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

template <int D, int CN, int CPW>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl, uint8_t* __restrict__ ws) {
  // Warps of the softmax, of the keys and of the values.  Wide chunks keep the
  // softmax busiest: two warpgroups share each of theirs, 32 columns apiece.  Narrow
  // ones wait for the codes: two warpgroups unpack each side, half a row apiece.
  constexpr int SW = CN == 64 ? 16 : 8, KW = CN == 64 ? 4 : 8, VW = KW;
  constexpr int SUB = CN == 64 ? 32 : CN, NJ = SUB / 8;  // columns of a warpgroup
  constexpr int MB = D == 256 ? 2 : 1;     // 128-channel blocks of the output
  constexpr int NG = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t misc = pl.sm_misc;
  if ((uint32_t)__cvta_generic_to_shared(smem) != kDynSmemBase) {  // the plan's addresses assume it
    if (tid == 0) atomicOr(cv.status, (int)kFlagLayout);
    return;
  }
  auto bar = [&](int i) { return misc + 8 * i; };
  volatile int* dead = reinterpret_cast<volatile int*>(smem + (misc + kMiscDead - kDynSmemBase));
  const bool split = pl.chunks == 1;

  // The kernel before this one waited for all before it: only its own results (the
  // queries) are waited for here, where they are needed.
#pragma unroll 1
  for (int i = 0; i < (pl.lut_v != pl.lut_k ? 2 : 1); ++i)
    fill_lut(i ? pl.lut_v : pl.lut_k, i ? tb.v_bits : tb.k_bits, i ? tb.v_cent : tb.k_cent, i ? tb.v_lam : tb.k_lam);
  if (tid < kBars) tm::mbar_init(bar(tid), bar_count(tid, split, SW, KW));
  if (tid == 0) *dead = 0;
  if (warp == 24) tm::alloc_all(misc + kMiscTmem);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tm::fence_before();
  __syncthreads();
  tm::fence_after();
  // all of the tensor memory is this block's, so it starts at address 0: a constant,
  // which the matrix instructions (operands in uniform registers) are issued fastest from
  constexpr uint32_t tmem = 0;
  if (tm::lds32(misc + kMiscTmem) != tmem) {
    if (tid == 0) atomicOr(cv.status, (int)kFlagLayout);
    if (warp == 24) tm::dealloc_all(tm::lds32(misc + kMiscTmem));
    return;
  }
  pdl_trigger();

  Segment sg;
  uint32_t seg_n = 0;
  bool fail = false;

  // Registers move to the softmax: 4 x 88 + 56 + 56 + 40 = 7 x 72, or
  // 2 x 128 + 5 x 48 = 496 of these 504.
  if (warp < SW) {
    tm::regs_up<CN == 64 ? 88 : 128>();
    // =========================== softmax ===================================
    const int wg = warp >> 2, w = warp & 3, g = lane >> 2, qd = lane & 3;
    // the score and weight buffers of this warpgroup, and its first column in them
    const int buf = CN == 64 ? wg >> 1 : wg, part = CN == 64 ? 32 * (wg & 1) : 0;
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    const uint32_t t_s = tmem + pl.tm_s + buf * CN + part + lanes, sm_p = pl.sm_p + buf * (CN == 64 ? 16384 : 0);
    const uint32_t sm_m = misc + kMiscM, sm_al = misc + kMiscAlpha + wg * 128, sm_red = misc + kMiscRed + wg * 1024;
    // scores: folds softmax scale, log2(e) and the 1/sqrt(d) of the rotation (and of the dequantization)
    const float post0 = ta.scale * 1.4426950408889634f / (tb.affine ? sqrtf((float)D) : (float)D * tb.k_lam);
    const int live_rows = ta.n_q << ta.log_group, words = (ta.n_q + 31) >> 5;
    const int stride = split ? 2 : 1, first = split ? buf : 0, units = cv.kv_heads * pl.blocks;
    float l[CPW][2 * NJ];               // this thread's part of the sums; the current chunk's first
    uint32_t n_items = 0, n_tiles = 0;  // chunks done, tiles of all segments before this one
    pdl_wait();
    while (true) {
      const bool more = next_segment(misc, seg_n, sg, fail, dead);
      if (tm::bar_or(1 + wg, 128, !more)) break;  // all four warps leave together
      const long unit = (long)sg.b * units + sg.unit;
      const int row0 = (sg.unit % pl.blocks) * pl.rows;
      // (the scale is a power of two: its division is exact)
      const float post = post0 / reinterpret_cast<const float*>(ws + pl.ws_scale)[unit];
      const int ctx = min(max(cv.seq_lens[sg.b], 0), cv.capacity) - ta.n_q;
      const uint32_t* mask = ta.mask ? ta.mask + sg.b * ta.mask_stride : nullptr;
      // column of the outputs (and maxima) of column i of this warpgroup's
      auto column = [&](int i) { return (split ? buf : 2 * (i / SUB) + buf) * CN + part + i % SUB; };
      if ((tid & 127) < SUB * CPW) tm::stsf(sm_m + 4 * column(tid & 127), kNoMax);
#pragma unroll
      for (int s = 0; s < CPW; ++s)
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j) l[s][j] = 0.f;
      tm::bar_sync(1 + wg, 128);

#pragma unroll 1
      for (int it = first; it < sg.tiles; it += stride) {
        const uint32_t tile_no = n_tiles + it;
        const int slot = tile_no % kMetaSlots, tok0 = sg.t0 + it * kTile + 32 * w + g;
        const bool masked = sg.t0 + (it + 1) * kTile > ctx;
        fail = !tm::mbar_wait(bar(kBarMetaFull + slot), (tile_no / kMetaSlots) & 1, dead) || fail;
        float kn[4], vn[4], ev[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = pl.sm_meta + slot * 1536 + 4 * (32 * w + 8 * k + g);
          kn[k] = tm::ldsf(a) * post;
          vn[k] = tm::ldsf(a + 512);
          ev[k] = tm::ldsf(a + 1024);
        }
        __syncwarp();
        if (lane == 0) tm::mbar_arrive(bar(kBarMetaEmpty + slot));
#pragma unroll 1
        for (int step = 0; step < CPW; ++step) {  // this warpgroup's chunks
          const int chunk = split ? 0 : 2 * step + buf;
          const int col0 = (split ? buf : chunk) * CN + part;  // of the outputs and of the maxima
          fail = !tm::mbar_wait(bar(kBarSFull + buf), n_items & 1, dead) || fail;
          tm::fence_after();
          float y[8 * NJ];
          uint32_t vis = 0xffffffffu;
          if (__builtin_expect(masked, 0))
            vis = visible<NJ>(tok0, sg.len, ctx, row0 + chunk * CN + part + 2 * qd, live_rows, ta.log_group, mask,
                              words);
          bool again = false;
          while (true) {
            float2 m2[NJ];
            tm::ld_16x256b(t_s, y);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint2 x = tm::lds64(sm_m + 4 * (col0 + 8 * j + 2 * qd));
              m2[j] = make_float2(-__uint_as_float(x.x), -__uint_as_float(x.y));
            }
            tm::wait_ld(y);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                const int i = y_at<NJ>(k, j);
                const float2 x = tm::fma2(make_float2(y[i], y[i + 1]), make_float2(kn[k], kn[k]), m2[j]);
                y[i] = x.x;
                y[i + 1] = x.y;
              }
            if (__builtin_expect(masked, 0)) {
#pragma unroll
              for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (!((vis >> (8 * j + 4 * c + k)) & 1u)) y[y_at<NJ>(k, j) + c] = -INFINITY;
            }
            if (again) break;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float t = -INFINITY;
#pragma unroll
              for (int j = 0; j < NJ; ++j) t = fmaxf(fmaxf(t, y[y_at<NJ>(k, j)]), y[y_at<NJ>(k, j) + 1]);
              top = fmaxf(top, t + ev[k]);
            }
            // The running maximum (of score + log2 |v|, so that every weight p |v| stays
            // below 2^14 whatever the norms) moves only when a score passes it by that:
            // after the first tiles almost never, and all four warps vote together.
            again = tm::bar_or(1 + wg, 128, top > kTreeLazyLog2);
            if (__builtin_expect(!again, 1)) break;
            const Raise r{t_s, tmem + lanes + col0, sm_m + 4 * col0, sm_al, sm_red,
                          (uint32_t)bar(kBarPEmpty + buf), vis, (n_items & 1) ^ 1, wg, pl.cols,
                          it > first && (D > 64 || w < 2) ? MB : 0};
            fail = !raise_max<NJ>(r, kn, ev, dead) || fail;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint2 x = tm::lds64(sm_al + 4 * (8 * j + 2 * qd));
              l[0][2 * j] *= __uint_as_float(x.x);
              l[0][2 * j + 1] *= __uint_as_float(x.y);
            }
          }
          // the scores are in registers: the next chunk's may come
          tm::fence_before();
          __syncwarp();
          if (lane == 0) tm::mbar_arrive(bar(kBarSEmpty + buf));
          fail = !tm::mbar_wait(bar(kBarPEmpty + buf), (n_items & 1) ^ 1, dead) || fail;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            uint32_t pk[4];
            float2 sum = make_float2(l[0][2 * j], l[0][2 * j + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = y_at<NJ>(k, j);
              const float2 p = make_float2(fast_exp2(y[i]), fast_exp2(y[i + 1]));
              sum = tm::add2(sum, p);
              const float2 wt = tm::mul2(p, make_float2(vn[k], vn[k]));
              const __half2 hw = __floats2half2_rn(wt.x, wt.y);
              pk[k] = *reinterpret_cast<const uint32_t*>(&hw);
            }
            l[0][2 * j] = sum.x;
            l[0][2 * j + 1] = sum.y;
            tm::stmatrix_x4(sm_p + (32 * w + lane) * 128 + (((j + (CN == 64 ? part / 8 : 4 * wg)) ^ (lane & 7)) << 4),
                            pk[0], pk[1], pk[2], pk[3]);
          }
          tm::fence_proxy_async();
          tm::fence_before();
          __syncwarp();
          if (lane == 0) tm::mbar_arrive(bar(kBarPFull + buf));
          ++n_items;
          if constexpr (CPW == 2) {  // the other chunk's sums come to the front (registers have no index)
#pragma unroll
            for (int j = 0; j < 2 * NJ; ++j) {
              const float x = l[0][j];
              l[0][j] = l[1][j];
              l[1][j] = x;
            }
          }
        }
      }
      n_tiles += sg.tiles;
      // ---- the unit's partial
      fail = !tm::mbar_wait(bar(kBarPEmpty + buf), (n_items & 1) ^ 1, dead) || fail;
      tm::fence_after();
      const bool any = first < sg.tiles;
      const long pcol = (blockIdx.x + unit) * pl.cols;  // first column of the partial
#pragma unroll
      for (int s = 0; s < CPW; ++s)
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j) {
          float x = l[s][j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (g == 0) tm::stsf(sm_red + 256 * w + 4 * (s * SUB + 8 * (j >> 1) + 2 * qd + (j & 1)), x);
        }
      tm::bar_sync(1 + wg, 128);
      const int i0 = tid & 127;
      if (i0 < SUB * CPW) {
        const float x = (tm::ldsf(sm_red + 4 * i0) + tm::ldsf(sm_red + 256 + 4 * i0)) +
                        (tm::ldsf(sm_red + 512 + 4 * i0) + tm::ldsf(sm_red + 768 + 4 * i0));
        reinterpret_cast<float2*>(ws + pl.ws_ml)[pcol + column(i0)] =
            make_float2(tm::ldsf(sm_m + 4 * column(i0)), any ? x : 0.f);
      }
      if (any && (D > 64 || w < 2)) {
        float* wo = reinterpret_cast<float*>(ws) + pcol * D + 32 * w + lane;
#pragma unroll 1
        for (int i = 0; i < MB * CPW * (SUB / 16); ++i) {  // 16 columns at a time
          const int mb = i / (CPW * (SUB / 16)), c = 16 * (i % (CPW * (SUB / 16))), col = column(c);
          if (row0 + (split ? col - buf * CN : col) >= live_rows) continue;  // (columns without rows)
          uint32_t o[16];
          tm::ld_32x32b(tmem + lanes + mb * pl.cols + col, o);
          tm::wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) wo[(col + e) * D + mb * 128] = __uint_as_float(o[e]);
        }
      }
      tm::fence_before();
    }
  } else if (warp < SW + KW) {
    tm::regs_down<CN == 64 ? 56 : 48>();
    // =========================== keys ======================================
    const int w = warp & 3, half = KW == 8 ? (warp >> 2) & 1 : 0, tok = 32 * w + lane, row_bytes = tb.k_bits * D / 8;
    const uint32_t lut = pl.lut_k | (tb.k_bits == 3 ? lane * 4 : tb.k_bits == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
    const float sketch = tb.affine ? sqrtf(3.14159265358979f / (2.0f * D)) : sqrtf(3.14159265358979f / 2.0f) * tb.k_lam;
    uint32_t n = 0;  // tiles done
    int st = 0, st_ph = 0, kb = 0, k_ph = 0;
    while (next_segment(misc, seg_n, sg, fail, dead)) {
#pragma unroll 1
      for (int it = 0; it < sg.tiles; ++it, ++n) {
        const int slot = n % kMetaSlots;
        const uint32_t stage = pl.sm_st + st * pl.st_bytes;
        fail = !tm::mbar_wait(bar(kBarStFull + st), st_ph, dead);
        fail = !tm::mbar_wait(bar(kBarMetaEmpty + slot), ((n / kMetaSlots) & 1) ^ 1, dead) || fail;
        fail = !tm::mbar_wait(bar(kBarKEmpty + kb), k_ph ^ 1, dead) || fail;
        fail = __any_sync(0xffffffffu, fail);
        if (fail) break;
        const bool valid = sg.t0 + it * kTile + tok < sg.len;
        // ---- the token's norms
        float kn = 1.f, vn, ev = 0.f, ratio = 0.f;
        if (tb.affine) {
          uint32_t f = 1u;  // largest fp16 exponent field among the value's |scale|, |bias|
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const uint32_t x = tm::lds32(stage + pl.st_vn + (tok * NG + i) * 4);
            f = max(f, max((x >> 10) & 31u, (x >> 26) & 31u));
          }
          const int e = min((int)f, 29) - 15;
          ev = valid ? (float)e : 0.f;
          vn = !valid ? 0.f : f == 31u ? __int_as_float(0x7fffffff) : __int_as_float((e + 127) << 23);
        } else {
          const uint32_t a = tm::lds_half(stage + pl.st_kn + 2 * tok), b = tm::lds_half(stage + pl.st_vn + 2 * tok);
          kn = __half2float(__ushort_as_half((uint16_t)a));
          vn = valid ? __half2float(__ushort_as_half((uint16_t)b)) : 0.f;
          ev = valid ? fast_log2(vn + 0x1p-30f) : 0.f;
        }
        if (tb.qjl) {
          // the sketch enters the reduction as its ratio to the key's norm; a norm below
          // 2^-14 of it is raised to that, where the codes no longer count
          const float r = sketch * __half2float(__ushort_as_half((uint16_t)tm::lds_half(stage + pl.st_rn + 2 * tok)));
          if (!tb.affine) {
            if (kn < r * 0x1p-14f) kn = r * 0x1p-14f;
            ratio = kn > 0.f ? r / kn : 0.f;
          } else {
            ratio = r;
          }
        }
        // A value without a finite norm makes its scores NaN instead, so that it reaches
        // those who attend the token and no one else (0 * NaN is not 0).
        if (!(fabsf(vn) < INFINITY)) {
          vn = 0.f;
          kn = __int_as_float(0x7fffffff);
        }
        if (half == 0) {
          const uint32_t a_meta = pl.sm_meta + slot * 1536 + 4 * tok;
          tm::stsf(a_meta, kn);
          tm::stsf(a_meta + 512, vn);
          tm::stsf(a_meta + 1024, ev);
          __syncwarp();
          if (lane == 0) tm::mbar_arrive(bar(kBarMetaFull + slot));
        }
        // ---- channels, then signs
        tm::fence_after();
        const uint32_t dst = tmem + pl.tm_k + kb * pl.kcols + ((uint32_t)(32 * w) << 16);
        unpack_row<D / 8 / KW>(tb.k_bits, stage + tok * row_bytes, lut, half, [&](int c, uint32_t (&r)[16]) {
          if (tb.affine) {
            const uint32_t x = tm::lds32(stage + pl.st_kn + (tok * NG + (c >> 1)) * 4);
            const uint32_t s = __byte_perm(x, x, 0x1010), b = __byte_perm(x, x, 0x3232);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = hfma2_bits(s, r[i], b);
          }
          tm::st_32x32b(dst + 16 * c, r);
        });
        if (tb.qjl) {
          const uint32_t rr = pack_half2(__float2half_rn(ratio), __float2half_rn(ratio));
#pragma unroll 1
          for (int c = half * (D / 8 / KW); c < (half + 1) * (D / 8 / KW); ++c) {
            const uint32_t x = ~tm::lds32(stage + pl.st_s + tok * (D / 8) + 4 * c);  // bit 1: +
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = rr ^ ((x << (15 - j)) & 0x80008000u);
            tm::st_32x32b(dst + D / 2 + 16 * c, r);
          }
        }
        tm::wait_st();
        tm::fence_before();
        __syncwarp();
        if (lane == 0) {
          tm::mbar_arrive(bar(kBarStEmpty + st));
          tm::mbar_arrive(bar(kBarKFull + kb));
        }
        if (++st == pl.nst) st = 0, st_ph ^= 1;
        if (++kb == pl.nkb) kb = 0, k_ph ^= 1;
      }
    }
  } else if (warp < SW + KW + VW) {
    tm::regs_down<CN == 64 ? 56 : 48>();
    // =========================== values ====================================
    const int w = warp & 3, half = KW == 8 ? (warp >> 2) & 1 : 0, tok = 32 * w + lane, row_bytes = tb.v_bits * D / 8;
    const uint32_t lut = pl.lut_v | (tb.v_bits == 3 ? lane * 4 : tb.v_bits == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
    int st = 0, st_ph = 0, vb = 0, v_ph = 0;
    while (next_segment(misc, seg_n, sg, fail, dead)) {
#pragma unroll 1
      for (int it = 0; it < sg.tiles; ++it) {
        const uint32_t stage = pl.sm_st + st * pl.st_bytes;
        fail = !tm::mbar_wait(bar(kBarStFull + st), st_ph, dead);
        fail = !tm::mbar_wait(bar(kBarVEmpty + vb), v_ph ^ 1, dead) || fail;
        fail = __any_sync(0xffffffffu, fail);
        if (fail) break;
        uint32_t mul = 0u;     // affine: 2^-ev, exact
        bool sound = true;     // affine: a value past the row or without a finite form gives zeros here
        if (tb.affine) {
          uint32_t f = 1u;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const uint32_t x = tm::lds32(stage + pl.st_vn + (tok * NG + i) * 4);
            f = max(f, max((x >> 10) & 31u, (x >> 26) & 31u));
          }
          sound = f != 31u && sg.t0 + it * kTile + tok < sg.len;
          mul = (uint32_t)(15 - (min((int)f, 29) - 15)) << 10;
          mul |= mul << 16;
        }
        const uint32_t dst = pl.sm_v + vb * (kTile * D * 2) + tok * 128;
        unpack_row<D / 8 / VW>(tb.v_bits, stage + pl.st_v + tok * row_bytes, lut, half, [&](int c, uint32_t (&r)[16]) {
          if (tb.affine) {
            const uint32_t x = hmul2_bits(tm::lds32(stage + pl.st_vn + (tok * NG + (c >> 1)) * 4), mul);
            const uint32_t s = __byte_perm(x, x, 0x1010), b = __byte_perm(x, x, 0x3232);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = sound ? hfma2_bits(s, r[i], b) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tm::sts128(dst + (c >> 1) * 16384 + (((4 * (c & 1) + i) ^ (tok & 7)) << 4), r[4 * i], r[4 * i + 1],
                       r[4 * i + 2], r[4 * i + 3]);
        });
        tm::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tm::mbar_arrive(bar(kBarStEmpty + st));
          tm::mbar_arrive(bar(kBarVFull + vb));
        }
        if (++st == pl.nst) st = 0, st_ph ^= 1;
        if (++vb == pl.nvb) vb = 0, v_ph ^= 1;
      }
    }
  } else {
    tm::regs_down<CN == 64 ? 40 : 48>();
    const uint32_t d_hi = tm::desc_hi(1024);
    if (warp == 24) {
      // ========================= scores ======================================
      const uint32_t id = tm::mma_idesc(CN, false, false), d_q = tm::desc_lo(pl.sm_q, 16);
      const uint32_t q_blk = pl.rows * 128 / 16, q_part = pl.rows * D * 2 / 16;
      const int code_parts = pl.parts - (tb.qjl ? 1 : 0);
      uint32_t kb = 0, k_ph = 0, s_ph = 0, buf = 0;  // s_ph: a bit for either score buffer
      while (next_segment(misc, seg_n, sg, fail, dead)) {
        fail = !tm::mbar_wait(bar(kBarQFull), (seg_n - 1) & 1, dead);
        buf = 0;
#pragma unroll 1
        for (int t = 0; !fail && __any_sync(0xffffffffu, t < sg.tiles); ++t) {  // (votes: uniform to the compiler too)
          fail = !tm::mbar_wait(bar(kBarKFull + kb), k_ph, dead);
          const uint32_t a = tmem + pl.tm_k + kb * pl.kcols;
          uint32_t bq = d_q;
#pragma unroll 1
          for (int c = 0; c < pl.chunks; ++c, buf ^= 1, bq += CN * 128 / 16) {
            fail = !tm::mbar_wait(bar(kBarSEmpty + buf), ((s_ph >> buf) & 1) ^ 1, dead) || fail;
            s_ph ^= 1u << buf;
            tm::fence_after();
            const uint32_t d = tmem + pl.tm_s + buf * CN;
            if (lane == 0 && !fail) {
              uint32_t b = bq;
              // codes (fp16 calls: the queries' high, then low parts), then signs
#pragma unroll 1
              for (int p = 0; p < pl.parts; ++p, b += q_part) {
                const uint32_t ap = a + (p == code_parts ? D / 2 : 0);
                tm::mma_ts(d, ap, b, d_hi, id, p);
#pragma unroll
                for (int k = 1; k < D / 16; ++k)
                  tm::mma_ts(d, ap + 8 * k, b + (k >> 2) * q_blk + 2 * (k & 3), d_hi, id, 1);
              }
              tm::mma_commit(bar(kBarSFull + buf));
              if (c == pl.chunks - 1) {
                tm::mma_commit(bar(kBarKEmpty + kb));
                if (t == sg.tiles - 1) tm::mma_commit(bar(kBarQEmpty));
              }
            }
            __syncwarp();
          }
          if (++kb == (uint32_t)pl.nkb) kb = 0, k_ph ^= 1;
        }
      }
    } else if (warp == 25) {
      // ========================= outputs =====================================
      const uint32_t id = tm::mma_idesc(CN, true, true), d_v = tm::desc_lo(pl.sm_v, D == 64 ? 0 : 16384),
                     d_p = tm::desc_lo(pl.sm_p, 16);
      uint32_t vb = 0, v_ph = 0, p_ph = 0, buf = 0;
      while (next_segment(misc, seg_n, sg, fail, dead)) {
        buf = 0;
#pragma unroll 1
        for (int t = 0; !fail && __any_sync(0xffffffffu, t < sg.tiles); ++t) {
          fail = !tm::mbar_wait(bar(kBarVFull + vb), v_ph, dead);
          const uint32_t acc = split ? t >= 2 : t >= 1;  // the first of a unit's products overwrites
          uint32_t d = tmem + (split ? buf * CN : 0);
#pragma unroll 1
          for (int c = 0; c < pl.chunks; ++c, buf ^= 1, d += CN) {
            fail = !tm::mbar_wait(bar(kBarPFull + buf), (p_ph >> buf) & 1, dead) || fail;
            p_ph ^= 1u << buf;
            tm::fence_after();
            if (lane == 0 && !fail) {
              const uint32_t b = d_p + buf * ((CN == 64 ? 16384 : 64) / 16);
#pragma unroll 1
              for (int mb = 0; mb < MB; ++mb) {
                const uint32_t a = d_v + vb * (kTile * D * 2 / 16) + mb * (2 * 16384 / 16), dm = d + mb * pl.cols;
                tm::mma_ss(dm, a, d_hi, b, d_hi, id, acc);
#pragma unroll
                for (int k = 1; k < kTile / 16; ++k)
                  tm::mma_ss(dm, a + k * (2048 / 16), d_hi, b + k * (2048 / 16), d_hi, id, 1);
              }
              tm::mma_commit(bar(kBarPEmpty + buf));
              if (c == pl.chunks - 1) tm::mma_commit(bar(kBarVEmpty + vb));
            }
            __syncwarp();
          }
          if (++vb == (uint32_t)pl.nvb) vb = 0, v_ph ^= 1;
        }
      }
    } else if (warp == 26) {
      // ========================= share, segments, packed tiles ===============
      // This block takes tiles [t, t1) of the T laid end to end over all units.
      const int n_q = ta.n_q, max_ctx = ta.max_ctx, units = cv.kv_heads * pl.blocks;
      long long T = 0;
      for (int r = lane; r < cv.batch; r += 32) T += tree_tiles(cv, r, n_q, max_ctx);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
      T *= units;
      long long t = tile_bound(blockIdx.x, T, gridDim.x);
      const long long t1 = tile_bound((long long)blockIdx.x + 1, T, gridDim.x);
      long long rs = 0;  // tiles before row b
      int b = 0;
      for (; b < cv.batch && t < t1; b += 32) {
        const int n = b + lane < cv.batch ? tree_tiles(cv, b + lane, n_q, max_ctx) : 0;
        long long e = n;  // tiles up to and with this row
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, e, o);
          if (lane >= o) e += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, rs + e * units > t);
        if (past) {
          const int f = __ffs(past) - 1;
          rs += (__shfl_sync(0xffffffffu, e, f) - __shfl_sync(0xffffffffu, n, f)) * units;
          b += f;
          break;
        }
        rs += __shfl_sync(0xffffffffu, e, 31) * units;
      }
      if (lane == 0) {
        const uint32_t k_row = tb.k_bits * D / 8, v_row = tb.v_bits * D / 8, meta = tb.affine ? 4 * NG : 2;
        int st = 0, st_ph = 0;
        uint32_t copies = 0;
        while (true) {
          Segment s{0, 0, 0, 0, 0};
          while (t < t1) {
            const int len = tree_len(cv, b, n_q, max_ctx), n = (len + kTile - 1) / kTile;
            const long long row = (long long)n * units;
            if (t >= rs + row) {
              rs += row;
              ++b;
              continue;
            }
            const long long at = t - rs;
            const int u = at < (1ll << 31) ? (int)((unsigned)at / (unsigned)n) : (int)(at / n);
            const long long us = rs + (long long)u * n, te = min(t1, us + n);
            s = Segment{b, u, (int)(t - us) * kTile, (int)(te - t), len};
            t = te;
            break;
          }
          const uint32_t slot = seg_n % kSegs, a = misc + kMiscSeg + 32 * slot;
          fail = !tm::mbar_wait_lane(bar(kBarSegEmpty + slot), ((seg_n / kSegs) & 1) ^ 1, dead);
          tm::sts128(a, s.b, s.unit, s.t0, fail ? 0 : s.tiles);
          tm::sts128(a + 16, s.len, 0, 0, 0);
          tm::mbar_arrive(bar(kBarSegFull + slot));
          ++seg_n;
          if (s.tiles == 0 || fail) break;
          const int kvh = s.unit / pl.blocks;
#pragma unroll 1
          for (int it = 0; it < s.tiles; ++it, ++copies) {
            fail = !tm::mbar_wait_lane(bar(kBarStEmpty + st), st_ph ^ 1, dead);
            if (fail) break;
            const int tk = s.t0 + it * kTile;
            const uint32_t m = min(kTile, (s.len - tk + 15) / 16 * 16);  // within the row: capacity is a multiple of 16
            const long at = ((long)s.b * cv.kv_heads + kvh) * cv.capacity + tk;
            const uint32_t dst = pl.sm_st + st * pl.st_bytes, full = bar(kBarStFull + st);
            tm::mbar_expect(full, m * (k_row + v_row + 2 * meta + (tb.qjl ? D / 8 + 2 : 0)));
            tm::bulk_load(dst, cv.k_codes + at * k_row, m * k_row, full);
            tm::bulk_load(dst + pl.st_kn, reinterpret_cast<const uint8_t*>(cv.k_norm) + at * meta, m * meta, full);
            tm::bulk_load(dst + pl.st_vn, reinterpret_cast<const uint8_t*>(cv.v_norm) + at * meta, m * meta, full);
            if (tb.qjl) {
              tm::bulk_load(dst + pl.st_s, cv.k_signs + at * (D / 8), m * (D / 8), full);
              tm::bulk_load(dst + pl.st_rn, cv.k_rnorm + at, m * 2, full);
            }
            tm::bulk_load(dst + pl.st_v, cv.v_codes + at * v_row, m * v_row, full);
            if (++st == pl.nst) st = 0, st_ph ^= 1;
          }
        }
        if (fail) {  // after a failure the copies in flight are waited for
          int never = 0;
          for (uint32_t i = copies > (uint32_t)pl.nst ? copies - pl.nst : 0; i < copies; ++i)
            tm::mbar_wait_lane(bar(kBarStFull + i % pl.nst), (i / pl.nst) & 1, &never);
        }
      }
      __syncwarp();
      if (blockIdx.x == 0)
        for (int r = lane; r < cv.batch; r += 32)
          if (min(max(cv.seq_lens[r], 0), cv.capacity) > max_ctx) atomicOr(cv.status, (int)kFlagMaxCtx);
    } else {
      // ========================= query tables ================================
      pdl_wait();
      uint32_t loads = 0;
      while (next_segment(misc, seg_n, sg, fail, dead)) {
        fail = !tm::mbar_wait(bar(kBarQEmpty), (loads & 1) ^ 1, dead);
        if (lane == 0 && !fail) {
          const long unit = (long)sg.b * (cv.kv_heads * pl.blocks) + sg.unit;
          tm::mbar_expect(bar(kBarQFull), pl.q_bytes);
          tm::bulk_load(pl.sm_q, ws + pl.ws_q + unit * pl.q_bytes, pl.q_bytes, bar(kBarQFull));
        }
        __syncwarp();
        if (!fail) ++loads;
      }
      if (fail && loads > 0 && lane == 0) {
        int never = 0;
        tm::mbar_wait_lane(bar(kBarQFull), (loads - 1) & 1, &never);
      }
      __syncwarp();
    }
    if (warp < 26 && fail && lane == 0) {  // after a failure the products in flight are waited for
      int never = 0;
      tm::mma_commit(bar(kBarDone + warp - 24));
      tm::mbar_wait_lane(bar(kBarDone + warp - 24), 0, &never);
    }
    __syncwarp();
  }
  tm::fence_before();
  __syncthreads();
  if (tid == 0 && *dead) atomicOr(cv.status, (int)kFlagTimeout);
  if (warp == 24) {
    tm::fence_after();
    tm::dealloc_all(tmem);
  }
}

constexpr int kMergeWarps = 4;
constexpr int kMergeMax = 2 * kTreeMaxCtas;  // partials of one row

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
    const long long x = tree_tiles(cv, k, ta.n_q, ta.max_ctx);
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
  const int n = tree_tiles(cv, b, ta.n_q, ta.max_ctx);
  const long out_at = (((long)b * ta.n_q + i) * ta.q_heads + h) * D;
  const long long T = all * units, unit = (long long)kvh * pl.blocks + rb, su = before * units + unit * n, eu = su + n;
  const int c_lo = n > 0 ? (int)(((su + 1) * nctas + T - 1) / T - 1) : 0;
  const int c_hi = n > 0 ? (int)((eu * nctas + T - 1) / T - 1) : -1;
  const int sides = pl.chunks == 1 ? 2 : 1, S = (c_hi - c_lo + 1) * sides;
  const long slot0 = c_lo + (long)b * units + unit;
  pdl_wait();
  float m = kNoMax;
  for (int s = tid; s < S; s += NT) {
    const long long c = c_lo + s / sides, f0 = tile_bound(c, T, nctas), f1 = tile_bound(c + 1, T, nctas);
    float ms = -INFINITY;
    if (max(f0, su) < min(f1, eu)) {  // a block with an empty range left no partial
      const float2 x = reinterpret_cast<const float2*>(ws + pl.ws_ml)[(slot0 + s / sides) * pl.cols + (s % sides) * pl.rows + col];
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
    const long at = (slot0 + s / sides) * pl.cols + (s % sides) * pl.rows + col;
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

// Shared addresses, first fit into the gaps that alignment leaves.
struct Arena {
  std::vector<std::pair<int, int>> free{{(int)kDynSmemBase, 228 * 1024}};  // 227 KB of a block, from kDynSmemBase
  int end = kDynSmemBase;
  bool ok = true;
  int take(int bytes, int align) {
    for (size_t i = 0; i < free.size(); ++i) {
      const int a = (free[i].first + align - 1) / align * align;
      if (a + bytes > free[i].second) continue;
      const int hi = free[i].second;
      free[i].second = a;
      free.insert(free.begin() + i + 1, {a + bytes, hi});
      end = std::max(end, a + bytes);
      return a;
    }
    ok = false;
    return 0;
  }
};

// The plan of `rows` query rows, or of blocks of them: the narrowest columns
// that hold them all and whose buffers fit, else the widest that fit.
bool plan_shape(const Tables& tb, int dtype, int cn, int chunks, int nkb, int nvb, int nst, TreePlan* p) {
  const int d = tb.d;
  p->cn = cn;
  p->chunks = chunks;
  p->rows = cn * chunks;
  p->cols = chunks == 1 ? 2 * cn : p->rows;
  p->parts = 1 + (dtype == kF16) + (tb.qjl != 0);
  p->nkb = nkb;
  p->nvb = nvb;
  p->nst = nst;
  p->kcols = d / 2 * (tb.qjl ? 2 : 1);
  p->tm_k = p->cols * (d == 256 ? 2 : 1);
  p->tm_s = p->tm_k + nkb * p->kcols;
  if (p->tm_s + 2 * cn > 512) return false;
  Arena a;
  p->lut_k = a.take(lut_bytes(tb.k_bits), lut_bytes(tb.k_bits));
  p->lut_v = tb.k_bits == tb.v_bits ? p->lut_k : a.take(lut_bytes(tb.v_bits), lut_bytes(tb.v_bits));
  p->sm_v = a.take(nvb * kTile * d * 2, 1024);
  p->sm_q = a.take(p->parts * p->rows * d * 2, 1024);
  p->sm_p = a.take(cn == 64 ? 2 * 16384 : 16384, 1024);  // narrow chunks: halves of one buffer's rows
  const int meta = tb.affine ? 4 * d / kAffineGroup : 2;
  int at = kTile * tb.k_bits * d / 8;
  auto part = [&](int bytes) {
    const int x = at;
    at += kTile * bytes;
    return x;
  };
  p->st_v = part(tb.v_bits * d / 8);
  p->st_s = part(tb.qjl ? d / 8 : 0);
  p->st_kn = part(meta);
  p->st_vn = part(meta);
  p->st_rn = part(tb.qjl ? 2 : 0);
  p->st_bytes = (at + 127) / 128 * 128;
  p->sm_st = a.take(nst * p->st_bytes, 128);
  p->sm_meta = a.take(kMetaSlots * 3 * kTile * 4, 128);
  p->sm_misc = a.take(kMiscBytes, 16);
  // at least half of an SM's shared memory: one block per SM, which owns its tensor memory
  p->smem = std::max(a.end - (int)kDynSmemBase, 120 * 1024);
  return a.ok;
}

void plan_tree(const Tables& tb, int dtype, int batch, int q_heads, int kv_heads, int n_q, int max_ctx, TreePlan* p) {
  const int rows = n_q * (q_heads / kv_heads);
  static const int shapes[][2] = {{64, 4}, {64, 2}, {64, 1}, {32, 1}, {16, 1}};
  int best = -1, nst = 2;
  for (int i = 0; i < 5; ++i) {
    if (!plan_shape(tb, dtype, shapes[i][0], shapes[i][1], 1, 1, nst, p)) continue;
    if (best < 0 || p->rows >= rows) best = i;
  }
  const int cn = shapes[best][0], chunks = shapes[best][1];
  // then as many buffers as fit: values first (their buffer waits for the product
  // of the weights), keys, packed stages
  int nkb = 1, nvb = 1;
  if (plan_shape(tb, dtype, cn, chunks, nkb, 2, nst, p)) nvb = 2;
  if (plan_shape(tb, dtype, cn, chunks, 2, nvb, nst, p)) nkb = 2;
  while (nst < kMaxStages && plan_shape(tb, dtype, cn, chunks, nkb, nvb, nst + 1, p)) ++nst;
  plan_shape(tb, dtype, cn, chunks, nkb, nvb, nst, p);
  p->blocks = (rows + p->rows - 1) / p->rows;
  const long units = (long)batch * kv_heads * p->blocks;
  p->ctas = (int)std::max(1L, std::min((long)kTreeMaxCtas, units * ((max_ctx + kTile - 1) / kTile)));
  p->slots = p->ctas + units;
  p->q_bytes = p->parts * p->rows * tb.d * 2;
  p->ws_ml = p->slots * p->cols * tb.d * 4;
  p->ws_q = (p->ws_ml + p->slots * p->cols * 8 + 127) / 128 * 128;
  p->ws_scale = p->ws_q + units * p->q_bytes;
}

size_t plan_bytes(const TreePlan& p) { return (size_t)p.ws_scale + (size_t)(p.slots - p.ctas) * 4; }

template <int D, int CN, int CPW>
cudaError_t launch_shape(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                         cudaStream_t stream) {
  static KernelConfig config;
  auto kern = tree_kernel<D, CN, CPW>;
  // the attribute is set once per device, for the largest plan
  cudaError_t e = configure_kernel(config, kern, 227 * 1024, kTreeThreads, nullptr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pl.slots - pl.ctas));
  cfg.blockDim = dim3(kPrepThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_query_kernel<D>, tb, cv, ta, pl, ws);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(pl.ctas);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = pl.smem;
  e = cudaLaunchKernelEx(&cfg, kern, tb, cv, ta, pl, ws);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(ta.n_q * ta.q_heads), (unsigned)cv.batch);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, tb, cv, ta, pl, (const uint8_t*)ws);
}

template <int D>
cudaError_t launch_dim(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                       cudaStream_t stream) {
  if (pl.cn == 16) return launch_shape<D, 16, 1>(tb, cv, ta, pl, ws, stream);
  if (pl.cn == 32) return launch_shape<D, 32, 1>(tb, cv, ta, pl, ws, stream);
  if (pl.chunks <= 2) return launch_shape<D, 64, 1>(tb, cv, ta, pl, ws, stream);
  if constexpr (D < 256) return launch_shape<D, 64, 2>(tb, cv, ta, pl, ws, stream);
  return cudaErrorNotSupported;
}

}  // namespace

size_t tree_workspace_bytes(const Tables& tb, int batch, int q_heads, int kv_heads, int n_q, int max_ctx) {
  TreePlan a, b;  // of either type, so that the size does not depend on it
  plan_tree(tb, kBF16, batch, q_heads, kv_heads, n_q, max_ctx, &a);
  plan_tree(tb, kF16, batch, q_heads, kv_heads, n_q, max_ctx, &b);
  return std::max(plan_bytes(a), plan_bytes(b));
}

cudaError_t launch_tree(const Tables& tb, const CacheView& cv, const TreeArgs& ta, float* workspace,
                        cudaStream_t stream) {
  TreePlan pl;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  plan_tree(tb, ta.dtype, cv.batch, ta.q_heads, cv.kv_heads, ta.n_q, ta.max_ctx, &pl);
  switch (tb.d) {
    case 64: return launch_dim<64>(tb, cv, ta, pl, ws, stream);
    case 128: return launch_dim<128>(tb, cv, ta, pl, ws, stream);
    case 256: return launch_dim<256>(tb, cv, ta, pl, ws, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace tq
