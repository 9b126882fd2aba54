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
//   softmax     1, 2 or 4 warpgroups share the columns of a chunk (16 to 128), keep
//               their maxima and sums and write P to shared memory;
//   keys        a thread unpacks a token's codes (or half of them) through a table
//               of code pairs into the token's lane of tensor memory, the product's
//               A operand (no shared-memory round trip, no swizzle);
//   values      the same into shared memory, token rows of 64 channels;
//   two warps   issue the matrix instructions, of scores and of outputs (one
//               thread's instructions would bound the kernel);
//   one warp    works out the block's share, announces its segments to the others
//               and copies the packed tiles in, a few stages ahead;
//   one warp    copies a segment's query table in.
// Chunks are 128 columns wide where the rows fill them: an instruction of 64 or
// fewer columns takes 50 cycles, of 128 no more than 64 (measured).  The roles share
// the instruction caches, and fetching instructions is what bounds them first (a
// third of all stalls): loops stay rolled where registers allow it, the codec is
// fixed at compile time, and nothing that runs once per segment is unrolled.
// A key's norm multiplies its scores, a value's norm its weights, both fp32, in
// the softmax; so the fp16 operands hold centroids (scaled by k_lam / v_lam, at
// which they are nearly exact) and lose nothing.  The sketch's signs follow the
// key's channels in the reduction, as +- rnorm / norm, against a second table of
// rotated queries; an fp16 call holds its queries in two fp16 parts (hi + lo).  The weights
// are one fp16 number each: a low part would double their buffers and the second product,
// and their roundings average out over a row (against 64 bits, fp16 calls are 1.1 to 1.4
// times as far off as by the output's rounding alone, bf16 calls 1.00 to 1.03).
// The affine codec's operands are scale * level + bias, rounded to fp16 (1.4 to 2.4 times
// in fp16 calls, 1.01 to 1.04 in bf16 ones).
//
// The token tiles of all (batch row, KV head, block of query rows) units are laid
// end to end and each block takes an equal share, as in the decode; a unit that
// a block meets leaves a partial (O, maximum, sum) in the workspace.  A kernel
// before it rotates the queries and lays them out as the product's B operand, once
// for all blocks; a kernel after it merges the partials and rotates back.
#pragma once

#include "tq_decode_impl.cuh"
#include "tq_tmem.cuh"

#include <atomic>

namespace tq {

constexpr int kTile = 128;          // tokens per tile: the matrix instruction's rows
constexpr int kTreeMaxCtas = 148;   // one block per SM; the workspace is sized for it
// Tiles whose norms are kept.  A slot is written for tile t when the scores of t - 2
// (at most two key buffers) are done; their buffer had been given back by then, by
// warps that had finished tile t - 5 or a later one: six slots need no barrier.
constexpr int kMetaSlots = 6;
constexpr int kMaxStages = 8;
// The running maximum (log2), of score + log2 |v|, moves when a weight passes 2^15.9
// (fp16 holds 2^16) and then brings the largest to 2^4.  Above: a key that resembles the
// query outscores the others by about 2^13 at head_dim 128, so that little room would
// raise the maximum of some column in most tiles.  Below: a weight under 2^-25 is lost,
// and a long flat tail's weights are small but many: 2^-29 of the largest for each token,
// 2^-12 for 128k of them.  63 drafts at 32k, 16 ragged rows, 4 x 128k with the sketch:
// 77, 195, 432 us; bringing it to 1 instead (2^-25, 0.4 % of such a row) 76, 194, 417 us;
// to 2^7 86, 212, 522 us.
constexpr float kTreeLazyLog2 = 15.9f, kTreeRaiseLog2 = 4.0f;
constexpr float kNoMax = -3e38f;    // running maximum before any score (finite: no inf - inf)

// What a score is multiplied by after its product, beside its query's and its key's
// scale: the softmax's scale, log2(e), and the 1/sqrt(d) of the rotation (and of the
// dequantization).
__device__ __forceinline__ float score_factor(const Tables& tb, float scale) {
  return scale * 1.4426950408889634f / (tb.affine ? sqrtf((float)tb.d) : (float)tb.d * tb.k_lam);
}

// Bytes of the tables: 2-bit codes four at a time (8 bytes, 16 copies), 3-bit
// pairs (32 copies), 4-bit pairs (16 copies: 32 would cost a stage).  A lane
// reads its own copy, so lookups meet in a bank at most twice.
constexpr int lut_bytes(int bits) { return bits == 2 ? 32768 : bits == 3 ? 8192 : 16384; }

// What the host settles about one call.
struct TreePlan {
  int cn, chunks;          // score columns per chunk, chunks
  int rows, blocks;        // query rows per unit (cn * chunks), blocks of them per KV head
  int parts;               // query tables: 1, + 1 (fp16 low parts), + 1 (sketch)
  int nkb, nvb, nst, nsb;  // key, value, packed, and score and weight buffers
  int tm_k, tm_s, kcols;   // tensor memory columns: keys, scores; columns of one key buffer
  int lut_k, lut_v, sm_q, sm_v, sm_p, sm_st, sm_meta, sm_misc, smem;  // shared addresses
  int st_v, st_s, st_kn, st_vn, st_rn, st_bytes;                      // inside a stage
  int ctas, q_bytes;       // q_bytes: one unit's query table
  // workspace: bytes to the maxima and sums, the query tables, their scales, the rows' factors
  long slots, ws_ml, ws_q, ws_scale, ws_rows;
};

// Shared misc area: barriers, segments, then floats.
constexpr int kSegs = 4;  // segments announced ahead
constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarStFull = 2, kBarStEmpty = kBarStFull + kMaxStages,
              kBarKFull = kBarStEmpty + kMaxStages, kBarKEmpty = kBarKFull + 2, kBarVFull = kBarKEmpty + 2,
              kBarVEmpty = kBarVFull + 2, kBarSFull = kBarVEmpty + 2, kBarSEmpty = kBarSFull + 2,
              kBarPFull = kBarSEmpty + 2, kBarPEmpty = kBarPFull + 2, kBarSegFull = kBarPEmpty + 2,
              kBarSegEmpty = kBarSegFull + kSegs, kBarDone = kBarSegEmpty + kSegs, kBars = kBarDone + 2;
constexpr int kMiscTmem = kBars * 8, kMiscDead = kMiscTmem + 4,
              kMiscSeg = (kMiscTmem + 8 + 31) / 32 * 32,  // [kSegs][8] ints
              kMiscM = kMiscSeg + kSegs * 32,             // running maxima [256]
              kMiscAlpha = kMiscM + 1024,                 // rescale factors [4][32]
              kMiscRed = kMiscAlpha + 512,                // [4 warpgroups][4 warps][64]
              kMiscBytes = kMiscRed + 4096;

// Arrivals that complete barrier i's phase.
__device__ __forceinline__ int bar_count(int i, int softmax_warps, int unpack_warps) {
  if (i >= kBarStEmpty && i < kBarKFull) return 2 * unpack_warps;
  if ((i >= kBarKFull && i < kBarKEmpty) || (i >= kBarVFull && i < kBarVEmpty)) return unpack_warps;
  if (i >= kBarSEmpty && i < kBarPEmpty) return softmax_warps;  // and kBarPFull
  if (i >= kBarSFull && i < kBarSEmpty) return 2;               // the products, and the warp that issued them
  if (i >= kBarSegEmpty && i < kBarDone) return softmax_warps + 2 * unpack_warps + 3;  // all but the announcer
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
// What a unit of `tiles` tiles counts for in the blocks' shares: its tiles, and a few
// more for what a segment costs besides (the queries' copy, the pipeline's filling,
// the partial's stores: about 9000 cycles, a tile takes 2500 to 6000).  Without them a
// block with many short rows took 1.2 times the average (16 ragged rows).
constexpr int kUnitCost = 3;
__device__ __forceinline__ int tree_span(int tiles) { return tiles > 0 ? tiles + kUnitCost : 0; }
__device__ __forceinline__ int tree_span(const CacheView& cv, int b, int n_q, int max_ctx) {
  return tree_span((tree_len(cv, b, n_q, max_ctx) + kTile - 1) / kTile);
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

// f(block, pairs) for each of N blocks of 32 channels of a packed row at shared
// address `row`: 16 fp16 pairs from the table.  The row's words are loaded first.
template <int N, int BITS, bool WIDE, typename F>
__device__ __forceinline__ void unpack_row(uint32_t row, uint32_t lut, F f) {
  uint32_t w[N * BITS];
  if constexpr (WIDE && N * BITS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N * BITS / 4; ++i) {
      const uint4 x = tm::lds128(row + 16 * i);
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  } else if constexpr (N * BITS % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N * BITS / 2; ++i) {
      const uint2 x = tm::lds64(row + 8 * i);
      w[2 * i] = x.x;
      w[2 * i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N * BITS; ++i) w[i] = tm::lds32(row + 4 * i);
  }
#pragma unroll
  for (int c = 0; c < N; ++c) {
    uint32_t r[16];
    const uint32_t* x = w + BITS * c;
    if constexpr (BITS == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // a byte of four codes, entries 128 bytes apart
        const uint2 y = tm::lut64(bits_at(x[i >> 2], 8 * (i & 3), 8, 7) | lut);
        r[2 * i] = y.x;
        r[2 * i + 1] = y.y;
      }
    } else if constexpr (BITS == 3) {
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = tm::lut32(field_scaled(x, 3, 6 * i, 6, 7) | lut);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = tm::lut32(bits_at(x[i >> 2], 8 * (i & 3), 8, 6) | lut);
    }
    f(c, r);
  }
}

// The same, in a rolled loop if ROLLED: beside the softmax of two wide chunks the
// unrolled one costs more in instruction fetches than it gains (gqa 32k 78 us
// instead of 74; with one chunk it gains: 4 x 128k with the sketch 450 -> 421 us).
template <bool ROLLED, int N, int BITS, bool WIDE, typename F>
__device__ __forceinline__ void unpack_blocks(uint32_t row, uint32_t lut, F f) {
  if constexpr (ROLLED) {
#pragma unroll 1
    for (int c = 0; c < N; ++c)
      unpack_row<1, BITS, WIDE>(row + 4 * BITS * c, lut, [&](int, uint32_t (&r)[16]) { f(c, r); });
  } else {
    unpack_row<N, BITS, WIDE>(row, lut, f);
  }
}

// Fills a table with every lane's copy of every entry.
__device__ __forceinline__ void fill_lut(uint32_t lut, int bits, const float* cent, float lam) {
  const uint32_t mask = (1u << bits) - 1u;
  // 16-byte pieces: a quad's two pairs twice, or a pair four times
  const int shift = bits == 4 ? 2 : 3, pieces = (bits == 2 ? 256 : 1 << (2 * bits)) << shift;
#pragma unroll 1
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
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
  uint32_t a_m, sm_al, sm_red, bar_p;  // maxima (negated) of the columns; factors; scratch; the products' barrier
  uint32_t vis, parity;
  int wg, cols, blocks;                // blocks: 128-channel blocks of the output to rescale
};

// Multiplies a warp's scores in tensor memory, `cols` columns, by the columns' factors
// and by the lane's token's norm.
__device__ __forceinline__ void finish_scores(uint32_t at, int cols, const float* factors, float norm) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 16) {
    uint32_t x[16];
    tm::ld_32x32b(at + c, x);
    tm::wait_ld(x);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * factors[c + e] * norm);
    tm::st_32x32b(at + c, x);
  }
  tm::wait_st();
}

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
    const float old = -tm::ldsf(at);
    const float mn = fmaxf(old, fmaxf(fmaxf(tm::ldsf(red), tm::ldsf(red + 256)),
                                      fmaxf(tm::ldsf(red + 512), tm::ldsf(red + 768))) - kTreeRaiseLog2);
    tm::stsf(at, -mn);
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

// Warps of a kernel: softmax (a warpgroup per 16 or 32 columns), keys (values as
// many), and the four others.  At head_dim 256 a second warpgroup unpacks each side,
// half a row apiece (157 us instead of 169 at 8 drafts and 200k); at 128 it gains
// nothing over fewer, larger warps.
template <int D, int CN>
struct Roles {
  static constexpr int SW = D < 256 && CN >= 64 ? 16 : CN == 16 ? 4 : 8, KW = D == 256 ? 8 : 4;
  static constexpr int WARPS = SW + 2 * KW + 4, THREADS = 32 * WARPS;
  // registers of a softmax, an unpacking and another thread: moved from what the block
  // is launched with, 72, 80, 96 or 128 for each of 7, 6, 5 or 4 warpgroups
  static constexpr int RS = SW == 16 ? 88 : 128, RU = WARPS == 28 ? (SW == 16 ? 56 : 48) : WARPS == 24 ? 64 : WARPS == 20 ? 72 : 96,
                       RO = SW == 16 ? 40 : WARPS == 28 ? 48 : WARPS == 24 ? 56 : WARPS == 20 ? 56 : 64;
  static constexpr int LAUNCH = WARPS == 28 ? 72 : WARPS == 24 ? 80 : WARPS == 20 ? 96 : 128;
  static_assert(SW * RS + 2 * KW * RU + 4 * RO <= WARPS * LAUNCH, "the shares' sum is within the launch's registers");
};

template <int D, int CN, int CPT, int KB, int VB, bool QJL, bool AFF>
__global__ void __launch_bounds__(Roles<D, CN>::THREADS, 1)
    tree_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl, uint8_t* __restrict__ ws) {
  using R = Roles<D, CN>;
  constexpr int SW = R::SW, KW = R::KW, OW = SW + 2 * KW;  // OW: the first of the others
  constexpr int SUB = CN / (SW / 4), NJ = SUB / 8;         // columns of a warpgroup
  constexpr int N = D / 8 / KW;                            // blocks of 32 channels that a thread unpacks
  constexpr int MB = D == 256 ? 2 : 1;     // 128-channel blocks of the output
  constexpr int NG = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t misc = pl.sm_misc;
  if ((uint32_t)__cvta_generic_to_shared(smem) != kDynSmemBase) {  // the plan's addresses assume it
    if (tid == 0) atomicOr(cv.status, (int)kFlagLayout);
    return;
  }
  auto bar = [&](int i) { return misc + 8 * i; };
  volatile int* dead = reinterpret_cast<volatile int*>(smem + (misc + kMiscDead - kDynSmemBase));

  // The kernel before this one waited for all before it: only its own results (the
  // queries) are waited for here, where they are needed.
#pragma unroll 1
  for (int i = 0; i < (pl.lut_v != pl.lut_k ? 2 : 1); ++i)
    fill_lut(i ? pl.lut_v : pl.lut_k, i ? VB : KB, i ? tb.v_cent : tb.k_cent, i ? tb.v_lam : tb.k_lam);
  if (tid < kBars) tm::mbar_init(bar(tid), bar_count(tid, SW, KW));
  if (tid == 0) *dead = 0;
  if (warp == OW) tm::alloc_all(misc + kMiscTmem);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tm::fence_before();
  __syncthreads();
  tm::fence_after();
  // all of the tensor memory is this block's, so it starts at address 0: a constant,
  // which the matrix instructions (operands in uniform registers) are issued fastest from
  constexpr uint32_t tmem = 0;
  if (tm::lds32(misc + kMiscTmem) != tmem) {
    if (tid == 0) atomicOr(cv.status, (int)kFlagLayout);
    if (warp == OW) tm::dealloc_all(tm::lds32(misc + kMiscTmem));
    return;
  }
  pdl_trigger();

  Segment sg;
  uint32_t seg_n = 0;
  bool fail = false;

  if (warp < SW) {
    tm::regs_up<R::RS>();
    // =========================== softmax ===================================
    const int wg = warp >> 2, w = warp & 3, g = lane >> 2, qd = lane & 3;
    const int part = SUB * wg;  // first column of this warpgroup's in a chunk
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    const uint32_t sm_m = misc + kMiscM, sm_al = misc + kMiscAlpha + wg * 128, sm_red = misc + kMiscRed + wg * 1024;
    const float post0 = score_factor(tb, ta.scale);
    const int live_rows = ta.n_q << ta.log_group, words = (ta.n_q + 31) >> 5;
    const int units = cv.kv_heads * pl.blocks;
    float l[CPT][2 * NJ];  // this thread's part of the sums
    uint32_t n_tiles = 0;  // tiles of all segments before this one
    int buf = 0, ph = 0;   // score and weight buffer, its phase
    pdl_wait();
    while (true) {
      const bool more = next_segment(misc, seg_n, sg, fail, dead);
      if (tm::bar_or(1 + wg, 128, !more)) break;  // all four warps leave together
      const long unit = (long)sg.b * units + sg.unit;
      const int row0 = (sg.unit % pl.blocks) * pl.rows;
      // (the scale is a power of two: its division is exact.  0 stands for a unit of wild
      // rows, post < 0: its scores are finished one by one, in tensor memory)
      const float q_scale = reinterpret_cast<const float*>(ws + pl.ws_scale)[unit];
      const float post = q_scale == 0.f ? -1.f : post0 / q_scale;
      const int ctx = min(max(cv.seq_lens[sg.b], 0), cv.capacity) - ta.n_q;
      const uint32_t* mask = ta.mask ? ta.mask + sg.b * ta.mask_stride : nullptr;
      // column of the outputs (and maxima) of column i of this warpgroup's
      auto column = [&](int i) { return i / SUB * CN + part + i % SUB; };
      if ((tid & 127) < SUB * CPT) tm::stsf(sm_m + 4 * column(tid & 127), -kNoMax);
#pragma unroll
      for (int s = 0; s < CPT; ++s)
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j) l[s][j] = 0.f;
      tm::bar_sync(1 + wg, 128);

#pragma unroll 1
      for (int it = 0; it < sg.tiles; ++it) {
        const int slot = (n_tiles + it) % kMetaSlots, tok0 = sg.t0 + it * kTile + 32 * w + g;
        // (past a row's end as past its context: max_ctx may cut the row inside it; a wild
        // unit's tiles all take the masked ones' way)
        const bool masked = sg.t0 + (it + 1) * kTile > (post < 0.f ? 0 : min(ctx, sg.len));
        float kn[4], vn[4], ev[4];
#pragma unroll
        for (int chunk = 0; chunk < CPT; ++chunk) {
          const int col0 = chunk * CN + part;  // of the outputs and of the maxima
          const uint32_t t_s = tmem + pl.tm_s + buf * CN + part + lanes;
          fail = !tm::mbar_wait(bar(kBarSFull + buf), ph, dead) || fail;
          tm::fence_after();
          if (CPT == 1 || chunk == 0) {  // the tile's norms, which were there before its keys were
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint2 x = tm::lds64(pl.sm_meta + slot * 1024 + 8 * (32 * w + 8 * k + g));
              kn[k] = __uint_as_float(x.x) * post;
              vn[k] = __uint_as_float(x.y);
              ev[k] = fast_log2(vn[k] + 0x1p-30f);  // a zero norm gives -30
            }
          }
          float y[8 * NJ];
          uint32_t vis = 0xffffffffu;
          if (__builtin_expect(masked, 0)) {
            vis = visible<NJ>(tok0, sg.len, ctx, row0 + chunk * CN + part + 2 * qd, live_rows, ta.log_group, mask,
                              words);
            if (post < 0.f) {
              finish_scores(t_s, SUB, reinterpret_cast<const float*>(ws + pl.ws_rows) + unit * pl.rows + col0,
                            tm::ldsf(pl.sm_meta + slot * 1024 + 8 * (32 * w + lane)));
#pragma unroll
              for (int k = 0; k < 4; ++k) kn[k] = 1.f;
            }
          }
          // The running maximum (of score + log2 |v|, so that every weight p |v| stays
          // an fp16 number whatever the norms) moves only when a score passes it by that: in
          // a unit's first tile, afterwards almost never, and all four warps vote together.
          for (bool raise = it == 0;;) {
            if (__builtin_expect(raise, 0)) {
              // (the products complete in order: those of the chunk before are the last)
              const Raise r{t_s, tmem + lanes + col0, sm_m + 4 * col0, sm_al, sm_red,
                            (uint32_t)bar(kBarPEmpty + (buf == 0 ? pl.nsb - 1 : buf - 1)), vis,
                            (uint32_t)(buf == 0 ? ph ^ 1 : ph), wg, pl.rows, it > 0 && (D > 64 || w < 2) ? MB : 0};
              fail = !raise_max<NJ>(r, kn, ev, dead) || fail;
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                const uint2 x = tm::lds64(sm_al + 4 * (8 * j + 2 * qd));
                l[chunk][2 * j] *= __uint_as_float(x.x);
                l[chunk][2 * j + 1] *= __uint_as_float(x.y);
              }
            }
            float2 m2[NJ];
            tm::ld_16x256b(t_s, y);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint2 x = tm::lds64(sm_m + 4 * (col0 + 8 * j + 2 * qd));
              m2[j] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));  // (negated)
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
            if (raise) break;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float t = -INFINITY;
#pragma unroll
              for (int j = 0; j < NJ; ++j) t = fmaxf(fmaxf(t, y[y_at<NJ>(k, j)]), y[y_at<NJ>(k, j) + 1]);
              top = fmaxf(top, t + ev[k]);
            }
            raise = tm::bar_or(1 + wg, 128, top > kTreeLazyLog2);
            if (__builtin_expect(!raise, 1)) break;
          }
          // the scores are in registers: the next chunk's may come
          tm::fence_before();
          __syncwarp();
          if (lane == 0) tm::mbar_arrive(bar(kBarSEmpty + buf));
          fail = !tm::mbar_wait(bar(kBarPEmpty + buf), ph ^ 1, dead) || fail;
          // weight buffers: blocks of 64 columns, or halves of one when narrower
          const uint32_t sm_p = pl.sm_p + (CN >= 64 ? buf * (CN / 64) + part / 64 : 0) * 16384 + (32 * w + lane) * 128;
          const int piece = CN >= 64 ? part % 64 / 8 : 4 * buf + part / 8;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            uint32_t pk[4];
            float2 sum = make_float2(l[chunk][2 * j], l[chunk][2 * j + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = y_at<NJ>(k, j);
              const float2 p = make_float2(fast_exp2(y[i]), fast_exp2(y[i + 1]));
              sum = tm::add2(sum, p);
              const float2 wt = tm::mul2(p, make_float2(vn[k], vn[k]));
              const __half2 hw = __floats2half2_rn(wt.x, wt.y);
              pk[k] = *reinterpret_cast<const uint32_t*>(&hw);
            }
            l[chunk][2 * j] = sum.x;
            l[chunk][2 * j + 1] = sum.y;
            tm::stmatrix_x4(sm_p + (((piece + j) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
          tm::fence_proxy_async();
          tm::fence_before();
          __syncwarp();
          if (lane == 0) {
            tm::mbar_arrive(bar(kBarPFull + buf));
          }
          if (++buf == pl.nsb) buf = 0, ph ^= 1;
        }
      }
      n_tiles += sg.tiles;
      // ---- the unit's partial
      // (the products complete in order: those of the last chunk are the last)
      {
        const int last = buf == 0 ? pl.nsb - 1 : buf - 1;
        fail = !tm::mbar_wait(bar(kBarPEmpty + last), buf == 0 ? ph ^ 1 : ph, dead) || fail;
      }
      tm::fence_after();
      const long pcol = (blockIdx.x + unit) * pl.rows;  // first column of the partial
#pragma unroll
      for (int s = 0; s < CPT; ++s)
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j) {
          float x = l[s][j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (g == 0) tm::stsf(sm_red + 256 * w + 4 * (s * SUB + 8 * (j >> 1) + 2 * qd + (j & 1)), x);
        }
      tm::bar_sync(1 + wg, 128);
      const int i0 = tid & 127;
      if (i0 < SUB * CPT) {
        const float x = (tm::ldsf(sm_red + 4 * i0) + tm::ldsf(sm_red + 256 + 4 * i0)) +
                        (tm::ldsf(sm_red + 512 + 4 * i0) + tm::ldsf(sm_red + 768 + 4 * i0));
        reinterpret_cast<float2*>(ws + pl.ws_ml)[pcol + column(i0)] =
            make_float2(-tm::ldsf(sm_m + 4 * column(i0)), x);
      }
      if (D > 64 || w < 2) {
        float* wo = reinterpret_cast<float*>(ws) + pcol * D + 32 * w + lane;
#pragma unroll 1
        for (int i = 0; i < MB * CPT * (SUB / 16); ++i) {  // 16 columns at a time
          const int mb = i / (CPT * (SUB / 16)), c = 16 * (i % (CPT * (SUB / 16))), col = column(c);
          if (row0 + col >= live_rows) continue;  // (columns without rows)
          uint32_t o[16];
          tm::ld_32x32b(tmem + lanes + mb * pl.rows + col, o);
          tm::wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) wo[(col + e) * D + mb * 128] = __uint_as_float(o[e]);
        }
      }
      tm::fence_before();
    }
  } else if (warp < SW + KW) {
    tm::regs_down<R::RU>();
    // =========================== keys ======================================
    const int w = warp & 3, half = KW == 8 ? (warp >> 2) & 1 : 0, tok = 32 * w + lane, row_bytes = KB * D / 8;
    const uint32_t lut = pl.lut_k | (KB == 3 ? lane * 4 : KB == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
    const float sketch = AFF ? sqrtf(3.14159265358979f / (2.0f * D)) : sqrtf(3.14159265358979f / 2.0f) * tb.k_lam;
    uint32_t n = 0;  // tiles done
    int st = 0, st_ph = 0, kb = 0, k_ph = 0;
    while (next_segment(misc, seg_n, sg, fail, dead)) {
#pragma unroll 1
      for (int it = 0; it < sg.tiles; ++it, ++n) {
        const int slot = n % kMetaSlots;
        const uint32_t stage = pl.sm_st + st * pl.st_bytes;
        fail = !tm::mbar_wait(bar(kBarStFull + st), st_ph, dead);
        fail = !tm::mbar_wait(bar(kBarKEmpty + kb), k_ph ^ 1, dead) || fail;
        fail = __any_sync(0xffffffffu, fail);
        if (fail) break;
        const bool valid = sg.t0 + it * kTile + tok < sg.len;
        // ---- the token's norms
        float kn = 1.f, vn, ratio = 0.f;
        if (AFF) {
          uint32_t f = 1u;  // largest fp16 exponent field among the value's |scale|, |bias|
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const uint32_t x = tm::lds32(stage + pl.st_vn + (tok * NG + i) * 4);
            f = max(f, max((x >> 10) & 31u, (x >> 26) & 31u));
          }
          const int e = min((int)f, 29) - 15;
          vn = !valid ? 0.f : f == 31u ? __int_as_float(0x7fffffff) : __int_as_float((e + 127) << 23);
        } else {
          const uint32_t a = tm::lds_half(stage + pl.st_kn + 2 * tok), b = tm::lds_half(stage + pl.st_vn + 2 * tok);
          kn = __half2float(__ushort_as_half((uint16_t)a));
          vn = valid ? __half2float(__ushort_as_half((uint16_t)b)) : 0.f;
        }
        if (QJL) {
          // the sketch enters the reduction as its ratio to the key's norm; a norm below
          // 2^-14 of it is raised to that, where the codes no longer count
          const float r = sketch * __half2float(__ushort_as_half((uint16_t)tm::lds_half(stage + pl.st_rn + 2 * tok)));
          if (!AFF) {
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
          tm::sts64(pl.sm_meta + slot * 1024 + 8 * tok, __float_as_uint(kn), __float_as_uint(vn));
        }
        // ---- channels, then signs
        tm::fence_after();
        const uint32_t dst = tmem + pl.tm_k + kb * pl.kcols + ((uint32_t)(32 * w) << 16);
        unpack_blocks<CPT == 2, N, KB, D * KB % 128 == 0>(stage + tok * row_bytes + half * (N * KB * 4), lut, [&](int ci, uint32_t (&r)[16]) {
          const int c = half * N + ci;
          if (AFF) {
            const uint32_t x = tm::lds32(stage + pl.st_kn + (tok * NG + (c >> 1)) * 4);
            const uint32_t s = __byte_perm(x, x, 0x1010), b = __byte_perm(x, x, 0x3232);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = hfma2_bits(s, r[i], b);
          }
          tm::st_32x32b(dst + 16 * c, r);
        });
        if (QJL) {
          const uint32_t rr = pack_half2(__float2half_rn(ratio), __float2half_rn(ratio));
#pragma unroll 1
          for (int c = half * N; c < (half + 1) * N; ++c) {
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
  } else if (warp < OW) {
    tm::regs_down<R::RU>();
    // =========================== values ====================================
    const int w = warp & 3, half = KW == 8 ? (warp >> 2) & 1 : 0, tok = 32 * w + lane, row_bytes = VB * D / 8;
    const uint32_t lut = pl.lut_v | (VB == 3 ? lane * 4 : VB == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
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
        if (AFF) {
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
        unpack_blocks<CPT == 2, N, VB, D * VB % 128 == 0>(stage + pl.st_v + tok * row_bytes + half * (N * VB * 4), lut, [&](int ci, uint32_t (&r)[16]) {
          const int c = half * N + ci;
          if (AFF) {
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
    tm::regs_down<R::RO>();
    const uint32_t d_hi = tm::desc_hi(1024);
    if (warp == OW) {
      // ========================= scores ======================================
      const uint32_t id = tm::mma_idesc(CN, false, false), d_q = tm::desc_lo(pl.sm_q, 16);
      const uint32_t q_blk = pl.rows * 128 / 16, q_part = pl.rows * D * 2 / 16;
      const int code_parts = pl.parts - (QJL ? 1 : 0);
      uint32_t kb = 0, k_ph = 0, s_ph = 0, buf = 0;
      while (next_segment(misc, seg_n, sg, fail, dead)) {
        fail = !tm::mbar_wait(bar(kBarQFull), (seg_n - 1) & 1, dead);
#pragma unroll 1
        for (int t = 0; !fail && __any_sync(0xffffffffu, t < sg.tiles); ++t) {  // (votes: uniform to the compiler too)
          fail = !tm::mbar_wait(bar(kBarKFull + kb), k_ph, dead);
          const uint32_t a = tmem + pl.tm_k + kb * pl.kcols;
          uint32_t bq = d_q;
#pragma unroll 1
          for (int c = 0; c < CPT; ++c, bq += CN * 128 / 16) {
            fail = !tm::mbar_wait(bar(kBarSEmpty + buf), s_ph ^ 1, dead) || fail;
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
              tm::mbar_arrive(bar(kBarSFull + buf));  // (passes on what this warp saw of the keys' warps: the norms)
              if (c == CPT - 1) {
                tm::mma_commit(bar(kBarKEmpty + kb));
                if (t == sg.tiles - 1) tm::mma_commit(bar(kBarQEmpty));
              }
            }
            __syncwarp();
            if (++buf == (uint32_t)pl.nsb) buf = 0, s_ph ^= 1;
          }
          if (++kb == (uint32_t)pl.nkb) kb = 0, k_ph ^= 1;
        }
      }
    } else if (warp == OW + 1) {
      // ========================= outputs =====================================
      const uint32_t id = tm::mma_idesc(CN, true, true), d_v = tm::desc_lo(pl.sm_v, D == 64 ? 0 : 16384),
                     d_p = tm::desc_lo(pl.sm_p, 16384);
      uint32_t vb = 0, v_ph = 0, p_ph = 0, buf = 0;
      while (next_segment(misc, seg_n, sg, fail, dead)) {
#pragma unroll 1
        for (int t = 0; !fail && __any_sync(0xffffffffu, t < sg.tiles); ++t) {
          fail = !tm::mbar_wait(bar(kBarVFull + vb), v_ph, dead);
          const uint32_t acc = t > 0;  // the first of a unit's products overwrites
          uint32_t d = tmem;
#pragma unroll 1
          for (int c = 0; c < CPT; ++c, d += CN) {
            fail = !tm::mbar_wait(bar(kBarPFull + buf), p_ph, dead) || fail;
            tm::fence_after();
            if (lane == 0 && !fail) {
              const uint32_t b = d_p + buf * ((CN >= 64 ? CN / 64 * 16384 : 64) / 16);
#pragma unroll 1
              for (int mb = 0; mb < MB; ++mb) {
                const uint32_t a = d_v + vb * (kTile * D * 2 / 16) + mb * (2 * 16384 / 16), dm = d + mb * pl.rows;
                tm::mma_ss(dm, a, d_hi, b, d_hi, id, acc);
#pragma unroll
                for (int k = 1; k < kTile / 16; ++k)
                  tm::mma_ss(dm, a + k * (2048 / 16), d_hi, b + k * (2048 / 16), d_hi, id, 1);
              }
              tm::mma_commit(bar(kBarPEmpty + buf));
              if (c == CPT - 1) tm::mma_commit(bar(kBarVEmpty + vb));
            }
            __syncwarp();
            if (++buf == (uint32_t)pl.nsb) buf = 0, p_ph ^= 1;
          }
          if (++vb == (uint32_t)pl.nvb) vb = 0, v_ph ^= 1;
        }
      }
    } else if (warp == OW + 2) {
      // ========================= share, segments, packed tiles ===============
      // This block takes [t, t1) of the units' spans, T laid end to end.
      const int n_q = ta.n_q, max_ctx = ta.max_ctx, units = cv.kv_heads * pl.blocks;
      long long T = 0;
      for (int r = lane; r < cv.batch; r += 32) T += tree_span(cv, r, n_q, max_ctx);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
      T *= units;
      long long t = tile_bound(blockIdx.x, T, gridDim.x);
      const long long t1 = tile_bound((long long)blockIdx.x + 1, T, gridDim.x);
      long long rs = 0;  // spans before row b
      int b = 0;
      for (; b < cv.batch && t < t1; b += 32) {
        const int n = b + lane < cv.batch ? tree_span(cv, b + lane, n_q, max_ctx) : 0;
        long long e = n;  // spans up to and with this row
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
        const uint32_t k_row = KB * D / 8, v_row = VB * D / 8, meta = AFF ? 4 * NG : 2;
        int st = 0, st_ph = 0;
        uint32_t copies = 0;
        while (true) {
          Segment s{0, 0, 0, 0, 0};
          while (t < t1) {
            const int len = tree_len(cv, b, n_q, max_ctx), n = tree_span((len + kTile - 1) / kTile);
            const long long row = (long long)n * units;
            if (t >= rs + row) {
              rs += row;
              ++b;
              continue;
            }
            const long long at = t - rs;
            const int u = at < (1ll << 31) ? (int)((unsigned)at / (unsigned)n) : (int)(at / n);
            const long long us = rs + (long long)u * n, te = min(t1, us + n);
            // a unit's first places stand for its cost, its tiles follow
            const int lo = max((int)(t - us) - kUnitCost, 0), hi = (int)(te - us) - kUnitCost;
            t = te;
            if (hi <= lo) continue;
            s = Segment{b, u, lo * kTile, hi - lo, len};
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
            tm::mbar_expect(full, m * (k_row + v_row + 2 * meta + (QJL ? D / 8 + 2 : 0)));
            tm::bulk_load(dst, cv.k_codes + at * k_row, m * k_row, full);
            tm::bulk_load(dst + pl.st_kn, reinterpret_cast<const uint8_t*>(cv.k_norm) + at * meta, m * meta, full);
            tm::bulk_load(dst + pl.st_vn, reinterpret_cast<const uint8_t*>(cv.v_norm) + at * meta, m * meta, full);
            if (QJL) {
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
    if (warp < OW + 2 && fail && lane == 0) {  // after a failure the products in flight are waited for
      int never = 0;
      tm::mma_commit(bar(kBarDone + warp - OW));
      tm::mbar_wait_lane(bar(kBarDone + warp - OW), 0, &never);
    }
    __syncwarp();
  }
  tm::fence_before();
  __syncthreads();
  if (tid == 0 && *dead) atomicOr(cv.status, (int)kFlagTimeout);
  if (warp == OW) {
    tm::fence_after();
    tm::dealloc_all(tmem);
  }
}

// Whether a kernel's dynamic shared memory starts at kDynSmemBase on the current device
// (no static shared memory, that much reserved per block), as its plans assume.  Asked
// once per device: `known` holds a bit for each that is sound.
template <typename Kernel>
cudaError_t check_smem_base(Kernel kern, std::atomic<uint64_t>& known) {
  int dev = 0, reserved = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= KernelConfig::kMaxDevices) return cudaErrorInvalidDevice;
  if ((known.load(std::memory_order_relaxed) >> dev) & 1u) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  if (fa.sharedSizeBytes != 0 || reserved != (int)kDynSmemBase) return cudaErrorNotSupported;
  known.fetch_or(1ull << dev, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches the kernel of one compile-time shape (the rest of *cfg is set); without cfg,
// only makes sure that it can be launched.
template <int D, int CN, int CPT, int KB, int VB, bool QJL, bool AFF>
cudaError_t launch_tree_shape(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                              cudaLaunchConfig_t* cfg) {
  static KernelConfig config;
  static std::atomic<uint64_t> at_base{0};
  static_assert(KernelConfig::kMaxDevices <= 64, "a bit per device");
  auto kern = tree_kernel<D, CN, CPT, KB, VB, QJL, AFF>;
  cudaError_t e = check_smem_base(kern, at_base);
  if (e != cudaSuccess) return e;
  // the attribute is set once per device, for the largest plan
  e = configure_kernel(config, kern, 227 * 1024, Roles<D, CN>::THREADS, nullptr);
  if (e != cudaSuccess || !cfg) return e;
  cfg->blockDim = dim3(Roles<D, CN>::THREADS);
  return cudaLaunchKernelEx(cfg, kern, tb, cv, ta, pl, ws);
}

// Per-head-dim, per-codec dispatch over shape and code widths; instantiated in the
// tq_tree_*.cu translation units.
template <int D, bool AFF, bool QJL>
cudaError_t launch_tree_dim(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                            cudaLaunchConfig_t* cfg);

template <int D, bool AFF, bool QJL, int CN, int CPT>
cudaError_t dispatch_tree_bits(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                               cudaLaunchConfig_t* cfg) {
#define TQ_BITS(KB, VB) \
  if (tb.k_bits == KB && tb.v_bits == VB) return launch_tree_shape<D, CN, CPT, KB, VB, QJL, AFF>(tb, cv, ta, pl, ws, cfg);
  TQ_BITS(2, 2) TQ_BITS(2, 3) TQ_BITS(3, 3) TQ_BITS(3, 4) TQ_BITS(4, 4)
#undef TQ_BITS
  return cudaErrorNotSupported;
}

template <int D, bool AFF, bool QJL>
cudaError_t dispatch_tree_dim(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, uint8_t* ws,
                              cudaLaunchConfig_t* cfg) {
  if (pl.cn == 16) return dispatch_tree_bits<D, AFF, QJL, 16, 1>(tb, cv, ta, pl, ws, cfg);
  if (pl.cn == 32) return dispatch_tree_bits<D, AFF, QJL, 32, 1>(tb, cv, ta, pl, ws, cfg);
  if (pl.cn == 64) return dispatch_tree_bits<D, AFF, QJL, 64, 1>(tb, cv, ta, pl, ws, cfg);
  if constexpr (D < 256) {
    if (pl.chunks == 1) return dispatch_tree_bits<D, AFF, QJL, 128, 1>(tb, cv, ta, pl, ws, cfg);
    return dispatch_tree_bits<D, AFF, QJL, 128, 2>(tb, cv, ta, pl, ws, cfg);
  }
  return cudaErrorNotSupported;
}

}  // namespace tq
