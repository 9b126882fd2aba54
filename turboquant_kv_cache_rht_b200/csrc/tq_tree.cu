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
//   warps 8-11  keys: a thread unpacks its token's codes through a table of code
//               pairs into its lane of tensor memory, the product's A operand
//               (no shared-memory round trip, no swizzle);
//   warps 12-15 values: the same into shared memory, token rows of 64 channels;
//   warp 16     issues the matrix instructions;
//   warp 17     copies the packed tiles in, a few stages ahead.
// A key's norm multiplies its scores, a value's norm its weights, both fp32, in
// the softmax; so the fp16 operands hold centroids (scaled by k_lam / v_lam, at
// which they are nearly exact) and lose nothing.  The sketch's signs follow the
// key's channels in the reduction, as +- rnorm / norm, against a second table of
// rotated queries; an fp16 call holds its queries in two fp16 parts (hi + lo).
// The affine codec's operands are scale * level + bias, rounded to fp16.
//
// The token tiles of all (batch row, KV head, block of query rows) units are laid
// end to end and each block takes an equal share, as in the decode; a unit that
// a block meets leaves a partial (O, maximum, sum) in the workspace, and a second
// kernel merges them and rotates back.
#include "tq_decode_impl.cuh"
#include "tq_tmem.cuh"

#include <algorithm>
#include <vector>

namespace tq {
namespace {

constexpr int kTile = 128;          // tokens per tile: the matrix instruction's rows
constexpr int kTreeThreads = 576;   // 18 warps: 112 registers a thread
constexpr int kTreeMaxCtas = 148;   // one block per SM; the workspace is sized for it
constexpr int kMetaSlots = 4;       // tiles whose norms are in flight
constexpr int kMaxStages = 4;
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
  int ctas;
  long slots;
};

// Shared misc area: barriers, then floats.
constexpr int kBarQ = 0, kBarStFull = 1, kBarStEmpty = kBarStFull + kMaxStages, kBarKFull = kBarStEmpty + kMaxStages,
              kBarKEmpty = kBarKFull + 2, kBarVFull = kBarKEmpty + 2, kBarVEmpty = kBarVFull + 2,
              kBarSFull = kBarVEmpty + 2, kBarSEmpty = kBarSFull + 2, kBarPFull = kBarSEmpty + 2,
              kBarPEmpty = kBarPFull + 2, kBarMetaFull = kBarPEmpty + 2, kBarMetaEmpty = kBarMetaFull + kMetaSlots,
              kBarDone = kBarMetaEmpty + kMetaSlots, kBars = kBarDone + 1;
constexpr int kMiscTmem = kBars * 8, kMiscDead = kMiscTmem + 4, kMiscScan = kMiscTmem + 16,  // scan: 18 x 8 + 24
              kMiscM = kMiscScan + 192,                  // running maxima [256]
              kMiscAlpha = kMiscM + 1024,                // rescale factors [2][64]
              kMiscRed = kMiscAlpha + 512,               // [2][4][128]
              kMiscFlag = kMiscRed + 4096,               // [2][4] failures
              kMiscBytes = kMiscFlag + 64;

struct Segment {
  int b, unit, t0, tiles, len;  // row, unit of the row, first token, tiles, tokens of the row
};

// Walks the units whose tiles meet [t, t1).
struct Walk {
  const CacheView* cv;
  int n_q, max_ctx, units;  // units per row
  int b;
  long long rs, t, t1;      // tiles before row b; position
  __device__ __forceinline__ int length(int r) const {
    const int stored = min(max(cv->seq_lens[r], 0), cv->capacity);
    return stored < n_q ? 0 : min(stored, max_ctx);
  }
  __device__ __forceinline__ bool next(Segment& s) {
    while (t < t1) {
      const int len = length(b), n = (len + kTile - 1) / kTile;
      if (n == 0 || t >= rs + (long long)n * units) {
        rs += (long long)n * units;
        ++b;
        continue;
      }
      const int u = (int)((t - rs) / n);
      const long long us = rs + (long long)u * n, te = min(t1, us + n);
      s = Segment{b, u, (int)(t - us) * kTile, (int)(te - t), len};
      t = te;
      return true;
    }
    return false;
  }
};

// 64 channels of a packed row at shared address `row` -> 32 fp16 pairs.
template <int BITS>
__device__ __forceinline__ void unpack64(uint32_t row, uint32_t lut, uint32_t (&r)[32]) {
  uint32_t w[2 * BITS];
  if constexpr (BITS == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint2 x = tm::lds64(row + 8 * i);
      w[2 * i] = x.x;
      w[2 * i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
      const uint4 x = tm::lds128(row + 16 * i);
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  }
  if constexpr (BITS == 2) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // a byte of four codes, entries 128 bytes apart
      const uint2 x = tm::lut64(bits_at(w[i >> 2], 8 * (i & 3), 8, 7) | lut);
      r[2 * i] = x.x;
      r[2 * i + 1] = x.y;
    }
  } else if constexpr (BITS == 3) {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = tm::lut32(field_scaled(w, 6, 6 * i, 6, 7) | lut);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = tm::lut32(bits_at(w[i >> 2], 8 * (i & 3), 8, 6) | lut);
  }
}

__device__ __forceinline__ void unpack64(int bits, uint32_t row, uint32_t lut, uint32_t (&r)[32]) {
  if (bits == 2) unpack64<2>(row, lut, r);
  else if (bits == 3) unpack64<3>(row, lut, r);
  else unpack64<4>(row, lut, r);
}

// Fills a table with every lane's copy of every entry.
__device__ __forceinline__ void fill_lut(uint32_t lut, int bits, const float* cent, float lam) {
  auto h = [&](int c) { return __half2float(__float2half_rn(cent[c] * lam)); };
  auto pair = [&](int a, int b) { return pack_half2(__float2half_rn(h(a)), __float2half_rn(h(b))); };
  if (bits == 2) {
    for (int i = threadIdx.x; i < 256 * 8; i += kTreeThreads) {
      const int p = i >> 3;
      const uint32_t x = pair(p & 3, (p >> 2) & 3), y = pair((p >> 4) & 3, p >> 6);
      tm::sts128(lut + 16 * i, x, y, x, y);
    }
  } else {
    const int per = bits == 3 ? 8 : 4, entries = 1 << (2 * bits);  // 16-byte pieces of an entry
    for (int i = threadIdx.x; i < entries * per; i += kTreeThreads) {
      const int p = i / per;
      const uint32_t x = pair(p & ((1 << bits) - 1), p >> bits);
      tm::sts128(lut + 16 * i, x, x, x, x);
    }
  }
}

// Sum of one value per thread over the block (all threads call), the sums of
// the threads before in *before.
__device__ __forceinline__ long long block_scan(long long x, long long* scratch, long long* before) {
  return block_exclusive_scan<kTreeThreads>(x, scratch, before);
}

template <int D, int CN, int CPW>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ Tables tb, const __grid_constant__ CacheView cv,
                const __grid_constant__ TreeArgs ta, const __grid_constant__ TreePlan pl, float* __restrict__ ws) {
  constexpr int SUB = CN < 32 ? CN : 32;   // columns a warpgroup holds at a time
  constexpr int NSUB = CN / SUB, NJ = SUB / 8;
  constexpr int MB = D == 256 ? 2 : 1;     // 128-channel blocks of the output
  constexpr int NG = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t misc = pl.sm_misc;
  if ((uint32_t)__cvta_generic_to_shared(smem) != kDynSmemBase) {  // the plan's addresses assume it
    if (tid == 0) atomicOr(cv.status, (int)kFlagLayout);
    return;
  }
  auto at = [&](uint32_t a) { return smem + (a - kDynSmemBase); };
  auto bar = [&](int i) { return misc + 8 * i; };
  volatile int* dead = reinterpret_cast<volatile int*>(at(misc + kMiscDead));
  const bool split = pl.chunks == 1;

  // ---- setup that needs nothing of the previous kernel
  fill_lut(pl.lut_k, tb.k_bits, tb.k_cent, tb.k_lam);
  if (pl.lut_v != pl.lut_k) fill_lut(pl.lut_v, tb.v_bits, tb.v_cent, tb.v_lam);
  if (tid == 0) {
    *dead = 0;
    tm::mbar_init(bar(kBarQ), 8);
    tm::mbar_init(bar(kBarDone), 1);
    for (int i = 0; i < kMaxStages; ++i) {
      tm::mbar_init(bar(kBarStFull + i), 1);
      tm::mbar_init(bar(kBarStEmpty + i), 8);
    }
    for (int i = 0; i < 2; ++i) {
      tm::mbar_init(bar(kBarKFull + i), 4);
      tm::mbar_init(bar(kBarKEmpty + i), 1);
      tm::mbar_init(bar(kBarVFull + i), 4);
      tm::mbar_init(bar(kBarVEmpty + i), 1);
      tm::mbar_init(bar(kBarSFull + i), 1);
      tm::mbar_init(bar(kBarSEmpty + i), 4);
      tm::mbar_init(bar(kBarPFull + i), 4);
      tm::mbar_init(bar(kBarPEmpty + i), 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) {
      tm::mbar_init(bar(kBarMetaFull + i), 4);
      tm::mbar_init(bar(kBarMetaEmpty + i), split ? 4 : 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tm::alloc_all(misc + kMiscTmem);
  pdl_wait();

  // ---- this block's tiles [t0, t1) of the T laid end to end over all units
  Walk walk{&cv, ta.n_q, ta.max_ctx, cv.kv_heads * pl.blocks, 0, 0, 0, 0};
  {
    long long* scan = reinterpret_cast<long long*>(at(misc + kMiscScan));
    long long* found = scan + kTreeThreads / 32;  // first row, its prefix
    long long T = 0;
    for (int b0 = 0; b0 < cv.batch; b0 += kTreeThreads) {
      const int r = b0 + tid;
      long long tot;
      block_scan(r < cv.batch ? (walk.length(r) + kTile - 1) / kTile : 0, scan, &tot);
      T += tot;
    }
    T *= walk.units;
    walk.t = tile_bound(blockIdx.x, T, gridDim.x);
    walk.t1 = tile_bound((long long)blockIdx.x + 1, T, gridDim.x);
    long long base = 0;
    for (int b0 = 0; b0 < cv.batch && base <= walk.t; b0 += kTreeThreads) {
      const int r = b0 + tid;
      long long tot;
      const long long n = r < cv.batch ? (walk.length(r) + kTile - 1) / kTile : 0;
      const long long p = base + block_scan(n, scan, &tot) * walk.units, e = p + n * walk.units;
      if (p <= walk.t && walk.t < e) {
        found[0] = r;
        found[1] = p;
      }
      base += tot * walk.units;
    }
    tm::fence_before();
    __syncthreads();
    tm::fence_after();
    if (walk.t < walk.t1) {
      walk.b = (int)found[0];
      walk.rs = found[1];
    }
  }
  const uint32_t tmem = tm::lds32(misc + kMiscTmem);
  if (blockIdx.x == 0)
    for (int r = tid; r < cv.batch; r += kTreeThreads)
      if (min(max(cv.seq_lens[r], 0), cv.capacity) > ta.max_ctx) atomicOr(cv.status, (int)kFlagMaxCtx);
  pdl_trigger();

  Segment sg;
  const int group = ta.q_heads / cv.kv_heads, live_rows = ta.n_q * group;
  bool fail = false;

  if (warp < 8) {
    // =========================== softmax ===================================
    const int wg = warp >> 2, w = warp & 3, g = lane >> 2, qd = lane & 3;
    const uint32_t lanes = (uint32_t)(32 * w) << 16;
    const uint32_t t_s = tmem + pl.tm_s + wg * CN + lanes, sm_p = pl.sm_p + wg * 16384;
    const uint32_t sm_m = misc + kMiscM, sm_al = misc + kMiscAlpha + wg * 256, sm_red = misc + kMiscRed + wg * 2048;
    const uint32_t sm_flag = misc + kMiscFlag + wg * 16;
    const float scale_log2 = ta.scale * 1.4426950408889634f;
    float l[CPW][NSUB][2 * NJ];
    uint32_t n_items = 0, n_tiles = 0;  // chunks done, tiles of all segments before this one
    bool over = false;
    while (walk.next(sg)) {
      // both warpgroups are done with the last segment's queries and scratch; a
      // failure of either ends both
      if (tm::bar_or(3, 256, over || fail)) break;
      const int kvh = sg.unit / pl.blocks, rb = sg.unit - kvh * pl.blocks, row0 = rb * pl.rows;
      // ---- queries: rotate, scale by a power of two, round to fp16 tables.  Eight
      // lanes hold a row (D/8 channels each); the scale is 1 unless the largest entry
      // is far from fp16's range, then it is measured and the rows are done again.
      float qscale = 1.f;
      for (int pass = 0; pass < 2; ++pass) {
        constexpr int E = D / 8;
        float amax = 0.f;
        for (int rr = 4 * warp + (lane >> 3); rr < pl.rows; rr += 32) {
          const int r = row0 + rr, c0 = (lane & 7) * E;
          float u[E];
          if (r < live_rows) {
            const int i = r / group, h = kvh * group + (r - i * group);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(ta.q) +
                                                              (((long)sg.b * ta.n_q + i) * ta.q_heads + h) * D + c0);
#pragma unroll
            for (int e = 0; e < E / 8; ++e) {
              const uint4 x = src[e];
              const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = ta.dtype == kBF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&y[k]))
                                                   : __half22float2(*reinterpret_cast<const __half2*>(&y[k]));
                u[8 * e + 2 * k] = f.x;
                u[8 * e + 2 * k + 1] = f.y;
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = 0.f;
          }
          auto signs = [&](const uint32_t* s, float by) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int c = c0 + e;
              u[e] *= ((s[c >> 5] >> (c & 31)) & 1u) ? -by : by;
            }
          };
          auto fwht = [&]() {
#pragma unroll
            for (int h = 1; h < E; h <<= 1)
#pragma unroll
              for (int j = 0; j < E; ++j)
                if ((j & h) == 0) {
                  const float a = u[j], c = u[j + h];
                  u[j] = a + c;
                  u[j + h] = a - c;
                }
#pragma unroll
            for (int m = 1; m < 8; m <<= 1)
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const float p = __shfl_xor_sync(0xffffffffu, u[e], m);
                u[e] = (lane & m) ? p - u[e] : u[e] + p;
              }
          };
          float top = 0.f;
          auto measure = [&]() {
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(u[e]));
          };
          const uint32_t qrow = pl.sm_q + rr * 128;
          signs(tb.s1, qscale);
          fwht();
          measure();
#pragma unroll
          for (int e = 0; e < E / 8; ++e) {
            const int c = c0 + 8 * e;
            const uint32_t a = qrow + (c >> 6) * (pl.rows * 128) + ((((c >> 3) & 7) ^ (rr & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) split_pair(u[8 * e + 2 * k], u[8 * e + 2 * k + 1], hi[k], lo[k]);
            tm::sts128(a, hi[0], hi[1], hi[2], hi[3]);
            if (ta.dtype == kF16) tm::sts128(a + pl.rows * D * 2, lo[0], lo[1], lo[2], lo[3]);
          }
          if (tb.qjl) {
            // channels j and j + 16 of a 32-channel word are neighbours in the reduction
            signs(tb.s2, 1.f / sqrtf((float)D));
            fwht();
            measure();
            const uint32_t base = qrow + (pl.parts - 1) * (pl.rows * D * 2);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int c = c0 + e, j = c & 31, pos = (c & ~31) + (j < 16 ? 2 * j : 2 * (j - 16) + 1);
              tm::sts16(base + (pos >> 6) * (pl.rows * 128) + ((((pos >> 3) & 7) ^ (rr & 7)) << 4) + (pos & 7) * 2,
                        __half_as_ushort(__float2half_rn(u[e])));
            }
          }
#pragma unroll
          for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
          if (top < INFINITY) amax = fmaxf(amax, top);  // a row with infinities keeps them to itself
        }
        if (pass == 1) break;
#pragma unroll
        for (int m = 8; m < 32; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        if (lane == 0) tm::stsf(misc + kMiscRed + 4 * warp, amax);
        tm::bar_sync(3, 256);
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, tm::ldsf(misc + kMiscRed + 4 * k));
        tm::bar_sync(3, 256);
        if (amax == 0.f || (amax >= 1.f && amax <= 16384.f)) break;
        int e;
        frexpf(amax, &e);
        qscale = ldexpf(1.f, max(min(13 - e, 100), -100));
      }
      for (int i = tid & 127; i < (split ? CN : CN * CPW); i += 128) {
        const int c = i / CN, col = split ? wg * CN + i : (2 * c + wg) * CN + (i - c * CN);
        tm::stsf(sm_m + 4 * col, kNoMax);
      }
      tm::fence_proxy_async();
      tm::fence_before();
      tm::bar_sync(1 + wg, 128);
      if (lane == 0) tm::mbar_arrive(bar(kBarQ));
#pragma unroll
      for (int c = 0; c < CPW; ++c)
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
          for (int j = 0; j < 2 * NJ; ++j) l[c][s][j] = 0.f;
      // scores: undoes the query's scale, folds softmax scale, log2(e) and the
      // 1/sqrt(d) of the rotation (and of the dequantization)
      const float post = tb.affine ? scale_log2 / (sqrtf((float)D) * qscale)
                                   : scale_log2 / ((float)D * qscale * tb.k_lam);
      const int ctx = min(max(cv.seq_lens[sg.b], 0), cv.capacity) - ta.n_q;
      const uint32_t* mask = ta.mask ? ta.mask + sg.b * ta.mask_stride : nullptr;
      const int words = (ta.n_q + 31) >> 5;

      for (int it = split ? wg : 0; it < sg.tiles && !over; it += split ? 2 : 1) {
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
#pragma unroll
        for (int cc = 0; cc < CPW; ++cc) {
          if (over) break;
          const int chunk = split ? 0 : 2 * cc + wg;
          const int col0 = split ? wg * CN : chunk * CN;   // of O and of the maxima
          fail = !tm::mbar_wait(bar(kBarSFull + wg), n_items & 1, dead) || fail;
          tm::fence_after();
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub) {
            if (over) break;
            float y[8 * NJ];  // 4 tokens x 2 NJ columns: (k, j, c) at index below
            float2 m2[NJ];
            const uint32_t a_m = sm_m + 4 * (col0 + sub * SUB + 2 * qd);
            auto at_y = [&](int k, int j) { return (k >> 1) * 4 * NJ + 4 * j + 2 * (k & 1); };
            auto get = [&](int k, int j) { return make_float2(y[at_y(k, j)], y[at_y(k, j) + 1]); };
            auto put = [&](int k, int j, float2 x) {
              y[at_y(k, j)] = x.x;
              y[at_y(k, j) + 1] = x.y;
            };
            tm::ld_16x256b(t_s + sub * SUB, y);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint2 x = tm::lds64(a_m + 32 * j);
              m2[j] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
            }
            tm::wait_ld(y);
            // hides what a row does not attend (tiles past the context only)
            auto hide = [&]() {
#pragma unroll
              for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const int r = row0 + chunk * CN + sub * SUB + 8 * j + 2 * qd + c, i = r / group;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const int t = tok0 + 8 * k, dj = t - ctx;
                    bool sees = t < sg.len && r < live_rows;
                    if (sees && dj >= 0) sees = mask ? (mask[i * words + (dj >> 5)] >> (dj & 31)) & 1u : dj <= i;
                    if (!sees) y[at_y(k, j) + c] = -INFINITY;
                  }
                }
            };
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int j = 0; j < NJ; ++j)
                put(k, j, tm::fma2(get(k, j), make_float2(kn[k], kn[k]), make_float2(-m2[j].x, -m2[j].y)));
            }
            if (masked) hide();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float t = -INFINITY;
#pragma unroll
              for (int j = 0; j < NJ; ++j) t = fmaxf(fmaxf(t, get(k, j).x), get(k, j).y);
              top = fmaxf(top, t + ev[k]);
            }
            // The running maximum (of score + log2 |v|, so that every weight p |v| stays
            // below 2^8 whatever the norms) moves only when a score passes it by 2^8:
            // after the first tiles almost never, and all four warps vote together.
            if (tm::bar_or(1 + wg, 128, top > kLazyLog2 || fail)) {
              const uint32_t a_red = sm_red + 4 * (2 * qd);
              fail = !tm::mbar_wait(bar(kBarPEmpty + wg), (n_items & 1) ^ 1, dead) || fail;
              tm::ld_16x256b(t_s + sub * SUB, y);
              tm::wait_ld(y);
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < NJ; ++j) put(k, j, tm::mul2(get(k, j), make_float2(kn[k], kn[k])));
              if (masked) hide();
#pragma unroll
              for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float x = -INFINITY;
#pragma unroll
                  for (int k = 0; k < 4; ++k) x = fmaxf(x, y[at_y(k, j) + c] + ev[k]);
#pragma unroll
                  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                  if (g == 0) tm::stsf(a_red + 512 * w + 4 * (8 * j + c), x);
                }
              fail = __any_sync(0xffffffffu, fail);
              if (lane == 0) tm::stsf(sm_flag + 4 * w, fail ? 1.f : 0.f);
              tm::bar_sync(1 + wg, 128);
#pragma unroll
              for (int k = 0; k < 4; ++k) over = over || tm::ldsf(sm_flag + 4 * k) != 0.f;
              float al[2 * NJ];
#pragma unroll
              for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const float old = c ? m2[j].y : m2[j].x;
                  float mn = old;
#pragma unroll
                  for (int k = 0; k < 4; ++k) mn = fmaxf(mn, tm::ldsf(a_red + 512 * k + 4 * (8 * j + c)));
                  al[2 * j + c] = fast_exp2(old - mn);
                  l[cc][sub][2 * j + c] *= al[2 * j + c];
                  (c ? m2[j].y : m2[j].x) = mn;
                }
              tm::bar_sync(1 + wg, 128);
              if (w == 0 && g == 0) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    tm::stsf(a_m + 32 * j + 4 * c, c ? m2[j].y : m2[j].x);
                    tm::stsf(sm_al + 4 * (8 * j + 2 * qd + c), al[2 * j + c]);
                  }
              }
              tm::bar_sync(1 + wg, 128);
              if (it > (split ? wg : 0) && (D > 64 || w < 2)) {  // the products so far, rescaled
                tm::fence_after();
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                  for (int h = 0; h < SUB / 16; ++h) {
                    uint32_t o[16];
                    const uint32_t a = tmem + lanes + mb * pl.cols + col0 + sub * SUB + 16 * h;
                    tm::ld_32x32b(a, o);
                    tm::wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      o[i] = __float_as_uint(__uint_as_float(o[i]) * tm::ldsf(sm_al + 4 * (16 * h + i)));
                    tm::st_32x32b(a, o);
                  }
                tm::wait_st();
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                  put(k, j, tm::add2(get(k, j), make_float2(-m2[j].x, -m2[j].y)));
            }
            if (sub == NSUB - 1) {  // the scores are in registers: the next chunk's may come
              tm::fence_before();
              __syncwarp();
              if (lane == 0) tm::mbar_arrive(bar(kBarSEmpty + wg));
            }
            if (sub == 0) fail = !tm::mbar_wait(bar(kBarPEmpty + wg), (n_items & 1) ^ 1, dead) || fail;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              uint32_t pk[4];
              float2 sum = make_float2(l[cc][sub][2 * j], l[cc][sub][2 * j + 1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 x = get(k, j);
                const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                sum = tm::add2(sum, p);
                float2 wt = tm::mul2(p, make_float2(vn[k], vn[k]));
                if (masked) {  // a hidden value's norm may be anything
                  if (x.x == -INFINITY) wt.x = 0.f;
                  if (x.y == -INFINITY) wt.y = 0.f;
                }
                const __half2 hw = __floats2half2_rn(wt.x, wt.y);
                pk[k] = *reinterpret_cast<const uint32_t*>(&hw);
              }
              l[cc][sub][2 * j] = sum.x;
              l[cc][sub][2 * j + 1] = sum.y;
              tm::stmatrix_x4(sm_p + (32 * w + lane) * 128 + (((sub * NJ + j) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2],
                              pk[3]);
            }
          }
          tm::fence_proxy_async();
          tm::fence_before();
          __syncwarp();
          if (lane == 0) tm::mbar_arrive(bar(kBarPFull + wg));
          ++n_items;
        }
      }
      if (over) continue;
      n_tiles += sg.tiles;
      // ---- the unit's partial
      fail = !tm::mbar_wait(bar(kBarPEmpty + wg), (n_items & 1) ^ 1, dead) || fail;
      tm::fence_after();
      const bool any = !split || wg < sg.tiles;
      const long pslot = blockIdx.x + (long)sg.b * walk.units + sg.unit;
      float* wo = ws + pslot * pl.cols * D;
      float* wml = ws + pl.slots * pl.cols * D + pslot * pl.cols * 2;
#pragma unroll
      for (int cc = 0; cc < CPW; ++cc)
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
          for (int j = 0; j < 2 * NJ; ++j) {
            float x = l[cc][s][j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (g == 0) tm::stsf(sm_red + 512 * w + 4 * (cc * CN + s * SUB + 8 * (j >> 1) + 2 * qd + (j & 1)), x);
          }
      tm::bar_sync(1 + wg, 128);
      for (int i = tid & 127; i < CN * CPW; i += 128) {
        const int cc = i / CN, chunk = split ? 0 : 2 * cc + wg, col = (split ? wg : chunk) * CN + (i - cc * CN);
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) x += tm::ldsf(sm_red + 512 * k + 4 * i);
        wml[2 * col] = tm::ldsf(sm_m + 4 * col);
        wml[2 * col + 1] = any ? x : 0.f;
      }
      if (any && (D > 64 || w < 2)) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int cc = 0; cc < CPW; ++cc) {
            const int chunk = split ? 0 : 2 * cc + wg, col = (split ? wg : chunk) * CN;
            const int live = min(CN, live_rows - row0 - chunk * CN);
#pragma unroll
            for (int h = 0; h < CN / 16; ++h) {
              if (16 * h >= live) break;
              uint32_t o[16];
              tm::ld_32x32b(tmem + lanes + mb * pl.cols + col + 16 * h, o);
              tm::wait_ld(o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (16 * h + i < live)
                  wo[(long)(col + 16 * h + i) * D + mb * 128 + 32 * w + lane] = __uint_as_float(o[i]);
            }
          }
      }
      tm::fence_before();
    }
  } else if (warp < 12) {
    // =========================== keys ======================================
    const int w = warp & 3, tok = 32 * w + lane, row_bytes = tb.k_bits * D / 8;
    const uint32_t lut = pl.lut_k | (tb.k_bits == 3 ? lane * 4 : tb.k_bits == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
    const float sketch = tb.affine ? sqrtf(3.14159265358979f / (2.0f * D)) : sqrtf(3.14159265358979f / 2.0f) * tb.k_lam;
    uint32_t n = 0;  // tiles done
    int st = 0, st_ph = 0;
    while (!fail && walk.next(sg)) {
      for (int it = 0; it < sg.tiles; ++it, ++n) {
        const int slot = n % kMetaSlots, kb = n % pl.nkb;
        const uint32_t stage = pl.sm_st + st * pl.st_bytes;
        fail = !tm::mbar_wait(bar(kBarStFull + st), st_ph, dead);
        fail = !tm::mbar_wait(bar(kBarMetaEmpty + slot), ((n / kMetaSlots) & 1) ^ 1, dead) || fail;
        fail = !tm::mbar_wait(bar(kBarKEmpty + kb), ((n / pl.nkb) & 1) ^ 1, dead) || fail;
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
        const uint32_t a_meta = pl.sm_meta + slot * 1536 + 4 * tok;
        tm::stsf(a_meta, kn);
        tm::stsf(a_meta + 512, vn);
        tm::stsf(a_meta + 1024, ev);
        __syncwarp();
        if (lane == 0) tm::mbar_arrive(bar(kBarMetaFull + slot));
        // ---- channels, then signs
        tm::fence_after();
        const uint32_t dst = tmem + pl.tm_k + kb * pl.kcols + ((uint32_t)(32 * w) << 16);
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          uint32_t r[32];
          unpack64(tb.k_bits, stage + tok * row_bytes + gi * 8 * tb.k_bits, lut, r);
          if (tb.affine) {
            const uint32_t x = tm::lds32(stage + pl.st_kn + (tok * NG + gi) * 4);
            const uint32_t s = __byte_perm(x, x, 0x1010), b = __byte_perm(x, x, 0x3232);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = hfma2_bits(s, r[i], b);
          }
          tm::st_32x32b(dst + 32 * gi, r);
        }
        if (tb.qjl) {
          const uint32_t rr = pack_half2(__float2half_rn(ratio), __float2half_rn(ratio));
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) {
            const uint2 x = tm::lds64(stage + pl.st_s + tok * (D / 8) + 8 * gi);
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // bit 1: +
              r[j] = rr ^ ((~x.x << (15 - j)) & 0x80008000u);
              r[16 + j] = rr ^ ((~x.y << (15 - j)) & 0x80008000u);
            }
            tm::st_32x32b(dst + D / 2 + 32 * gi, r);
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
      }
    }
  } else if (warp < 16) {
    // =========================== values ====================================
    const int w = warp & 3, tok = 32 * w + lane, row_bytes = tb.v_bits * D / 8;
    const uint32_t lut = pl.lut_v | (tb.v_bits == 3 ? lane * 4 : tb.v_bits == 2 ? (lane & 15) * 8 : (lane & 15) * 4);
    uint32_t n = 0;
    int st = 0, st_ph = 0;
    while (!fail && walk.next(sg)) {
      for (int it = 0; it < sg.tiles; ++it, ++n) {
        const int vb = n % pl.nvb;
        const uint32_t stage = pl.sm_st + st * pl.st_bytes;
        fail = !tm::mbar_wait(bar(kBarStFull + st), st_ph, dead);
        fail = !tm::mbar_wait(bar(kBarVEmpty + vb), ((n / pl.nvb) & 1) ^ 1, dead) || fail;
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
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          uint32_t r[32];
          unpack64(tb.v_bits, stage + pl.st_v + tok * row_bytes + gi * 8 * tb.v_bits, lut, r);
          if (tb.affine) {
            const uint32_t x = hmul2_bits(tm::lds32(stage + pl.st_vn + (tok * NG + gi) * 4), mul);
            const uint32_t s = __byte_perm(x, x, 0x1010), b = __byte_perm(x, x, 0x3232);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = sound ? hfma2_bits(s, r[i], b) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            tm::sts128(dst + gi * 16384 + ((i ^ (tok & 7)) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
        tm::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          tm::mbar_arrive(bar(kBarStEmpty + st));
          tm::mbar_arrive(bar(kBarVFull + vb));
        }
        if (++st == pl.nst) st = 0, st_ph ^= 1;
      }
    }
  } else if (warp == 16) {
    // =========================== matrix instructions =======================
    if (lane == 0) {
      const uint32_t id_s = tm::mma_idesc(CN, false, false), id_o = tm::mma_idesc(CN, true, true);
      const uint64_t d_q = tm::mma_desc(pl.sm_q, 16, 1024);
      const uint64_t d_v = tm::mma_desc(pl.sm_v, D == 64 ? 0 : 16384, 1024);
      const uint64_t d_p = tm::mma_desc(pl.sm_p, 16, 1024);
      const uint32_t q_blk = pl.rows * 128 / 16, q_part = pl.rows * D * 2 / 16;
      const int code_parts = pl.parts - (tb.qjl ? 1 : 0);
      uint32_t n = 0, items = 0, segs = 0;  // tiles and chunks before this segment, segments
      while (!fail && walk.next(sg)) {
        fail = !tm::mbar_wait_lane(bar(kBarQ), segs & 1, dead);
        if (fail) break;
        tm::fence_after();
        const int C = pl.chunks, total = sg.tiles * C;
        for (int i = 0; i <= total && !fail; ++i) {
          if (i < total) {  // scores of chunk i
            const int t = i / C, c = i - t * C, buf = split ? t & 1 : c & 1;
            const uint32_t tn = n + t, kb = tn % pl.nkb;
            // uses of this score buffer so far: this segment's and those before (per warpgroup)
            const uint32_t uses = (buf ? (items >> 16) : (items & 0xffffu)) + (split ? t >> 1 : i >> 1);
            if (c == 0) fail = !tm::mbar_wait_lane(bar(kBarKFull + kb), (tn / pl.nkb) & 1, dead);
            fail = !tm::mbar_wait_lane(bar(kBarSEmpty + buf), (uses & 1) ^ 1, dead) || fail;
            if (fail) break;
            tm::fence_after();
            const uint32_t d = tmem + pl.tm_s + buf * CN, a = tmem + pl.tm_k + kb * pl.kcols;
            const uint64_t b = d_q + c * (CN * 128 / 16);
            for (int p = 0; p < code_parts; ++p)
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tm::mma_ts(d, a + 8 * k, b + p * q_part + (k >> 2) * q_blk + 2 * (k & 3), id_s, p > 0 || k > 0);
            if (tb.qjl) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tm::mma_ts(d, a + D / 2 + 8 * k, b + code_parts * q_part + (k >> 2) * q_blk + 2 * (k & 3), id_s, true);
            }
            tm::mma_commit(bar(kBarSFull + buf));
            if (c == C - 1) tm::mma_commit(bar(kBarKEmpty + kb));
          }
          if (i > 0) {  // outputs of chunk i - 1
            const int j = i - 1, t = j / C, c = j - t * C, buf = split ? t & 1 : c & 1;
            const uint32_t tn = n + t, vb = tn % pl.nvb;
            const uint32_t uses = (buf ? (items >> 16) : (items & 0xffffu)) + (split ? t >> 1 : j >> 1);
            if (c == 0) fail = !tm::mbar_wait_lane(bar(kBarVFull + vb), (tn / pl.nvb) & 1, dead);
            fail = !tm::mbar_wait_lane(bar(kBarPFull + buf), uses & 1, dead) || fail;
            if (fail) break;
            tm::fence_after();
            const bool first = split ? t < 2 : t == 0;
            const uint32_t col = split ? buf * CN : c * CN;
            const uint64_t b = d_p + buf * (16384 / 16);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              const uint64_t a = d_v + vb * (kTile * D * 2 / 16) + mb * (2 * 16384 / 16);
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                tm::mma_ss(tmem + mb * pl.cols + col, a + k * (2048 / 16), b + k * (2048 / 16), id_o, !first || k > 0);
            }
            tm::mma_commit(bar(kBarPEmpty + buf));
            if (c == C - 1) tm::mma_commit(bar(kBarVEmpty + vb));
          }
        }
        n += sg.tiles;
        // buffer uses: chunk counts are even per tile, tiles alternate when split (parity is all that counts)
        const uint32_t u0 = split ? (sg.tiles + 1) >> 1 : total >> 1, u1 = split ? sg.tiles >> 1 : total >> 1;
        items = (((items & 0xffffu) + u0) & 1u) | ((((items >> 16) + u1) & 1u) << 16);
        ++segs;
      }
      if (fail) {  // after a failure the products in flight are waited for
        int never = 0;
        tm::mma_commit(bar(kBarDone));
        tm::mbar_wait_lane(bar(kBarDone), 0, &never);
      }
    }
    __syncwarp();
  } else {
    // =========================== copies ====================================
    if (lane == 0) {
      const uint32_t k_row = tb.k_bits * D / 8, v_row = tb.v_bits * D / 8, meta = tb.affine ? 4 * NG : 2;
      int st = 0, st_ph = 0;
      uint32_t n = 0;
      while (!fail && walk.next(sg)) {
        const int kvh = sg.unit / pl.blocks;
        for (int it = 0; it < sg.tiles; ++it, ++n) {
          fail = !tm::mbar_wait_lane(bar(kBarStEmpty + st), st_ph ^ 1, dead);
          if (fail) break;
          const int t = sg.t0 + it * kTile;
          const uint32_t m = min(kTile, (sg.len - t + 15) / 16 * 16);  // within the row: capacity is a multiple of 16
          const long s = ((long)sg.b * cv.kv_heads + kvh) * cv.capacity + t;
          const uint32_t dst = pl.sm_st + st * pl.st_bytes, full = bar(kBarStFull + st);
          tm::mbar_expect(full, m * (k_row + v_row + 2 * meta + (tb.qjl ? D / 8 + 2 : 0)));
          tm::bulk_load(dst, cv.k_codes + s * k_row, m * k_row, full);
          tm::bulk_load(dst + pl.st_kn, reinterpret_cast<const uint8_t*>(cv.k_norm) + s * meta, m * meta, full);
          tm::bulk_load(dst + pl.st_vn, reinterpret_cast<const uint8_t*>(cv.v_norm) + s * meta, m * meta, full);
          if (tb.qjl) {
            tm::bulk_load(dst + pl.st_s, cv.k_signs + s * (D / 8), m * (D / 8), full);
            tm::bulk_load(dst + pl.st_rn, cv.k_rnorm + s, m * 2, full);
          }
          tm::bulk_load(dst + pl.st_v, cv.v_codes + s * v_row, m * v_row, full);
          if (++st == pl.nst) st = 0, st_ph ^= 1;
        }
      }
      // after a failure the copies in flight are waited for
      if (fail) {
        int never = 0;
        for (uint32_t i = n > (uint32_t)pl.nst ? n - pl.nst : 0; i < n; ++i)
          tm::mbar_wait_lane(bar(kBarStFull + i % pl.nst), (i / pl.nst) & 1, &never);
      }
    }
    __syncwarp();
  }
  tm::fence_before();
  __syncthreads();
  if (tid == 0 && *dead) atomicOr(cv.status, (int)kFlagTimeout);
  if (warp == 16) {
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
                      const float* __restrict__ ws) {
  constexpr int E = D / 32, NT = 32 * kMergeWarps;
  __shared__ float wgt[kMergeMax];
  __shared__ float part[kMergeWarps][D];
  __shared__ float red[kMergeWarps];
  __shared__ long long tiles[2][kMergeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int i = blockIdx.x / ta.q_heads, h = blockIdx.x - i * ta.q_heads, H = cv.kv_heads, group = ta.q_heads / H;
  const int kvh = h / group, r = i * group + (h - kvh * group), rb = r / pl.rows, col = r - rb * pl.rows;
  const int units = H * pl.blocks, nctas = pl.ctas;
  const Walk walk{&cv, ta.n_q, ta.max_ctx, units, 0, 0, 0, 0};
  long long before = 0, all = 0;
  for (int k = tid; k < cv.batch; k += NT) {
    const long long x = (walk.length(k) + kTile - 1) / kTile;
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
  const int n = (walk.length(b) + kTile - 1) / kTile;
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
      const float* ml = ws + pl.slots * pl.cols * D + ((slot0 + s / sides) * pl.cols + (s % sides) * pl.rows + col) * 2;
      if (ml[1] != 0.f) ms = ml[0];
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
      const float2 y = *reinterpret_cast<const float2*>(ws + at * D + lane * E);
      v[0] = y.x;
      v[1] = y.y;
    } else {
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        const float4 y = reinterpret_cast<const float4*>(ws + at * D + lane * E)[e];
        v[4 * e] = y.x;
        v[4 * e + 1] = y.y;
        v[4 * e + 2] = y.z;
        v[4 * e + 3] = y.w;
      }
    }
    l = fmaf(ws[pl.slots * pl.cols * D + at * 2 + 1], x, l);
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
  p->sm_p = a.take(2 * 16384, 1024);
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
  int best = -1, nst = 2;  // (the widest rows, head_dim 256 with the affine codec and the sketch, fit one stage)
  for (; best < 0; --nst)
    for (int i = 0; i < 5; ++i) {
      if (!plan_shape(tb, dtype, shapes[i][0], shapes[i][1], 1, 1, nst, p)) continue;
      if (best < 0 || p->rows >= rows) best = i;
    }
  ++nst;
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
}

size_t plan_bytes(const TreePlan& p, int d) { return (size_t)p.slots * p.cols * (d + 2) * sizeof(float); }

template <int D, int CN, int CPW>
cudaError_t launch_shape(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, float* ws,
                         cudaStream_t stream) {
  static KernelConfig config;
  auto kern = tree_kernel<D, CN, CPW>;
  // the attribute is set once per device, for the largest plan
  cudaError_t e = configure_kernel(config, kern, 227 * 1024, kTreeThreads, nullptr);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ctas);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tb, cv, ta, pl, ws);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(ta.n_q * ta.q_heads), (unsigned)cv.batch);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, tb, cv, ta, pl, (const float*)ws);
}

template <int D>
cudaError_t launch_dim(const Tables& tb, const CacheView& cv, const TreeArgs& ta, const TreePlan& pl, float* ws,
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
  return std::max(plan_bytes(a, tb.d), plan_bytes(b, tb.d));
}

cudaError_t launch_tree(const Tables& tb, const CacheView& cv, const TreeArgs& ta, float* workspace,
                        cudaStream_t stream) {
  TreePlan pl;
  plan_tree(tb, ta.dtype, cv.batch, ta.q_heads, cv.kv_heads, ta.n_q, ta.max_ctx, &pl);
  switch (tb.d) {
    case 64: return launch_dim<64>(tb, cv, ta, pl, workspace, stream);
    case 128: return launch_dim<128>(tb, cv, ta, pl, workspace, stream);
    case 256: return launch_dim<256>(tb, cv, ta, pl, workspace, stream);
  }
  return cudaErrorNotSupported;
}

}  // namespace tq
