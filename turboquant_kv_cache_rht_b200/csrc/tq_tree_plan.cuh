// Plans of the tree attention: how a call's query rows are split into chunks of columns,
// and where the kernel's buffers lie in shared and tensor memory (host only).
#pragma once

#include "tq_tree_impl.cuh"

#include <algorithm>

namespace tq {

// Shared addresses, first fit into the gaps that alignment leaves.
struct Arena {
  static constexpr int kGaps = 16;  // one more than the buffers that a plan takes
  int lo[kGaps] = {(int)kDynSmemBase}, hi[kGaps] = {228 * 1024};  // 227 KB of a block, from kDynSmemBase
  int n = 1, end = kDynSmemBase;
  bool ok = true;
  int take(int bytes, int align) {
    for (int i = 0; i < n && n < kGaps; ++i) {
      const int a = (lo[i] + align - 1) / align * align;
      if (a + bytes > hi[i]) continue;
      for (int j = n++; j > i + 1; --j) {
        lo[j] = lo[j - 1];
        hi[j] = hi[j - 1];
      }
      lo[i + 1] = a + bytes;
      hi[i + 1] = hi[i];
      hi[i] = a;
      end = std::max(end, a + bytes);
      return a;
    }
    ok = false;
    return 0;
  }
};

// The plan of chunks x cn query rows; false if its buffers do not fit.
inline bool plan_shape(const Tables& tb, int dtype, int cn, int chunks, int nkb, int nvb, int nst, int nsb, TreePlan* p) {
  const int d = tb.d;
  p->cn = cn;
  p->chunks = chunks;
  p->rows = cn * chunks;
  p->parts = 1 + (dtype == kF16) + (tb.qjl != 0);
  p->nkb = nkb;
  p->nvb = nvb;
  p->nst = nst;
  p->nsb = nsb;
  p->kcols = d / 2 * (tb.qjl ? 2 : 1);
  p->tm_k = p->rows * (d == 256 ? 2 : 1);
  p->tm_s = p->tm_k + nkb * p->kcols;
  if (p->tm_s + nsb * cn > 512) return false;
  Arena a;
  p->lut_k = a.take(lut_bytes(tb.k_bits), lut_bytes(tb.k_bits));
  p->lut_v = tb.k_bits == tb.v_bits ? p->lut_k : a.take(lut_bytes(tb.v_bits), lut_bytes(tb.v_bits));
  p->sm_v = a.take(nvb * kTile * d * 2, 1024);
  p->sm_q = a.take(p->parts * p->rows * d * 2, 1024);
  p->sm_p = a.take(cn >= 64 ? nsb * (cn / 64) * 16384 : 16384, 1024);  // narrow chunks: halves of one buffer's rows
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
  p->sm_meta = a.take(kMetaSlots * kTile * 8, 128);
  p->sm_misc = a.take(kMiscBytes, 16);
  // at least half of an SM's shared memory: one block per SM, which owns its tensor memory
  p->smem = std::max(a.end - (int)kDynSmemBase, 120 * 1024);
  p->q_bytes = p->parts * p->rows * d * 2;
  return a.ok;
}

// The narrowest columns that hold `rows` query rows, or the widest that fit, and
// then as many buffers as fit: of the scores and weights (two chunks under way), of
// the keys, of the values, of packed stages.  (Two score buffers where chunks are
// narrow; a wide chunk's scores are given back before its exponentials.)  It depends
// on the codec, the type and the class of the rows alone, so a thread keeps it.  NULL if
// nothing fits.
inline const TreePlan* shape_of(const Tables& tb, int dtype, int rows) {
  static const int shapes[][2] = {{16, 1}, {32, 1}, {64, 1}, {128, 1}, {128, 2}};
  struct Kept {
    int key = -1;
    TreePlan plan;
  };
  static thread_local Kept kept[16];
  const int cls = rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 ? 3 : 4;
  const int key = ((((((tb.d / 64) * 4 + tb.k_bits - 1) * 4 + tb.v_bits - 1) * 2 + (tb.qjl != 0)) * 2 + (tb.affine != 0)) * 2 +
                   (dtype == kF16)) * 5 + cls;
  Kept& k = kept[key % 16];
  if (k.key == key) return &k.plan;
  TreePlan* p = &k.plan;
  k.key = -1;
  for (int c = cls; c >= 0; --c) {
    const int cn = shapes[c][0], chunks = shapes[c][1], narrow = cn < 128 ? 2 : 1;
    if ((tb.d == 256 && cn == 128) || !plan_shape(tb, dtype, cn, chunks, 1, 1, 2, narrow, p)) continue;
    int nkb = 1, nvb = 1, nst = 2, nsb = narrow;
    if (plan_shape(tb, dtype, cn, chunks, 2, nvb, nst, nsb, p)) nkb = 2;
    if (plan_shape(tb, dtype, cn, chunks, nkb, 2, nst, nsb, p)) nvb = 2;
    if (plan_shape(tb, dtype, cn, chunks, nkb, nvb, nst, 2, p)) nsb = 2;
    while (nst < kMaxStages && plan_shape(tb, dtype, cn, chunks, nkb, nvb, nst + 1, nsb, p)) ++nst;
    plan_shape(tb, dtype, cn, chunks, nkb, nvb, nst, nsb, p);
    k.key = key;
    return p;
  }
  return nullptr;
}

// False where no shape of this codec and type fits.
inline bool plan_tree(const Tables& tb, int dtype, int batch, int q_heads, int kv_heads, int n_q, int max_ctx, TreePlan* p) {
  const int rows = n_q * (q_heads / kv_heads);
  const TreePlan* shape = shape_of(tb, dtype, rows);
  if (!shape) return false;
  *p = *shape;
  p->blocks = (rows + p->rows - 1) / p->rows;
  const long units = (long)batch * kv_heads * p->blocks;
  p->ctas = (int)std::max(1L, std::min((long)kTreeMaxCtas, units * ((max_ctx + kTile - 1) / kTile)));
  p->slots = p->ctas + units;
  p->ws_ml = p->slots * p->rows * tb.d * 4;
  p->ws_q = (p->ws_ml + p->slots * p->rows * 8 + 127) / 128 * 128;
  p->ws_scale = p->ws_q + units * p->q_bytes;
  p->ws_rows = (p->ws_scale + units * 4 + 15) / 16 * 16;
  return true;
}

inline size_t plan_bytes(const TreePlan& p) { return (size_t)(p.ws_rows + (p.slots - p.ctas) * p.rows * 4); }

}  // namespace tq
