// Host-side check of the tree attention's plans (no GPU): every accepted codec, type
// and row count has one whose buffers lie apart, aligned and inside shared and tensor
// memory, and a codec whose buffers cannot fit has none instead of a wrong one.
// Built and run by tests/test_tree_plan_layout.py.
#include "tq_tree_plan.cuh"

#include <cstdio>
#include <vector>

using namespace tq;

static int g_bad = 0;
#define CHECK(c)                                                        \
  do {                                                                  \
    if (!(c)) {                                                         \
      if (g_bad < 20) std::printf("  failed: %s (line %d)\n", #c, __LINE__); \
      ++g_bad;                                                          \
    }                                                                   \
  } while (0)

struct Region {
  int at, bytes, align;
};

static void check(const Tables& tb, int dtype, int n_q, int group) {
  TreePlan p;
  if (!plan_tree(tb, dtype, 3, 2 * group, 2, n_q, 5000, &p)) {
    CHECK(!"a plan");
    return;
  }
  const int d = tb.d, rows = n_q * group;
  CHECK(p.rows == p.cn * p.chunks && p.rows * p.blocks >= rows && p.rows * (p.blocks - 1) < rows);
  CHECK(p.nkb >= 1 && p.nkb <= 2 && p.nvb >= 1 && p.nvb <= 2 && p.nsb >= 1 && p.nsb <= 2);
  CHECK(p.nst >= 2 && p.nst <= kMaxStages);
  // tensor memory: outputs, keys, scores
  CHECK(p.tm_k == p.rows * (d == 256 ? 2 : 1) && p.tm_s == p.tm_k + p.nkb * p.kcols && p.tm_s + p.nsb * p.cn <= 512);
  CHECK(p.kcols == d / 2 * (tb.qjl ? 2 : 1));
  // a stage's pieces follow one another
  const int meta = tb.affine ? 4 * d / kAffineGroup : 2;
  CHECK(p.st_v == kTile * tb.k_bits * d / 8 && p.st_s == p.st_v + kTile * tb.v_bits * d / 8);
  CHECK(p.st_kn == p.st_s + (tb.qjl ? kTile * d / 8 : 0) && p.st_vn == p.st_kn + kTile * meta);
  CHECK(p.st_rn == p.st_vn + kTile * meta && p.st_bytes >= p.st_rn + (tb.qjl ? 2 * kTile : 0) && p.st_bytes % 128 == 0);
  for (int x : {p.st_v, p.st_s, p.st_kn, p.st_vn, p.st_rn}) CHECK(x % 16 == 0);  // bulk copies' targets
  // shared memory
  std::vector<Region> r = {{p.lut_k, lut_bytes(tb.k_bits), lut_bytes(tb.k_bits)},
                           {p.sm_v, p.nvb * kTile * d * 2, 1024},
                           {p.sm_q, p.parts * p.rows * d * 2, 1024},
                           {p.sm_p, p.cn >= 64 ? p.nsb * (p.cn / 64) * 16384 : 16384, 1024},
                           {p.sm_st, p.nst * p.st_bytes, 128},
                           {p.sm_meta, kMetaSlots * kTile * 8, 128},
                           {p.sm_misc, kMiscBytes, 16}};
  if (tb.k_bits == tb.v_bits) CHECK(p.lut_v == p.lut_k);
  else r.push_back({p.lut_v, lut_bytes(tb.v_bits), lut_bytes(tb.v_bits)});
  CHECK(p.smem >= 120 * 1024 && p.smem <= 227 * 1024);
  for (size_t i = 0; i < r.size(); ++i) {
    CHECK(r[i].at % r[i].align == 0 && r[i].at >= (int)kDynSmemBase && r[i].at + r[i].bytes <= (int)kDynSmemBase + p.smem);
    for (size_t j = 0; j < i; ++j) CHECK(r[i].at + r[i].bytes <= r[j].at || r[j].at + r[j].bytes <= r[i].at);
  }
  // workspace: partials, maxima and sums, query tables, scales
  const long units = 3L * 2 * p.blocks;
  CHECK(p.ctas >= 1 && p.ctas <= kTreeMaxCtas && p.slots == p.ctas + units && p.q_bytes == p.parts * p.rows * d * 2);
  CHECK(p.ws_ml >= p.slots * p.rows * d * 4 && p.ws_ml % 8 == 0 && p.ws_q >= p.ws_ml + p.slots * p.rows * 8);
  CHECK(p.ws_q % 128 == 0 && p.ws_scale >= p.ws_q + units * p.q_bytes && p.ws_scale % 4 == 0);
  CHECK(p.ws_rows >= p.ws_scale + 4 * units && p.ws_rows % 8 == 0 && (long)plan_bytes(p) >= p.ws_rows + units * p.rows * 4);
}

int main() {
  Tables tb = {};
  int shapes = 0;
  for (int d : {64, 128, 256})
    for (int kb = 2; kb <= 4; ++kb)
      for (int vb = kb; vb <= std::min(kb + 1, 4); ++vb)
        for (int qjl = 0; qjl < 2; ++qjl)
          for (int affine = 0; affine < 2; ++affine)
            for (int dtype : {(int)kBF16, (int)kF16})
              for (int n : {1, 2, 5, 16, 17, 33, 64, 65, 128, 256})
                for (int group : {1, 2, 4, 8}) {
                  tb.d = d;
                  tb.k_bits = kb;
                  tb.v_bits = vb;
                  tb.qjl = qjl;
                  tb.affine = affine;
                  check(tb, dtype, n, group);
                  ++shapes;
                }
  // codes of 8 bits at head_dim 256: the tables, two stages and one value buffer pass 227 KB
  tb.d = 256;
  tb.k_bits = tb.v_bits = 8;
  tb.qjl = 1;
  for (int affine = 0; affine < 2; ++affine)
    for (int dtype : {(int)kBF16, (int)kF16})
      for (int n : {1, 17, 40, 100, 256}) {
        tb.affine = affine;
        TreePlan p;
        CHECK(!plan_tree(tb, dtype, 1, 8, 1, n, 1000, &p));
        CHECK(!plan_tree(tb, dtype, 1, 8, 1, n, 1000, &p));  // and it is not remembered as one
      }
  std::printf("%d shapes, total bad %d\n", shapes, g_bad);
  return g_bad != 0;
}
