// C ABI of libtq: argument validation, codebook/sign construction on the host,
// and kernel dispatch.  See include/tq.h for the contract of every entry point.
#include "../../include/tq.h"
#include "tq_internal.cuh"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>

struct tq_codebook {
  tq_params params;
  tq::Tables tables;
};

namespace {

thread_local std::string g_last_error;

tq_status fail(tq_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

tq_status ok() {
  g_last_error.clear();
  return TQ_OK;
}

// ---------------------------------------------------------------------------
// Lloyd-Max quantizer of the standard normal distribution ("How to Use
// TurboQuant with the MLX-VLM Python API", "What is TurboQuant?": _codebook;
// "mlx-turboquant" README: Lloyd-Max codebook for the near-Gaussian rotated
// coordinates).  Lloyd's two conditions are iterated in double precision until
// no level moves by 1e-14: boundaries at the midpoints of adjacent levels,
// levels at the conditional means of their cells.
// ---------------------------------------------------------------------------
double normal_density(double x) {
  if (std::isinf(x)) return 0.0;
  return std::exp(-0.5 * x * x) / std::sqrt(2.0 * M_PI);
}

// P(X > x)
double normal_tail(double x) { return 0.5 * std::erfc(x / std::sqrt(2.0)); }

// P(lo < X < hi), arranged so that neither tail is obtained by cancellation.
double normal_mass(double lo, double hi) {
  if (lo >= 0.0) return normal_tail(lo) - normal_tail(hi);
  if (hi <= 0.0) return normal_tail(-hi) - normal_tail(-lo);
  return 1.0 - normal_tail(-lo) - normal_tail(hi);
}

double normal_cell_mean(double lo, double hi) {
  return (normal_density(lo) - normal_density(hi)) / normal_mass(lo, hi);
}

// The exact distribution of a rotated coordinate.  For a fixed x, each
// coordinate of R x / ||x|| is a coordinate of a uniformly random unit vector
// of R^d, so Z = sqrt(d) (R x)_i / ||x|| has density
// f(z) = C_d (1 - z^2/d)^((d-3)/2) on |z| < sqrt(d), C_d = Gamma(d/2) /
// (sqrt(pi d) Gamma((d-1)/2)); the rotated coordinates are only near-Gaussian
// ("mlx-turboquant" README, introduction).  Cell masses are integrated
// directly (composite 10-point Gauss-Legendre on pieces at most 1/4 wide,
// compensated sums), so a small outer cell is not the difference of two
// nearly equal cumulative integrals.
struct Sphere {
  int d;
  double c;  // C_d
};

struct GaussLegendre10 {
  double x[10], w[10];
  GaussLegendre10() {  // roots of the Legendre polynomial P_10 by Newton's method
    for (int i = 0; i < 10; ++i) {
      double z = std::cos(M_PI * (i + 0.75) / 10.5), dp = 1.0;
      for (int it = 0; it < 100; ++it) {
        double p0 = 1.0, p1 = z;  // P_0, P_1, then the three-term recurrence
        for (int k = 2; k <= 10; ++k) {
          const double pk = ((2 * k - 1) * z * p1 - (k - 1) * p0) / k;
          p0 = p1;
          p1 = pk;
        }
        dp = 10 * (z * p1 - p0) / (z * z - 1.0);
        const double step = p1 / dp;
        z -= step;
        if (std::fabs(step) < 1e-16) break;
      }
      x[i] = z;
      w[i] = 2.0 / ((1.0 - z * z) * dp * dp);
    }
  }
};

// (1 - z^2/d)^k as exp(k log1p(-z^2/d)): a power of the rounded base would
// carry k times the base's rounding error, which is what limits Lloyd's
// iteration near its tolerance.
double sphere_power(double z, int d, double k) {
  const double x = z * z / d;
  return x >= 1.0 ? 0.0 : std::exp(k * std::log1p(-x));
}

double sphere_density(const Sphere& sp, double z) { return sp.c * sphere_power(z, sp.d, (sp.d - 3) / 2.0); }

double sphere_mass(const Sphere& sp, double lo, double hi) {
  static const GaussLegendre10 gl;
  const double r = std::sqrt((double)sp.d);
  lo = std::fmax(lo, -r);
  hi = std::fmin(hi, r);
  if (!(hi > lo)) return 0.0;
  const int pieces = std::max(1, (int)std::ceil((hi - lo) * 4.0));
  const double h = (hi - lo) / pieces;
  double sum = 0.0, comp = 0.0;  // Kahan summation
  for (int p = 0; p < pieces; ++p) {
    const double mid = lo + (p + 0.5) * h;
    for (int i = 0; i < 10; ++i) {
      const double term = gl.w[i] * sphere_density(sp, mid + 0.5 * h * gl.x[i]) * 0.5 * h - comp;
      const double next = sum + term;
      comp = (next - sum) - term;
      sum = next;
    }
  }
  return sum;
}

// Integral of z f(z) over (lo, hi): an antiderivative of z (1 - z^2/d)^k is
// -(d / (2 (k + 1))) (1 - z^2/d)^(k + 1), here with k = (d - 3) / 2.
double sphere_cell_mean(const Sphere& sp, double lo, double hi) {
  const double d = sp.d, r = std::sqrt(d);
  auto g = [&](double z) { return std::fabs(z) >= r ? 0.0 : sphere_power(z, sp.d, (d - 1) / 2); };
  return sp.c * d / (d - 1) * (g(lo) - g(hi)) / sphere_mass(sp, lo, hi);
}

// Lloyd's iteration from `lv` (levels ascending) with the given cell-mean rule.
template <typename CellMean>
bool lloyd_iterate(int levels, double* lv, CellMean cell_mean) {
  double next[16], edge[17];
  for (int iter = 0; iter < 1000000; ++iter) {
    edge[0] = -INFINITY;
    edge[levels] = INFINITY;
    for (int j = 1; j < levels; ++j) edge[j] = 0.5 * (lv[j - 1] + lv[j]);
    double moved = 0.0;
    for (int j = 0; j < levels; ++j) {
      next[j] = cell_mean(edge[j], edge[j + 1]);
      moved = std::fmax(moved, std::fabs(next[j] - lv[j]));
    }
    std::memcpy(lv, next, sizeof(double) * levels);
    if (moved < 1e-14) return true;
  }
  return false;
}

// Levels of the Lloyd-Max quantizer of N(0,1) (kind 0) or of the rotated-
// coordinate distribution for head_dim d (kind 1, started from the N(0,1)
// solution).
bool lloyd_max(int levels, int kind, int d, double* lv) {
  for (int j = 0; j < levels; ++j) lv[j] = -2.0 + 4.0 * (j + 0.5) / levels;
  if (!lloyd_iterate(levels, lv, normal_cell_mean)) return false;
  if (kind == 0) return true;
  const Sphere sp{d, std::exp(std::lgamma(d / 2.0) - std::lgamma((d - 1) / 2.0)) /
                         std::sqrt(M_PI * d)};
  return lloyd_iterate(levels, lv, [&](double lo, double hi) { return sphere_cell_mean(sp, lo, hi); });
}

// float32 table: odd-symmetric levels, boundaries = float32 midpoints.
bool build_codebook(int bits, int kind, int d, float* cent, float* bnd) {
  const int levels = 1 << bits, half = levels / 2;
  double lv[16];
  if (!lloyd_max(levels, kind, d, lv)) return false;
  for (int j = 0; j < half; ++j) {
    const float pos = (float)((lv[half + j] - lv[half - 1 - j]) / 2.0);
    cent[half + j] = pos;
    cent[half - 1 - j] = -pos;
  }
  for (int j = 0; j + 1 < levels; ++j) {
    volatile float s = cent[j] + cent[j + 1];  // two float32 roundings, no contraction
    bnd[j] = s * 0.5f;
  }
  for (int j = levels - 1; j < 16; ++j) bnd[j] = INFINITY;
  for (int j = levels; j < 16; ++j) cent[j] = 0.0f;
  return true;
}

// fp16 rounding of a float in fp16's normal range, to nearest even (the
// table scale search below only meets magnitudes in [2^-14, 2^15)).
double round_fp16_normal(float x) {
  int e = 0;
  const double m = std::frexp((double)x, &e);       // x = m 2^e, 0.5 <= |m| < 1
  return std::ldexp(std::nearbyint(std::ldexp(m, 11)), e - 11);  // 11 significant bits
}

// Scale lam in [1, 2) under which the fp16 roundings of lam * c_j (formed as
// an fp32 product, as the decode kernel forms it) come closest to the exact
// products: the largest relative rounding error over the nonzero entries is
// minimal.  The decode kernel's code tables hold fp16(lam * c_j) and undo lam
// in fp32, so a table of 4, 8 or 16 Lloyd-Max levels carries ~2^-22, ~2^-16
// or ~2^-13 relative error instead of fp16's 2^-12.
float fp16_table_scale(const float* cent, int levels) {
  constexpr int kSteps = 1 << 16;
  float best = 1.0f;
  double best_err = INFINITY;
  for (int i = 0; i < kSteps; ++i) {
    const float lam = 1.0f + (float)i / (float)kSteps;
    double err = 0.0;
    for (int j = levels / 2; j < levels && err < best_err; ++j) {  // odd symmetry
      const float x = cent[j] * lam;
      if (x == 0.0f) continue;
      err = std::max(err, std::fabs(round_fp16_normal(x) - (double)x) / std::fabs((double)x));
    }
    if (err < best_err) {
      best_err = err;
      best = lam;
    }
  }
  return best;
}

// Affine codec tables: the integer levels 0 .. 2^bits - 1 and their midpoints
// (the decode kernel's pair tables turn code pairs into these levels).
void build_affine_levels(int bits, float* cent, float* bnd) {
  const int levels = 1 << bits;
  for (int j = 0; j < 16; ++j) {
    cent[j] = j < levels ? (float)j : 0.0f;
    bnd[j] = j + 1 < levels ? (float)j + 0.5f : INFINITY;
  }
}

// SplitMix64 (Steele, Lea & Flood, OOPSLA 2014): the sign of channel i is the
// top bit of the i-th output.
void build_signs(uint64_t state, int d, uint32_t* mask) {
  for (int w = 0; w < 8; ++w) mask[w] = 0;
  for (int i = 0; i < d; ++i) {
    state += 0x9E3779B97F4A7C15ull;
    uint64_t z = state;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    z ^= z >> 31;
    if (z >> 63) mask[i >> 5] |= 1u << (i & 31);
  }
}

tq_status check_params(const tq_params* p) {
  if (!p) return fail(TQ_ERR_INVALID, "params is NULL");
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return fail(TQ_ERR_INVALID, "head_dim %d: supported values are 64, 128 and 256", p->head_dim);
  if (p->k_bits < 2 || p->k_bits > 4 || p->v_bits < 2 || p->v_bits > 4)
    return fail(TQ_ERR_INVALID, "k_bits=%d v_bits=%d: each must be 2, 3 or 4", p->k_bits,
                p->v_bits);
  if (p->qjl != 0 && p->qjl != 1) return fail(TQ_ERR_INVALID, "qjl must be 0 or 1");
  if (p->codebook != TQ_CODEBOOK_GAUSSIAN && p->codebook != TQ_CODEBOOK_SPHERE &&
      p->codebook != TQ_CODEBOOK_AFFINE)
    return fail(TQ_ERR_INVALID,
                "codebook %d: must be TQ_CODEBOOK_GAUSSIAN, TQ_CODEBOOK_SPHERE or TQ_CODEBOOK_AFFINE",
                p->codebook);
  return TQ_OK;
}

// Rotations per position of each pair, with the scaling for long contexts
// applied (the formulas stand at tq_rope_params).
tq_status rope_frequencies(const tq_rope_params& p, tq::RopeFrequencies* out) {
  if (p.rot_dim < 2 || p.rot_dim % 2 || p.rot_dim > 256)
    return fail(TQ_ERR_INVALID, "rot_dim %d: even, 2 .. 256", p.rot_dim);
  if (p.scaling < TQ_ROPE_NONE || p.scaling > TQ_ROPE_BANDS)
    return fail(TQ_ERR_INVALID, "scaling %d: one of TQ_ROPE_NONE .. TQ_ROPE_BANDS", p.scaling);
  if (!(p.base > 1.0) || !std::isfinite(p.base)) return fail(TQ_ERR_INVALID, "base must be above 1 and finite");
  if (p.scaling != TQ_ROPE_NONE && (!(p.factor >= 1.0) || !std::isfinite(p.factor)))
    return fail(TQ_ERR_INVALID, "factor must be at least 1 and finite");
  if ((p.scaling == TQ_ROPE_YARN || p.scaling == TQ_ROPE_BANDS) && p.original_max < 1)
    return fail(TQ_ERR_INVALID, "original_max %d: at least 1", p.original_max);
  if (p.scaling == TQ_ROPE_YARN && !(p.beta_fast > p.beta_slow && p.beta_slow > 0.0 && std::isfinite(p.beta_fast)))
    return fail(TQ_ERR_INVALID, "beta_fast must be above beta_slow, both above 0");
  if (p.scaling == TQ_ROPE_BANDS && !(p.high_freq > p.low_freq && p.low_freq > 0.0 && std::isfinite(p.high_freq)))
    return fail(TQ_ERR_INVALID, "high_freq must be above low_freq, both above 0");
  if (!(p.attention_factor >= 0.0) || !std::isfinite(p.attention_factor))
    return fail(TQ_ERR_INVALID, "attention_factor must be finite and not negative");
  const double rot = p.rot_dim, two_pi = 2.0 * M_PI;
  double base = p.base;
  if (p.scaling == TQ_ROPE_NTK && p.rot_dim > 2) base = p.base * std::pow(p.factor, rot / (rot - 2.0));
  double low = 0.0, high = 0.0;
  if (p.scaling == TQ_ROPE_YARN) {
    auto pair_of = [&](double turns) {  // the pair that turns so often over original_max positions
      return rot * std::log(p.original_max / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_of(p.beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(p.beta_slow)), rot - 1.0);
  }
  for (int i = 0; i < p.rot_dim / 2; ++i) {
    const double f = std::pow(base, -(2.0 * i) / rot);
    double g = f;
    if (p.scaling == TQ_ROPE_LINEAR) {
      g = f / p.factor;
    } else if (p.scaling == TQ_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      g = f / p.factor * r + f * (1.0 - r);
    } else if (p.scaling == TQ_ROPE_BANDS) {
      const double turns = p.original_max * f / two_pi;
      const double s = std::fmin(std::fmax((turns - p.low_freq) / (p.high_freq - p.low_freq), 0.0), 1.0);
      g = (1.0 - s) * (f / p.factor) + s * f;
    }
    out->freq[i] = g;
  }
  out->factor = p.attention_factor != 0.0 ? p.attention_factor
                : p.scaling == TQ_ROPE_YARN && p.factor > 1.0 ? 0.1 * std::log(p.factor) + 1.0 : 1.0;
  return TQ_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

tq_status check_cache(const tq_codebook* cb, const tq_cache* c) {
  if (!cb) return fail(TQ_ERR_INVALID, "codebook is NULL");
  if (!c) return fail(TQ_ERR_INVALID, "cache is NULL");
  if (c->batch <= 0 || c->kv_heads <= 0 || c->capacity <= 0)
    return fail(TQ_ERR_INVALID, "cache sizes must be positive (batch=%d kv_heads=%d capacity=%d)",
                c->batch, c->kv_heads, c->capacity);
  if (c->capacity % 16 != 0)
    return fail(TQ_ERR_INVALID, "capacity %d is not a multiple of 16", c->capacity);
  // the append, conversion and merge grids index batch rows by blockIdx.y
  if (c->batch > 65535) return fail(TQ_ERR_INVALID, "batch %d: at most 65535 rows", c->batch);
  const void* need[] = {c->k_codes, c->v_codes, c->k_norm, c->v_norm, c->seq_lens, c->status,
                        c->append_sync};
  const char* names[] = {"k_codes", "v_codes", "k_norm", "v_norm", "seq_lens", "status",
                         "append_sync"};
  for (int i = 0; i < 7; ++i) {
    if (!need[i]) return fail(TQ_ERR_INVALID, "cache.%s is NULL", names[i]);
    if (i < 4 && !aligned16(need[i]))
      return fail(TQ_ERR_INVALID, "cache.%s is not 16-byte aligned", names[i]);
  }
  if (cb->params.qjl) {
    if (!c->k_signs || !c->k_rnorm)
      return fail(TQ_ERR_INVALID, "QJL codebook needs cache.k_signs and cache.k_rnorm");
    if (!aligned16(c->k_signs) || !aligned16(c->k_rnorm))
      return fail(TQ_ERR_INVALID, "cache.k_signs / k_rnorm are not 16-byte aligned");
  }
  const double slots = (double)c->batch * c->kv_heads * c->capacity;
  if (slots * 128.0 > 9.0e18) return fail(TQ_ERR_INVALID, "cache too large");
  return TQ_OK;
}

tq::CacheView view_of(const tq_cache* c) {
  tq::CacheView v;
  v.k_codes = c->k_codes;
  v.v_codes = c->v_codes;
  v.k_signs = c->k_signs;
  v.k_norm = c->k_norm;
  v.v_norm = c->v_norm;
  v.k_rnorm = c->k_rnorm;
  v.seq_lens = c->seq_lens;
  v.status = c->status;
  v.append_sync = c->append_sync;
  v.batch = c->batch;
  v.kv_heads = c->kv_heads;
  v.capacity = c->capacity;
  return v;
}

// The arrays whose slots a copy or a compaction moves, with the bytes of a slot.
tq::SlotArrays arrays_of(const tq_codebook* cb, const tq_cache* c) {
  const tq::Tables& t = cb->tables;
  const int meta = t.affine ? 4 * t.d / tq::kAffineGroup : 2;
  tq::SlotArrays a = {};
  auto add = [&](void* p, int bytes) {
    a.p[a.n] = static_cast<uint8_t*>(p);
    a.bytes[a.n++] = bytes;
  };
  add(c->k_codes, t.k_bits * t.d / 8);
  add(c->v_codes, t.v_bits * t.d / 8);
  add(c->k_norm, meta);
  add(c->v_norm, meta);
  if (t.qjl) {
    add(c->k_signs, t.d / 8);
    add(c->k_rnorm, 2);
  }
  return a;
}

// Whether two caches share memory without being one cache (the same arrays, rows of the
// same capacity): a copy could then read what it writes.
bool overlap(const tq::SlotArrays& a, const tq_cache* ca, const tq::SlotArrays& b, const tq_cache* cb) {
  bool one = ca->capacity == cb->capacity;
  for (int i = 0; i < a.n; ++i) one = one && a.p[i] == b.p[i];
  if (one) return false;
  auto end = [](const tq::SlotArrays& x, const tq_cache* c, int i) {
    return (uintptr_t)x.p[i] + (uintptr_t)c->batch * c->kv_heads * c->capacity * x.bytes[i];
  };
  for (int i = 0; i < a.n; ++i)
    for (int j = 0; j < b.n; ++j)
      if ((uintptr_t)a.p[i] < end(b, cb, j) && (uintptr_t)b.p[j] < end(a, ca, i)) return true;
  return false;
}

tq_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  if (e == cudaErrorNotSupported) return fail(TQ_ERR_UNSUPPORTED, "%s: no kernel for this shape on this device", what);
  return fail(TQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

namespace tq {
int record_error(int status, const char* message) {
  g_last_error = message;
  return status;
}
}  // namespace tq

extern "C" {

tq_status tq_codebook_init(const tq_params* params, tq_codebook** out, tq_layout* layout) {
  if (!out) return fail(TQ_ERR_INVALID, "out is NULL");
  *out = nullptr;
  tq_status st = check_params(params);
  if (st != TQ_OK) return st;
  tq_codebook* cb = new (std::nothrow) tq_codebook;
  if (!cb) return fail(TQ_ERR_NOMEM, "host allocation of the codebook failed");
  std::memset(cb, 0, sizeof *cb);
  cb->params = *params;
  tq::Tables& t = cb->tables;
  t.d = params->head_dim;
  t.k_bits = params->k_bits;
  t.v_bits = params->v_bits;
  t.qjl = params->qjl;
  const int kind = params->codebook, d = params->head_dim;
  t.affine = kind == TQ_CODEBOOK_AFFINE;
  if (t.affine) {
    build_affine_levels(params->k_bits, t.k_cent, t.k_bnd);
    build_affine_levels(params->v_bits, t.v_cent, t.v_bnd);
  } else if (!build_codebook(params->k_bits, kind, d, t.k_cent, t.k_bnd) ||
             !build_codebook(params->v_bits, kind, d, t.v_cent, t.v_bnd)) {
    delete cb;
    return fail(TQ_ERR_INVALID, "Lloyd-Max iteration did not converge");
  }
  t.k_lam = t.affine ? 1.0f : fp16_table_scale(t.k_cent, 1 << params->k_bits);
  t.v_lam = t.affine ? 1.0f : fp16_table_scale(t.v_cent, 1 << params->v_bits);
  build_signs(params->seed, params->head_dim, t.s1);
  build_signs(params->seed ^ 0x9E3779B97F4A7C15ull, params->head_dim, t.s2);
  if (layout) {
    layout->k_code_bytes = (size_t)params->k_bits * params->head_dim / 8;
    layout->v_code_bytes = (size_t)params->v_bits * params->head_dim / 8;
    layout->k_sign_bytes = params->qjl ? (size_t)params->head_dim / 8 : 0;
    layout->norm_halves = t.affine ? (size_t)2 * params->head_dim / tq::kAffineGroup : 1;
  }
  *out = cb;
  return ok();
}

tq_status tq_codebook_tables(const tq_codebook* cb, float* k_centroids, float* k_boundaries,
                             float* v_centroids, float* v_boundaries, int8_t* signs1,
                             int8_t* signs2) {
  if (!cb) return fail(TQ_ERR_INVALID, "codebook is NULL");
  const tq::Tables& t = cb->tables;
  const int lk = 1 << t.k_bits, lv = 1 << t.v_bits;
  if (k_centroids) std::memcpy(k_centroids, t.k_cent, sizeof(float) * lk);
  if (k_boundaries) std::memcpy(k_boundaries, t.k_bnd, sizeof(float) * (lk - 1));
  if (v_centroids) std::memcpy(v_centroids, t.v_cent, sizeof(float) * lv);
  if (v_boundaries) std::memcpy(v_boundaries, t.v_bnd, sizeof(float) * (lv - 1));
  for (int i = 0; i < t.d; ++i) {
    if (signs1) signs1[i] = ((t.s1[i >> 5] >> (i & 31)) & 1u) ? -1 : 1;
    if (signs2) signs2[i] = ((t.s2[i >> 5] >> (i & 31)) & 1u) ? -1 : 1;
  }
  return ok();
}

tq_status tq_quantize_append(const tq_codebook* cb, const tq_cache* cache, const void* k,
                             const void* v, tq_dtype dtype, int n_new, void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (n_new < 0) return fail(TQ_ERR_INVALID, "n_new %d is negative", n_new);
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "unknown dtype %d", (int)dtype);
  if (n_new == 0) return ok();
  if (!k || !v) return fail(TQ_ERR_INVALID, "k or v is NULL");
  if (n_new > cache->capacity)
    return fail(TQ_ERR_INVALID, "n_new %d exceeds capacity %d", n_new, cache->capacity);
  const size_t esz = dtype == TQ_F32 ? 4 : 2;
  const size_t vec_bytes = esz * cb->params.head_dim;
  if (((uintptr_t)k % vec_bytes) % 8 != 0 || ((uintptr_t)v % vec_bytes) % 8 != 0 ||
      !aligned16(k) || !aligned16(v))
    return fail(TQ_ERR_INVALID, "k and v must be 16-byte aligned");
  return cuda_status(tq::launch_quantize_append(cb->tables, view_of(cache), k, v, (int)dtype,
                                                n_new, (cudaStream_t)stream),
                     "quantize-append launch");
}

tq_status tq_quantize_cache(const tq_codebook* cb, const tq_cache* cache, const void* k,
                            const void* v, tq_dtype dtype, int64_t stride_b, int64_t stride_h,
                            int64_t stride_t, const int32_t* lengths, int max_len, void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "unknown dtype %d", (int)dtype);
  if (max_len < 0) return fail(TQ_ERR_INVALID, "max_len %d is negative", max_len);
  if (max_len == 0) return ok();
  if (!k || !v || !lengths) return fail(TQ_ERR_INVALID, "k, v or lengths is NULL");
  if (stride_b < 0 || stride_h < 0 || stride_t < 0)
    return fail(TQ_ERR_INVALID, "negative stride");
  const int64_t esz = dtype == TQ_F32 ? 4 : 2;
  if ((stride_b * esz) % 16 || (stride_h * esz) % 16 || (stride_t * esz) % 16)
    return fail(TQ_ERR_INVALID, "strides (%lld, %lld, %lld) are not multiples of 16 bytes",
                (long long)stride_b, (long long)stride_h, (long long)stride_t);
  if (!aligned16(k) || !aligned16(v)) return fail(TQ_ERR_INVALID, "k and v must be 16-byte aligned");
  if ((uintptr_t)lengths % 4) return fail(TQ_ERR_INVALID, "lengths must be 4-byte aligned");
  return cuda_status(tq::launch_quantize_cache(cb->tables, view_of(cache), k, v, (int)dtype,
                                               stride_b, stride_h, stride_t, lengths, max_len,
                                               (cudaStream_t)stream),
                     "quantize-cache launch");
}

static tq_status check_weights(const tq_codebook* cb, int rows, int k, tq_dtype dtype) {
  if (!cb) return fail(TQ_ERR_INVALID, "codebook is NULL");
  if (cb->tables.affine)
    return fail(TQ_ERR_UNSUPPORTED, "the weights regime takes a Lloyd-Max codebook, not the affine codec");
  if (rows <= 0 || rows % 16) return fail(TQ_ERR_INVALID, "rows %d: a positive multiple of 16", rows);
  const int d = cb->params.head_dim;
  if (k <= 0 || k % d) return fail(TQ_ERR_INVALID, "k %d: a positive multiple of head_dim %d", k, d);
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "unknown dtype %d", (int)dtype);
  return TQ_OK;
}

tq_status tq_weights_quantize(const tq_codebook* cb, const void* w, tq_dtype dtype, int rows, int k,
                              uint8_t* codes, uint16_t* norms, void* stream) {
  tq_status st = check_weights(cb, rows, k, dtype);
  if (st != TQ_OK) return st;
  if (!w || !codes || !norms) return fail(TQ_ERR_INVALID, "w, codes or norms is NULL");
  if (!aligned16(w) || !aligned16(codes) || !aligned16(norms))
    return fail(TQ_ERR_INVALID, "w, codes and norms must be 16-byte aligned");
  return cuda_status(tq::launch_weights_quantize(cb->tables, w, (int)dtype, rows, k, codes, norms,
                                                 (cudaStream_t)stream),
                     "weights-quantize launch");
}

size_t tq_lut_matmul_workspace_bytes(const tq_codebook* cb, int rows, int k, int m) {
  if (!cb || rows <= 0 || rows % 16 || k <= 0 || k % cb->params.head_dim || m <= 0) return 0;
  return tq::lut_matmul_workspace_bytes(tq::plan_lut_matmul(rows, k, m, cb->params.head_dim, tq::kLutMatmulMaxCtas), rows, m);
}

tq_status tq_lut_matmul(const tq_codebook* cb, const uint8_t* codes, const uint16_t* norms, int rows,
                        int k, const void* x, tq_dtype dtype, int m, float* y, void* workspace,
                        size_t workspace_bytes, void* stream) {
  tq_status st = check_weights(cb, rows, k, dtype);
  if (st != TQ_OK) return st;
  if (m <= 0 || m > 65535 * 4) return fail(TQ_ERR_INVALID, "m %d out of range", m);
  if (!codes || !norms || !x || !y) return fail(TQ_ERR_INVALID, "codes, norms, x or y is NULL");
  if (!aligned16(codes) || !aligned16(norms) || !aligned16(x) || !aligned16(y))
    return fail(TQ_ERR_INVALID, "codes, norms, x and y must be 16-byte aligned");
  const size_t need =
      tq::lut_matmul_workspace_bytes(tq::plan_lut_matmul(rows, k, m, cb->params.head_dim, tq::kLutMatmulMaxCtas), rows, m);
  if (workspace_bytes < need || (need > 0 && !workspace))
    return fail(TQ_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (need > 0 && !aligned16(workspace)) return fail(TQ_ERR_INVALID, "workspace must be 16-byte aligned");
  return cuda_status(tq::launch_lut_matmul(cb->tables, codes, norms, rows, k, x, (int)dtype, m, y,
                                           (float*)workspace, (cudaStream_t)stream),
                     "lut-matmul launch");
}

size_t tq_decode_workspace_bytes(const tq_codebook* cb, int batch, int q_heads, int kv_heads,
                                 int max_ctx) {
  if (!cb || batch <= 0 || q_heads <= 0 || kv_heads <= 0 || max_ctx < 0 ||
      q_heads % kv_heads != 0)
    return 0;
  const tq::DecodePlan plan = tq::plan_decode(batch, kv_heads, max_ctx, tq::kMaxTargetCtas);
  return tq::decode_workspace_bytes(plan, q_heads, kv_heads, cb->params.head_dim);
}

tq_status tq_decode_attention(const tq_codebook* cb, const tq_cache* cache, const void* q,
                              tq_dtype dtype, int q_heads, float softmax_scale, int max_ctx,
                              float* out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (!q || !out) return fail(TQ_ERR_INVALID, "q or out is NULL");
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "unknown dtype %d", (int)dtype);
  if (q_heads <= 0 || q_heads % cache->kv_heads != 0)
    return fail(TQ_ERR_INVALID, "q_heads %d is not a positive multiple of kv_heads %d", q_heads,
                cache->kv_heads);
  if (max_ctx < 0 || max_ctx > cache->capacity)
    return fail(TQ_ERR_INVALID, "max_ctx %d outside [0, capacity %d]", max_ctx, cache->capacity);
  if (!aligned16(q) || !aligned16(out))
    return fail(TQ_ERR_INVALID, "q and out must be 16-byte aligned");
  if (!std::isfinite(softmax_scale)) return fail(TQ_ERR_INVALID, "softmax_scale is not finite");
  const int d = cb->params.head_dim;
  const int group = q_heads / cache->kv_heads;
  if (!tq::decode_supported(d, group, cb->params.k_bits, cb->params.v_bits, cb->params.qjl))
    return fail(TQ_ERR_UNSUPPORTED,
                "no decode kernel for head_dim=%d group=%d k_bits=%d v_bits=%d qjl=%d "
                "(group must be 1, 2, 4 or 8; v_bits must be k_bits or k_bits + 1)",
                d, group, cb->params.k_bits, cb->params.v_bits, cb->params.qjl);
  const tq::DecodePlan plan = tq::plan_decode(cache->batch, cache->kv_heads, max_ctx, tq::kMaxTargetCtas);
  const size_t need = tq::decode_workspace_bytes(plan, q_heads, cache->kv_heads, d);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(TQ_ERR_CAPACITY, "workspace of %zu bytes is smaller than the %zu needed",
                workspace_bytes, need);
  if (need > 0 && !aligned16(workspace))
    return fail(TQ_ERR_INVALID, "workspace must be 16-byte aligned");
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)d);
  return cuda_status(tq::launch_decode(cb->tables, view_of(cache), q, (int)dtype, q_heads, scale,
                                       max_ctx, out, (float*)workspace, (cudaStream_t)stream),
                     "decode launch");
}

tq_status tq_rope_table(const tq_rope_params* params, int max_pos, float* table, void* stream) {
  if (!params) return fail(TQ_ERR_INVALID, "params is NULL");
  if (!table) return fail(TQ_ERR_INVALID, "table is NULL");
  if (!aligned16(table)) return fail(TQ_ERR_INVALID, "table must be 16-byte aligned");
  if (max_pos < 1) return fail(TQ_ERR_INVALID, "max_pos %d: at least 1", max_pos);
  tq::RopeFrequencies rf;
  const tq_status st = rope_frequencies(*params, &rf);
  if (st != TQ_OK) return st;
  return cuda_status(tq::launch_rope_table(rf, params->rot_dim / 2, max_pos, table, (cudaStream_t)stream),
                     "rope-table launch");
}

tq_status tq_rope_append(const tq_codebook* cb, const tq_cache* cache, const tq_rope* rope,
                         const tq_heads* q, int q_heads, const tq_heads* k, const tq_heads* v,
                         tq_dtype dtype, int n_new, const int32_t* positions, int relative,
                         const int32_t* start, void* q_out, void* k_out, void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (!rope || !rope->table) return fail(TQ_ERR_INVALID, "rope or its table is NULL");
  const int d = cb->params.head_dim;
  if (rope->rot_dim < 2 || rope->rot_dim % 2 || rope->rot_dim > d)
    return fail(TQ_ERR_INVALID, "rot_dim %d: even, 2 .. head_dim %d", rope->rot_dim, d);
  if (rope->max_pos < 1) return fail(TQ_ERR_INVALID, "rope max_pos %d: at least 1", rope->max_pos);
  if (!aligned16(rope->table)) return fail(TQ_ERR_INVALID, "rope table must be 16-byte aligned");
  if (n_new < 0) return fail(TQ_ERR_INVALID, "n_new %d is negative", n_new);
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "unknown dtype %d", (int)dtype);
  if (n_new > cache->capacity)
    return fail(TQ_ERR_INVALID, "n_new %d exceeds capacity %d", n_new, cache->capacity);
  if (q && q_heads <= 0) return fail(TQ_ERR_INVALID, "q_heads %d must be positive", q_heads);
  if (n_new == 0) return ok();
  if (!k || !v || !k->data || !v->data) return fail(TQ_ERR_INVALID, "k or v is NULL");
  if (q && (!q->data || !q_out)) return fail(TQ_ERR_INVALID, "q needs data and q_out");
  const tq_heads* views[] = {k, v, q};
  const char* names[] = {"k", "v", "q"};
  const int64_t esz = dtype == TQ_F32 ? 4 : 2;
  for (int i = 0; i < (q ? 3 : 2); ++i) {
    const tq_heads& h = *views[i];
    if (h.stride_b < 0 || h.stride_h < 0 || h.stride_t < 0)
      return fail(TQ_ERR_INVALID, "%s has a negative stride", names[i]);
    if ((h.stride_b * esz) % 16 || (h.stride_h * esz) % 16 || (h.stride_t * esz) % 16)
      return fail(TQ_ERR_INVALID, "strides of %s (%lld, %lld, %lld) are not multiples of 16 bytes", names[i],
                  (long long)h.stride_b, (long long)h.stride_h, (long long)h.stride_t);
    if (!aligned16(h.data)) return fail(TQ_ERR_INVALID, "%s must be 16-byte aligned", names[i]);
  }
  if (!aligned16(q_out) || !aligned16(k_out))
    return fail(TQ_ERR_INVALID, "q_out and k_out must be 16-byte aligned");
  if ((uintptr_t)positions % 4 || (uintptr_t)start % 4)
    return fail(TQ_ERR_INVALID, "positions and start must be 4-byte aligned");
  // blocks read one token's heads while others write: no output may lie where an input does
  struct Range {
    uintptr_t lo, hi;
    bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
  };
  auto dense = [&](const void* p, int heads) {
    const uintptr_t at = (uintptr_t)p;
    return Range{at, p ? at + (uintptr_t)esz * cache->batch * n_new * heads * d : at};
  };
  const int counts[] = {cache->kv_heads, cache->kv_heads, q ? q_heads : 0};
  const Range outs[] = {dense(q ? q_out : nullptr, counts[2]), dense(k_out, counts[0])};
  for (int i = 0; i < (q ? 3 : 2); ++i) {
    const tq_heads& h = *views[i];
    const uintptr_t last = (uintptr_t)(h.stride_b * (cache->batch - 1) + h.stride_h * (counts[i] - 1) +
                                       h.stride_t * (int64_t)(n_new - 1) + d);
    const Range in{(uintptr_t)h.data, (uintptr_t)h.data + (uintptr_t)esz * last};
    if (in.meets(outs[0]) || in.meets(outs[1])) return fail(TQ_ERR_INVALID, "q_out or k_out overlaps %s", names[i]);
  }
  if (outs[0].meets(outs[1])) return fail(TQ_ERR_INVALID, "q_out and k_out overlap");
  tq::RopeAppend ra;
  ra.table = rope->table;
  ra.max_pos = rope->max_pos;
  ra.rot_dim = rope->rot_dim;
  ra.interleaved = rope->interleaved != 0;
  auto heads = [](const tq_heads* h) {
    return h ? tq::Heads{h->data, (long)h->stride_b, (long)h->stride_h, (long)h->stride_t} : tq::Heads{};
  };
  ra.q = heads(q);
  ra.k = heads(k);
  ra.v = heads(v);
  ra.q_out = q ? q_out : nullptr;
  ra.k_out = k_out;
  ra.positions = positions;
  ra.start = start;
  ra.relative = relative != 0;
  ra.q_heads = q ? q_heads : 0;
  ra.n_new = n_new;
  return cuda_status(tq::launch_rope_append(cb->tables, view_of(cache), ra, (int)dtype, (cudaStream_t)stream),
                     "rope-append launch");
}

tq_status tq_cache_compact(const tq_codebook* cb, const tq_cache* cache, const int32_t* index,
                           int64_t stride_b, int64_t stride_h, const int32_t* counts, int max_count,
                           const int32_t* start, void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (!counts || (!index && max_count > 0)) return fail(TQ_ERR_INVALID, "index or counts is NULL");
  if (max_count < 0 || max_count > cache->capacity)
    return fail(TQ_ERR_INVALID, "max_count %d outside [0, capacity %d]", max_count, cache->capacity);
  if (stride_b < 0 || stride_h < 0) return fail(TQ_ERR_INVALID, "negative stride");
  if ((uintptr_t)index % 4 || (uintptr_t)counts % 4 || (uintptr_t)start % 4)
    return fail(TQ_ERR_INVALID, "index, counts and start must be 4-byte aligned");
  if (cache->kv_heads > 65535) return fail(TQ_ERR_INVALID, "kv_heads %d: at most 65535", cache->kv_heads);
  return cuda_status(tq::launch_cache_compact(arrays_of(cb, cache), view_of(cache), index, (long)stride_b,
                                              (long)stride_h, counts, max_count, start, (cudaStream_t)stream),
                     "cache-compact launch");
}

tq_status tq_cache_copy(const tq_codebook* cb, const tq_cache* dst, const tq_cache* src,
                        const int32_t* dst_rows, const int32_t* src_rows, const int32_t* lengths,
                        int n, int max_len, void* stream) {
  tq_status st = check_cache(cb, dst);
  if (st != TQ_OK) return st;
  st = check_cache(cb, src);
  if (st != TQ_OK) return st;
  if (dst->kv_heads != src->kv_heads)
    return fail(TQ_ERR_INVALID, "kv_heads differ (dst %d, src %d)", dst->kv_heads, src->kv_heads);
  if (dst->kv_heads > 65535) return fail(TQ_ERR_INVALID, "kv_heads %d: at most 65535", dst->kv_heads);
  const tq::SlotArrays da = arrays_of(cb, dst), sa = arrays_of(cb, src);
  if (overlap(da, dst, sa, src))
    return fail(TQ_ERR_INVALID, "dst and src overlap in memory, but are not one cache");
  if (n < 0 || n > 65535) return fail(TQ_ERR_INVALID, "n %d outside [0, 65535]", n);
  if (max_len < 0) return fail(TQ_ERR_INVALID, "max_len %d is negative", max_len);
  if (n == 0) return ok();
  if (!dst_rows || !src_rows) return fail(TQ_ERR_INVALID, "dst_rows or src_rows is NULL");
  if ((uintptr_t)dst_rows % 4 || (uintptr_t)src_rows % 4 || (uintptr_t)lengths % 4)
    return fail(TQ_ERR_INVALID, "dst_rows, src_rows and lengths must be 4-byte aligned");
  return cuda_status(tq::launch_cache_copy(da, view_of(dst), sa, view_of(src), dst_rows, src_rows, lengths, n, max_len,
                                           (cudaStream_t)stream),
                     "cache-copy launch");
}

size_t tq_tree_workspace_bytes(const tq_codebook* cb, int batch, int q_heads, int kv_heads, int n_q,
                               int max_ctx) {
  if (!cb || batch <= 0 || q_heads <= 0 || kv_heads <= 0 || max_ctx < 0 || q_heads % kv_heads != 0 ||
      n_q < 1 || n_q > 256)
    return 0;
  return tq::tree_workspace_bytes(cb->tables, batch, q_heads, kv_heads, n_q, max_ctx);
}

tq_status tq_tree_attention(const tq_codebook* cb, const tq_cache* cache, const void* q,
                            tq_dtype dtype, int q_heads, int n_q, const uint32_t* mask,
                            int64_t mask_stride, float softmax_scale, int max_ctx, void* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_cache(cb, cache);
  if (st != TQ_OK) return st;
  if (!q || !out) return fail(TQ_ERR_INVALID, "q or out is NULL");
  if (dtype != TQ_BF16 && dtype != TQ_F16)
    return fail(TQ_ERR_INVALID, "dtype %d: the tree attention takes bf16 or fp16", (int)dtype);
  if (n_q < 1 || n_q > 256) return fail(TQ_ERR_INVALID, "n_q %d outside [1, 256]", n_q);
  if (q_heads <= 0 || q_heads % cache->kv_heads != 0)
    return fail(TQ_ERR_INVALID, "q_heads %d is not a positive multiple of kv_heads %d", q_heads,
                cache->kv_heads);
  if (max_ctx < 0 || max_ctx > cache->capacity)
    return fail(TQ_ERR_INVALID, "max_ctx %d outside [0, capacity %d]", max_ctx, cache->capacity);
  if (!aligned16(q) || !aligned16(out)) return fail(TQ_ERR_INVALID, "q and out must be 16-byte aligned");
  if ((uintptr_t)mask % 4) return fail(TQ_ERR_INVALID, "mask must be 4-byte aligned");
  if (mask && mask_stride != 0 && mask_stride < (int64_t)n_q * ((n_q + 31) / 32))
    return fail(TQ_ERR_INVALID, "mask_stride %lld is neither 0 nor a whole mask", (long long)mask_stride);
  if (!std::isfinite(softmax_scale)) return fail(TQ_ERR_INVALID, "softmax_scale is not finite");
  const int d = cb->params.head_dim, group = q_heads / cache->kv_heads;
  if (!tq::decode_supported(d, group, cb->params.k_bits, cb->params.v_bits, cb->params.qjl))
    return fail(TQ_ERR_UNSUPPORTED,
                "no tree attention for head_dim=%d group=%d k_bits=%d v_bits=%d qjl=%d "
                "(group must be 1, 2, 4 or 8; v_bits must be k_bits or k_bits + 1)",
                d, group, cb->params.k_bits, cb->params.v_bits, cb->params.qjl);
  const size_t need = tq::tree_workspace_bytes(cb->tables, cache->batch, q_heads, cache->kv_heads, n_q, max_ctx);
  if (need == 0)
    return fail(TQ_ERR_UNSUPPORTED, "no tree attention for head_dim=%d k_bits=%d v_bits=%d qjl=%d: its buffers do not fit",
                d, cb->params.k_bits, cb->params.v_bits, cb->params.qjl);
  if (!workspace || workspace_bytes < need)
    return fail(TQ_ERR_CAPACITY, "workspace of %zu bytes is smaller than the %zu needed",
                workspace_bytes, need);
  if (!aligned16(workspace)) return fail(TQ_ERR_INVALID, "workspace must be 16-byte aligned");
  tq::TreeArgs ta;
  ta.q = q;
  ta.out = out;
  ta.mask = mask;
  ta.mask_stride = (long)mask_stride;
  ta.dtype = (int)dtype;
  ta.q_heads = q_heads;
  ta.n_q = n_q;
  ta.max_ctx = max_ctx;
  ta.log_group = group == 8 ? 3 : group == 4 ? 2 : group == 2 ? 1 : 0;
  ta.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)d);
  return cuda_status(tq::launch_tree(cb->tables, view_of(cache), ta, (float*)workspace, (cudaStream_t)stream),
                     "tree-attention launch");
}

void tq_free(tq_codebook* cb) { delete cb; }

const char* tq_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
