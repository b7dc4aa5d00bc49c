// C ABI of the paged K/V cache (include/qi21.h): the rotation's frequencies
// on the host, argument validation, and the launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/qi21.h"
#include "internal.h"

namespace qi21 {

static int refuse(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}

static int cuda_refuse(cudaError_t e, const char* what) {
  return refuse(QI21_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

static bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// The frequencies (angle per position) of an axis of width d.
static double rope_freq(int j, int d, double base, int kind, double factor, double orig_len, double fast, double slow) {
  if (kind == QI21_ROPE_BASE && d > 2) base *= std::pow(factor, static_cast<double>(d) / (d - 2));
  const double f = std::pow(base, -2.0 * j / d);
  const double two_pi = 6.283185307179586476925;
  if (kind == QI21_ROPE_LINEAR) return f / factor;
  if (kind == QI21_ROPE_RAMP) {
    auto pair_of = [&](double n) { return d * std::log(orig_len / (two_pi * n)) / (2.0 * std::log(base)); };
    const double lo = std::fmax(0.0, std::floor(pair_of(fast)));
    const double hi = std::fmin(d - 1.0, std::ceil(pair_of(slow)));
    const double r = std::fmin(1.0, std::fmax(0.0, (j - lo) / std::fmax(hi - lo, 1e-3)));
    return f * (1.0 - r) + f * r / factor;
  }
  if (kind == QI21_ROPE_BAND) {
    const double r = std::fmin(1.0, std::fmax(0.0, (orig_len * f / two_pi - slow) / (fast - slow)));
    return f * r + f * (1.0 - r) / factor;
  }
  return f;
}

static int check_rope(const qi21_rope* r) {
  if (r == nullptr) return refuse(QI21_ERR_ARG, "null rope");
  if (r->head_dim < 2 || r->head_dim > 256 || r->head_dim % 2)
    return refuse(QI21_ERR_GEOM, "rope head_dim %d (even, 2 .. 256)", r->head_dim);
  if (r->rot_dim < 2 || r->rot_dim > r->head_dim || r->rot_dim % 2)
    return refuse(QI21_ERR_GEOM, "rope rot_dim %d (even, 2 .. head_dim %d)", r->rot_dim, r->head_dim);
  if (r->layout != QI21_ROPE_INTERLEAVED && r->layout != QI21_ROPE_HALF)
    return refuse(QI21_ERR_ARG, "rope layout %d", r->layout);
  if (r->naxes != 1 && r->naxes != 3) return refuse(QI21_ERR_ARG, "rope naxes %d (1 or 3)", r->naxes);
  if (!(std::fabs(r->out_scale) <= 3.0e38f)) return refuse(QI21_ERR_ARG, "rope out_scale is not finite");
  for (int j = 0; j < r->rot_dim / 2; ++j)
    if (r->axis[j] >= r->naxes) return refuse(QI21_ERR_ARG, "rope pair %d: axis %d of %d", j, r->axis[j], r->naxes);
  return QI21_OK;
}

static RopeDev rope_dev(const qi21_rope* r) {
  static_assert(kRopePairs == QI21_ROPE_MAX_PAIRS, "pairs");
  RopeDev d;
  memset(&d, 0, sizeof d);
  if (r == nullptr) return d;
  d.rot = r->rot_dim;
  d.naxes = r->naxes;
  d.scale = r->out_scale;
  memcpy(d.axis, r->axis, sizeof d.axis);
  memcpy(d.turns, r->turns, sizeof d.turns);
  return d;
}

static int check_paged(const qi21_paged* kv) {
  if (kv == nullptr) return refuse(QI21_ERR_ARG, "null paged cache");
  if (kv->dtype != QI21_DTYPE_F16 && kv->dtype != QI21_DTYPE_BF16) return refuse(QI21_ERR_ARG, "dtype %d", kv->dtype);
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return refuse(QI21_ERR_GEOM, "head_dim %d (64 or 128)", kv->head_dim);
  if (kv->kv_heads < 1 || kv->kv_heads > 1024) return refuse(QI21_ERR_GEOM, "kv_heads %d (1 .. 1024)", kv->kv_heads);
  if (kv->page_rows < 16 || kv->page_rows % 16 || kv->page_rows > (1 << 20))
    return refuse(QI21_ERR_GEOM, "page_rows %d (a multiple of 16)", kv->page_rows);
  if (kv->npages < 1 || static_cast<int64_t>(kv->npages) * kv->page_rows > 0x7fffffff)
    return refuse(QI21_ERR_SHAPE, "npages %d of %d rows (at least one page, at most 2^31 - 1 rows in all)", kv->npages, kv->page_rows);
  if (kv->nseq < 0 || kv->table_stride < 0 || kv->prefix_len < 0 || kv->prefix_len >= (1 << 30))
    return refuse(QI21_ERR_SHAPE, "nseq %d table_stride %d prefix_len %d", kv->nseq, kv->table_stride, kv->prefix_len);
  return QI21_OK;
}

static int check_paged_ptrs(const qi21_paged* kv) {
  if (!kv->cu || !kv->lens || (kv->table_stride > 0 && !kv->table) || !kv->pool ||
      (kv->prefix_len > 0 && !kv->prefix_pages))
    return refuse(QI21_ERR_ARG, "null pointer in the paged cache");
  if (misaligned(kv->pool, 16)) return refuse(QI21_ERR_ARG, "the pool must be 16-byte aligned");
  return QI21_OK;
}

static PagedArgs paged_args(const qi21_paged* kv) {
  PagedArgs p{};
  p.pool = kv->pool;
  p.dt = kv->dtype;
  p.npages = kv->npages;
  p.page_rows = kv->page_rows;
  p.kv_heads = kv->kv_heads;
  p.dim = kv->head_dim;
  p.nseq = kv->nseq;
  p.table = kv->table;
  p.table_stride = kv->table_stride;
  const int64_t cap = static_cast<int64_t>(kv->table_stride) * kv->page_rows;
  p.table_rows = static_cast<int>(cap < (1 << 30) ? cap : (1 << 30));
  p.lens = kv->lens;
  p.cu = kv->cu;
  p.prefix_pages = kv->prefix_pages;
  p.prefix_len = kv->prefix_len;
  return p;
}

}  // namespace qi21

using namespace qi21;

extern "C" {

int qi21_rope_init(qi21_rope* r, int32_t head_dim, int32_t rot_dim, int32_t layout, const int32_t* axes, double base,
                   int32_t kind, double factor, double orig_len, double fast_turns, double slow_turns,
                   double out_scale) {
  if (r == nullptr) return refuse(QI21_ERR_ARG, "null rope");
  qi21_rope t;
  memset(&t, 0, sizeof t);
  t.head_dim = head_dim;
  t.rot_dim = rot_dim;
  t.layout = layout;
  t.naxes = axes ? 3 : 1;
  t.out_scale = 1.f;
  int rc = check_rope(&t);
  if (rc != QI21_OK) return rc;
  if (!(base > 1.0) || !std::isfinite(base)) return refuse(QI21_ERR_ARG, "rope base %g (must be > 1)", base);
  if (kind < QI21_ROPE_PLAIN || kind > QI21_ROPE_BAND) return refuse(QI21_ERR_ARG, "rope kind %d", kind);
  if (!(factor >= 1.0) || !std::isfinite(factor)) return refuse(QI21_ERR_ARG, "rope factor %g (must be >= 1)", factor);
  if (kind == QI21_ROPE_RAMP || kind == QI21_ROPE_BAND) {
    if (fast_turns == 0.0) fast_turns = kind == QI21_ROPE_RAMP ? 32.0 : 4.0;
    if (slow_turns == 0.0) slow_turns = 1.0;
    if (!(orig_len >= 1.0) || !std::isfinite(orig_len)) return refuse(QI21_ERR_ARG, "rope orig_len %g", orig_len);
    if (!(slow_turns > 0.0) || !(fast_turns > slow_turns) || !std::isfinite(fast_turns))
      return refuse(QI21_ERR_ARG, "rope turns %g, %g (fast > slow > 0)", fast_turns, slow_turns);
  }
  if (out_scale == 0.0) out_scale = kind == QI21_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  if (!(std::fabs(out_scale) <= 3.0e38)) return refuse(QI21_ERR_ARG, "rope out_scale is not finite");
  t.out_scale = static_cast<float>(out_scale);
  const int whole[1] = {rot_dim};
  const int32_t* width = axes ? axes : whole;
  int sum = 0;
  for (int a = 0; a < t.naxes; ++a) {
    if (width[a] < 0 || width[a] % 2 || width[a] > rot_dim)
      return refuse(QI21_ERR_GEOM, "RoPE axis %d width %d must be even and at most rot_dim", a, width[a]);
    sum += width[a];
  }
  if (sum != rot_dim) return refuse(QI21_ERR_GEOM, "RoPE axes sum to %d, rot_dim %d", sum, rot_dim);
  int k = 0;
  for (int a = 0; a < t.naxes; ++a)
    for (int j = 0; j < width[a] / 2; ++j, ++k) {
      // turns per position in (0, 1): the fraction of 2^64, to f64 precision
      const double turns = rope_freq(j, width[a], base, kind, factor, orig_len, fast_turns, slow_turns) /
                           6.283185307179586476925;
      t.axis[k] = static_cast<uint8_t>(a);
      t.turns[k] = static_cast<uint64_t>(std::ldexp(turns, 64));
    }
  *r = t;
  return QI21_OK;
}

int qi21_op_rope(const qi21_rope* r, int32_t elem_type, int32_t rows, int32_t heads, const void* x, int64_t ldx,
                 void* out, int64_t ldo, const int64_t* pos, int32_t grad, void* stream) {
  const int rc = check_rope(r);
  if (rc != QI21_OK) return rc;
  if (elem_type != QI21_ELEM_F16 && elem_type != QI21_ELEM_BF16 && elem_type != QI21_ELEM_F32)
    return refuse(QI21_ERR_ARG, "elem_type %d (QI21_ELEM_F16, _BF16 or _F32)", elem_type);
  if (grad != 0 && grad != 1) return refuse(QI21_ERR_ARG, "grad %d (0 or 1)", grad);
  if (rows < 0 || heads < 1 || heads > 1024) return refuse(QI21_ERR_SHAPE, "rows %d heads %d", rows, heads);
  const int64_t wide = static_cast<int64_t>(heads) * r->head_dim;
  if (ldx < wide || ldo < wide)
    return refuse(QI21_ERR_SHAPE, "ldx %lld ldo %lld below heads * head_dim %lld", static_cast<long long>(ldx),
                  static_cast<long long>(ldo), static_cast<long long>(wide));
  if (rows == 0) return QI21_OK;
  if (!x || !out || !pos) return refuse(QI21_ERR_ARG, "null pointer");
  const size_t eb = elem_type == QI21_ELEM_F32 ? 4 : 2;
  if (misaligned(x, eb) || misaligned(out, eb) || misaligned(pos, 8))
    return refuse(QI21_ERR_ARG, "x, out and pos must be aligned to their elements");
  if (x == out && ldx != ldo) return refuse(QI21_ERR_ARG, "in place, ldo must be ldx");
  const cudaError_t e = launch_rope(rope_dev(r), r->layout == QI21_ROPE_HALF, elem_type, rows, heads, r->head_dim, x,
                                    ldx, out, ldo, pos, grad != 0, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI21_OK : cuda_refuse(e, "rope");
}

int qi21_op_kv_append(const qi21_paged* kv, int32_t rows, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      const qi21_rope* rope, const int64_t* pos, void* stream) {
  int rc = check_paged(kv);
  if (rc != QI21_OK) return rc;
  if (rows < 0) return refuse(QI21_ERR_SHAPE, "rows %d", rows);
  const int64_t wide = static_cast<int64_t>(kv->kv_heads) * kv->head_dim;
  if (ldk < wide || ldv < wide)
    return refuse(QI21_ERR_SHAPE, "ldk %lld ldv %lld below kv_heads * head_dim %lld", static_cast<long long>(ldk),
                  static_cast<long long>(ldv), static_cast<long long>(wide));
  if (rope) {
    if ((rc = check_rope(rope)) != QI21_OK) return rc;
    if (rope->head_dim != kv->head_dim)
      return refuse(QI21_ERR_SHAPE, "rope head_dim %d, cache %d", rope->head_dim, kv->head_dim);
    if (rope->naxes != 1 && pos == nullptr) return refuse(QI21_ERR_ARG, "three-axis positions must be given");
  }
  if (rows == 0 || kv->nseq == 0) return QI21_OK;
  if (!k || !v) return refuse(QI21_ERR_ARG, "null pointer");
  if (misaligned(k, 2) || misaligned(v, 2) || misaligned(pos, 8))
    return refuse(QI21_ERR_ARG, "k, v and pos must be aligned to their elements");
  if ((rc = check_paged_ptrs(kv)) != QI21_OK) return rc;
  const cudaError_t e = launch_kv_append(paged_args(kv), rope_dev(rope), rope && rope->layout == QI21_ROPE_HALF, rows,
                                         k, ldk, v, ldv, pos, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI21_OK : cuda_refuse(e, "kv append");
}

static int check_heads(const qi21_paged* kv, int32_t rows, int32_t heads) {
  const int rc = check_paged(kv);
  if (rc != QI21_OK) return rc;
  if (rows < 0 || rows > (1 << 24)) return refuse(QI21_ERR_SHAPE, "rows %d (at most 2^24)", rows);
  if (heads < 1 || heads > 1024 || heads % kv->kv_heads)
    return refuse(QI21_ERR_SHAPE, "heads %d (a multiple of kv_heads %d, at most 1024)", heads, kv->kv_heads);
  if (static_cast<int64_t>(rows) * heads > (1 << 30))
    return refuse(QI21_ERR_SHAPE, "rows * heads above 2^30 (%d * %d)", rows, heads);
  return QI21_OK;
}

size_t qi21_attention_paged_bytes(const qi21_paged* kv, int32_t rows, int32_t heads) {
  if (check_heads(kv, rows, heads) != QI21_OK) return 0;
  return attn_paged_bytes(paged_args(kv), rows, heads);
}

int qi21_op_attention_paged(const qi21_paged* kv, int32_t rows, int32_t heads, const void* q, int64_t ldq, void* out,
                            int64_t ldo, int32_t causal, const uint32_t* vis, float scale, void* workspace,
                            size_t ws_bytes, void* stream) {
  int rc = check_heads(kv, rows, heads);
  if (rc != QI21_OK) return rc;
  const int64_t wide = static_cast<int64_t>(heads) * kv->head_dim;
  if (ldq < wide || ldo < wide || ldq % 8 || ldo % 8)
    return refuse(QI21_ERR_SHAPE, "ldq %lld ldo %lld (at least heads * head_dim %lld, multiples of 8)",
                  static_cast<long long>(ldq), static_cast<long long>(ldo), static_cast<long long>(wide));
  if (!(scale > 0.f) || !(scale <= 1e38f)) return refuse(QI21_ERR_ARG, "scale must be > 0 and at most 1e38");
  if (rows == 0 || kv->nseq == 0) return QI21_OK;
  if (!q || !out) return refuse(QI21_ERR_ARG, "null pointer");
  if (misaligned(q, 16) || misaligned(out, 16)) return refuse(QI21_ERR_ARG, "q and out must be 16-byte aligned");
  if (misaligned(vis, 4)) return refuse(QI21_ERR_ARG, "vis not aligned to its element");
  if ((rc = check_paged_ptrs(kv)) != QI21_OK) return rc;
  const PagedArgs p = paged_args(kv);
  const size_t need = attn_paged_bytes(p, rows, heads);
  if (workspace == nullptr) return refuse(QI21_ERR_WORKSPACE, "null workspace");
  if (misaligned(workspace, 256)) return refuse(QI21_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return refuse(QI21_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, need);
  const cudaError_t e = launch_attn_paged(p, rows, heads, q, ldq, out, ldo, causal != 0, vis, scale, workspace,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QI21_OK : cuda_refuse(e, "paged attention");
}

}  // extern "C"
