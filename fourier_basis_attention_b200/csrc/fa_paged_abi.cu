// fa_paged_abi.cu -- the extern "C" entry points of rotary positions and of the paged cache:
// argument checks and launches. See include/fourier_attention.h for the contract.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "fa_host.h"

namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return fa::set_last_error(code, buf);
}

int launched(cudaError_t e, const char* where, const char* why = nullptr) {
  if (e == cudaSuccess) return FA_OK;
  if (why) return fail(FA_ERR_CUDA, "%s: %s", where, why);
  return fail(FA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

int check_ptr(const void* p, const char* name, unsigned align = 16) {
  if (!p) return fail(FA_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return fail(FA_ERR_INVALID, "%s is not %u-byte aligned", name, align);
  return FA_OK;
}

int check_shape(const fa_paged_shape* shape) {
  if (!shape) return fail(FA_ERR_INVALID, "shape is NULL");
  const fa_paged_shape& s = *shape;
  if (s.D != FA_HEAD_DIM) return fail(FA_ERR_UNSUPPORTED, "head dim %d != 128", s.D);
  if (s.B < 0 || s.Hkv < 1 || s.Hq < 1 || s.Hq % s.Hkv != 0 || s.page_size < 1 ||
      s.num_pages < 1 || s.max_pages < 0 || s.total_q < 0 || s.max_q < 0 || s.max_kv < 0)
    return fail(FA_ERR_INVALID,
                "shape fields out of range (B=%d Hq=%d Hkv=%d page_size=%d num_pages=%d "
                "max_pages=%d total_q=%d max_q=%d max_kv=%d)",
                s.B, s.Hq, s.Hkv, s.page_size, s.num_pages, s.max_pages, s.total_q, s.max_q,
                s.max_kv);
  if (s.B > 65535) return fail(FA_ERR_UNSUPPORTED, "B=%d exceeds 65535", s.B);
  if (s.Hq > FA_MAX_Q_HEADS)
    return fail(FA_ERR_UNSUPPORTED, "Hq=%d exceeds %d", s.Hq, FA_MAX_Q_HEADS);
  if (s.max_kv > (long long)s.max_pages * s.page_size)
    return fail(FA_ERR_INVALID, "max_kv=%d exceeds max_pages x page_size = %d x %d", s.max_kv,
                s.max_pages, s.page_size);
  if (s.max_kv >= 1 << 30) return fail(FA_ERR_UNSUPPORTED, "max_kv=%d is not below 2^30", s.max_kv);
  if ((double)s.num_pages * s.Hkv * s.page_size >= 2147483648.0)
    return fail(FA_ERR_UNSUPPORTED, "num_pages x Hkv x page_size = %d x %d x %d is not below 2^31",
                s.num_pages, s.Hkv, s.page_size);
  if (s.total_q >= (1 << 30) / s.Hq)
    return fail(FA_ERR_UNSUPPORTED, "total_q x Hq = %d x %d is not below 2^30", s.total_q, s.Hq);
  return FA_OK;
}

// Shape, pools and table; the batch arrays where `batch` is set (rows of new tokens).
int check_cache(const fa_paged_shape* shape, const fa_paged_cache* cache, bool batch, bool values) {
  if (int r = check_shape(shape)) return r;
  if (!cache) return fail(FA_ERR_INVALID, "cache is NULL");
  if (int r = check_ptr(cache->K, "cache->K")) return r;
  if (values)
    if (int r = check_ptr(cache->V, "cache->V")) return r;
  if (shape->B == 0) return FA_OK;
  if (shape->max_kv > 0)
    if (int r = check_ptr(cache->page_table, "cache->page_table", 4)) return r;
  if (batch) {
    if (int r = check_ptr(cache->q_start, "cache->q_start", 4)) return r;
    if (int r = check_ptr(cache->kv_len, "cache->kv_len", 4)) return r;
  }
  return FA_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A [total_q][heads][128] bf16 tensor with a token stride.
int check_rows(const void* p, int64_t stride, int heads, const char* name) {
  if (int r = check_ptr(p, name)) return r;
  if (stride < (int64_t)heads * FA_HEAD_DIM || stride % 8 != 0)
    return fail(FA_ERR_INVALID, "%s_stride=%lld must be a multiple of 8, at least %d", name,
                (long long)stride, heads * FA_HEAD_DIM);
  return FA_OK;
}

int check_rope(const fa_rope_plan* rope) {
  if (!rope) return fail(FA_ERR_INVALID, "rope is NULL");
  if (rope->rot_dim < 2 || rope->rot_dim > FA_HEAD_DIM || rope->rot_dim % 2 != 0 ||
      (rope->interleaved != 0 && rope->interleaved != 1) || !isfinite(rope->magnitude))
    return fail(FA_ERR_INVALID, "rope plan is inconsistent (rot_dim=%d interleaved=%d)",
                rope->rot_dim, rope->interleaved);
  return FA_OK;
}

int check_softmax(const fa_paged_shape& s, float* scale, int32_t* window) {
  if (s.page_size % 16 != 0 && s.max_kv > s.page_size)
    return fail(FA_ERR_UNSUPPORTED, "page_size=%d is not a multiple of 16 (max_kv=%d takes several pages)",
                s.page_size, s.max_kv);
  if (!isfinite(*scale) || *scale < 0.0f)
    return fail(FA_ERR_INVALID, "scale must be finite and >= 0");
  if (*scale != 0.0f && (*scale < 1e-20f || *scale > 1e20f))
    return fail(FA_ERR_UNSUPPORTED, "scale=%g is outside [1e-20, 1e20]", *scale);
  if (*window < 0) return fail(FA_ERR_INVALID, "window=%d is negative", *window);
  if (*window >= s.max_kv) *window = 0;  // hides nothing
  if (*scale == 0.0f) *scale = 0.08838834764831845f;  // 1 / sqrt(128)
  return FA_OK;
}

// Strides of [n0][n1][n2][128] rows: multiples of 16 bytes, >= 0; `apart`: rows do not overlap. An
// axis of size 1 may have any.
int check_row_strides(const int64_t* st, const int64_t* n, int elem, bool apart, const char* name) {
  if (!st) return fail(FA_ERR_INVALID, "%s_stride is NULL", name);
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] < 0 || st[i] > (1LL << 40) || st[i] * elem % 16 != 0))
      return fail(FA_ERR_INVALID, "%s_stride[%d]=%lld must be a multiple of 16 bytes, >= 0", name, i,
                  (long long)st[i]);
  if (!apart) return FA_OK;
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[order[j]] < st[order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  int64_t extent = FA_HEAD_DIM;
  for (int i = 0; i < 3; ++i) {
    const int a = order[i];
    if (n[a] <= 1) continue;
    if (st[a] < extent)
      return fail(FA_ERR_INVALID, "rows of %s overlap (stride %lld of axis %d)", name,
                  (long long)st[a], a);
    extent += (n[a] - 1) * st[a];
  }
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_rope_init(const fa_rope_config* config, fa_rope_plan* rope) {
  if (!config || !rope) return fail(FA_ERR_INVALID, "NULL argument");
  const fa_rope_config& c = *config;
  if (c.rot_dim < 2 || c.rot_dim > FA_HEAD_DIM || c.rot_dim % 2 != 0)
    return fail(FA_ERR_INVALID, "rot_dim=%d must be even, 2 to 128", c.rot_dim);
  if (c.interleaved != 0 && c.interleaved != 1)
    return fail(FA_ERR_INVALID, "interleaved=%d must be 0 or 1", c.interleaved);
  if (c.scaling < FA_ROPE_PLAIN || c.scaling > FA_ROPE_YARN)
    return fail(FA_ERR_INVALID, "unknown scaling %d", c.scaling);
  if (!(c.base > 1.0) || !isfinite(c.base) || !(c.factor >= 1.0) || !isfinite(c.factor) ||
      !(c.magnitude >= 0.0) || c.magnitude > 1e30)
    return fail(FA_ERR_INVALID, "base must exceed 1, factor be at least 1, magnitude at least 0");
  if (c.scaling == FA_ROPE_BANDS || c.scaling == FA_ROPE_YARN)
    if (!(c.low > 0.0) || !(c.high > c.low) || !isfinite(c.high) || c.original_len < 1)
      return fail(FA_ERR_INVALID, "need 0 < low < high and original_len >= 1");
  fa::rope_init(config, rope);
  return FA_OK;
}

int fa_rope(const fa_rope_plan* rope, int32_t B, int32_t T, int32_t H, const int32_t* positions,
            const void* x, const int64_t* x_stride, void* y, const int64_t* y_stride,
            int32_t dtype, int32_t transpose, void* stream) {
  if (int r = check_rope(rope)) return r;
  if (B < 0 || T < 0 || H < 0) return fail(FA_ERR_INVALID, "B=%d T=%d H=%d", B, T, H);
  if (dtype != FA_BF16 && dtype != FA_F32) return fail(FA_ERR_INVALID, "unknown dtype %d", dtype);
  if (transpose != 0 && transpose != 1)
    return fail(FA_ERR_INVALID, "transpose=%d must be 0 or 1", transpose);
  if ((long long)B * T >= (1LL << 30) || H > (1 << 20))
    return fail(FA_ERR_UNSUPPORTED, "B x T = %d x %d or H = %d too large", B, T, H);
  const int64_t n[3] = {B, T, H};
  const int elem = dtype == FA_F32 ? 4 : 2;
  if (int r = check_row_strides(x_stride, n, elem, false, "x")) return r;
  if (int r = check_row_strides(y_stride, n, elem, true, "y")) return r;
  if (B == 0 || T == 0 || H == 0) return FA_OK;
  if (int r = check_ptr(positions, "positions", 4)) return r;
  if (int r = check_ptr(x, "x")) return r;
  if (int r = check_ptr(y, "y")) return r;
  if (x == y)
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && x_stride[i] != y_stride[i])
        return fail(FA_ERR_INVALID, "y is x, but stride %d differs", i);
  return launched(fa::launch_rope(rope, B, T, H, positions, x, x_stride, y, y_stride, dtype,
                                  transpose, static_cast<cudaStream_t>(stream)),
                  "fa_rope: launch");
}

int fa_paged_append(const fa_paged_shape* shape, const fa_paged_cache* cache,
                    const fa_rope_plan* rope, const int32_t* positions, const void* q,
                    int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
  if (int r = check_cache(shape, cache, true, true)) return r;
  if (rope)
    if (int r = check_rope(rope)) return r;
  if ((q != nullptr) != (q_out != nullptr))
    return fail(FA_ERR_INVALID, "q and q_out come together");
  if (!rope && (q || positions))
    return fail(FA_ERR_INVALID, "q, q_out and positions need a rope plan");
  const fa_paged_shape& s = *shape;
  if (s.B == 0 || s.total_q == 0) return FA_OK;
  if (positions)
    if (int r = check_ptr(positions, "positions", 4)) return r;
  if (q) {
    if (int r = check_rows(q, q_stride, s.Hq, "q")) return r;
    if (int r = check_rows(q_out, q_out_stride, s.Hq, "q_out")) return r;
    if (q == q_out && q_stride != q_out_stride && s.total_q > 1)
      return fail(FA_ERR_INVALID, "q_out is q, but the strides differ");
  }
  if (int r = check_rows(k, k_stride, s.Hkv, "k")) return r;
  if (int r = check_rows(v, v_stride, s.Hkv, "v")) return r;
  return launched(fa::launch_paged_append(s, *cache, rope, positions, q, q_stride, q_out,
                                          q_out_stride, k, k_stride, v, v_stride,
                                          static_cast<cudaStream_t>(stream)),
                  "fa_paged_append: launch");
}

size_t fa_paged_attend_workspace_size(const fa_paged_shape* shape, int32_t window) {
  float scale = 0.0f;
  size_t bytes = 0;
  if (check_shape(shape) || check_softmax(*shape, &scale, &window)) return 0;
  if (shape->B == 0 || shape->total_q == 0) return 0;
  if (launched(fa::paged_attend_workspace(*shape, window, &bytes), "fa_paged_attend: configure"))
    return 0;
  return bytes;
}

int fa_paged_attend(const fa_paged_shape* shape, const fa_paged_cache* cache, const void* q,
                    int64_t q_stride, float scale, int32_t window, void* out, int64_t out_stride,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (int r = check_cache(shape, cache, true, true)) return r;
  const fa_paged_shape& s = *shape;
  if (int r = check_softmax(s, &scale, &window)) return r;
  if (s.B == 0 || s.total_q == 0) return FA_OK;
  if (int r = check_rows(q, q_stride, s.Hq, "q")) return r;
  if (int r = check_rows(out, out_stride, s.Hq, "out")) return r;
  if (out == q) return fail(FA_ERR_INVALID, "out must not be q");
  if (lse)
    if (int r = check_ptr(lse, "lse", 4)) return r;
  size_t need = 0;
  if (int r = launched(fa::paged_attend_workspace(s, window, &need), "fa_paged_attend: configure"))
    return r;
  if (need > 0) {
    if (int r = check_ptr(workspace, "workspace")) return r;
    if (workspace_bytes < need)
      return fail(FA_ERR_INVALID, "workspace of %zu bytes is smaller than the %zu required",
                  workspace_bytes, need);
  }
  const char* why = nullptr;
  const cudaError_t e =
      fa::launch_paged_attend(s, *cache, q, q_stride, scale, window, out, out_stride, lse,
                              workspace, static_cast<cudaStream_t>(stream), &why);
  return launched(e, "fa_paged_attend: launch", why);
}

int fa_paged_weights(const fa_paged_shape* shape, const fa_paged_cache* cache, const void* q,
                     int64_t q_stride, float scale, int32_t window, const float* lse,
                     float* weights, int64_t weights_ld, void* stream) {
  if (int r = check_cache(shape, cache, true, false)) return r;
  const fa_paged_shape& s = *shape;
  if (int r = check_softmax(s, &scale, &window)) return r;
  if (weights_ld < s.max_kv)
    return fail(FA_ERR_INVALID, "weights_ld=%lld is below max_kv=%d", (long long)weights_ld, s.max_kv);
  if (s.B == 0 || s.total_q == 0 || s.max_kv == 0) return FA_OK;
  if (int r = check_rows(q, q_stride, s.Hq, "q")) return r;
  if (int r = check_ptr(lse, "lse", 4)) return r;
  if (int r = check_ptr(weights, "weights", 4)) return r;
  const char* why = nullptr;
  const cudaError_t e =
      fa::launch_paged_weights(s, *cache, q, q_stride, scale, window, lse, weights, weights_ld,
                               static_cast<cudaStream_t>(stream), &why);
  return launched(e, "fa_paged_weights: launch", why);
}

size_t fa_evict_workspace_size(const fa_paged_shape* shape, int32_t keep) {
  size_t bytes = 0;
  if (check_shape(shape)) return 0;
  if (keep < 1) {
    fail(FA_ERR_INVALID, "keep=%d must be at least 1", keep);
    return 0;
  }
  if (launched(fa::evict_workspace(*shape, keep, &bytes), "fa_evict: configure")) return 0;
  return bytes;
}

int fa_evict(const fa_paged_shape* shape, const fa_paged_cache* cache, const float* weights,
             int64_t weights_ld, int32_t keep, int32_t sink, int32_t recent,
             const fa_paged_shape* dst_shape, const fa_paged_cache* dst_cache, float* dst_weights,
             int64_t dst_weights_ld, int32_t* index, int32_t* dst_len, void* workspace,
             size_t workspace_bytes, void* stream) {
  if (int r = check_cache(shape, cache, false, true)) return r;
  if (int r = check_cache(dst_shape, dst_cache, false, true)) return r;
  const fa_paged_shape &s = *shape, &d = *dst_shape;
  if (d.B != s.B || d.Hkv != s.Hkv)
    return fail(FA_ERR_INVALID, "dst has B=%d Hkv=%d, the source %d %d", d.B, d.Hkv, s.B, s.Hkv);
  if (keep < 1 || sink < 0 || recent < 0 || (long long)sink + recent > keep)
    return fail(FA_ERR_INVALID, "need keep >= 1, sink, recent >= 0 and sink + recent <= keep "
                "(keep=%d sink=%d recent=%d)", keep, sink, recent);
  if (d.max_kv < keep)
    return fail(FA_ERR_INVALID, "dst max_kv=%d is below keep=%d", d.max_kv, keep);
  if (weights_ld < s.max_kv)
    return fail(FA_ERR_INVALID, "weights_ld=%lld is below max_kv=%d", (long long)weights_ld, s.max_kv);
  if (s.B == 0) return FA_OK;
  if (int r = check_ptr(cache->kv_len, "cache->kv_len", 4)) return r;
  if (s.max_kv > 0)
    if (int r = check_ptr(weights, "weights", 4)) return r;
  if (int r = check_ptr(index, "index", 4)) return r;
  if (int r = check_ptr(dst_len, "dst_len", 4)) return r;
  if (overlap(dst_len, 4 * (size_t)s.B, cache->kv_len, 4 * (size_t)s.B))
    return fail(FA_ERR_INVALID, "dst_len overlaps the source's kv_len");
  if (dst_weights) {
    if (int r = check_ptr(dst_weights, "dst_weights", 4)) return r;
    if (dst_weights_ld < keep)
      return fail(FA_ERR_INVALID, "dst_weights_ld=%lld is below keep=%d", (long long)dst_weights_ld, keep);
    const size_t rows = (size_t)s.B * s.Hkv;
    if (s.max_kv > 0 && overlap(dst_weights, 4 * rows * dst_weights_ld, weights, 4 * rows * weights_ld))
      return fail(FA_ERR_INVALID, "dst_weights overlaps weights");
  }
  size_t need = 0;
  if (int r = launched(fa::evict_workspace(s, keep, &need), "fa_evict: configure")) return r;
  if (need > 0) {
    if (int r = check_ptr(workspace, "workspace")) return r;
    if (workspace_bytes < need)
      return fail(FA_ERR_INVALID, "workspace of %zu bytes is smaller than the %zu required",
                  workspace_bytes, need);
  }
  return launched(fa::launch_evict(s, *cache, weights, weights_ld, keep, sink, recent, d, *dst_cache,
                                   dst_weights, dst_weights_ld, index, dst_len, workspace,
                                   static_cast<cudaStream_t>(stream)),
                  "fa_evict: launch");
}

}  // extern "C"
