// extern "C" entry points around the prompt pass: argument validation and
// launches of the rotary-position, paging and 4-bit-cache kernels on the
// caller's stream.  See include/sparge.h.
#include <cstdint>

#include "sparge_internal.h"

using namespace sparge;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// (the failed call's error is reported here, not by the next call that asks for the last)
sparge_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return SPARGE_OK;
  cudaGetLastError();
  if (e == cudaErrorNotSupported) return SPARGE_EUNSUPPORTED;
  return SPARGE_ECUDA;
}

bool is_dtype(sparge_dtype_t t) { return t == SPARGE_F16 || t == SPARGE_BF16 || t == SPARGE_F32; }
int64_t elem_size(sparge_dtype_t t) { return t == SPARGE_F32 ? 4 : 2; }

// Rows of `row` bytes at every index of ext[n] with strides in bytes.
struct Rows {
  int64_t ext[3], stride[3];
  int64_t row;
};

// Bytes from the first to one past the last; -1 when it does not fit 62 bits.
int64_t extent(const Rows& r) {
  int64_t sum = r.row;
  for (int i = 0; i < 3; ++i) {
    const int64_t n = r.ext[i] - 1;
    if (n > 0 && r.stride[i] > (int64_t(1) << 61) / n) return -1;
    sum += n * r.stride[i];
    if (sum > (int64_t(1) << 61)) return -1;
  }
  return sum;
}

// Whether each stride, in ascending order, steps over what the smaller span.
bool disjoint(Rows r) {
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j + 1 < 3; ++j)
      if (r.stride[j] > r.stride[j + 1]) {
        const int64_t s = r.stride[j], e = r.ext[j];
        r.stride[j] = r.stride[j + 1], r.ext[j] = r.ext[j + 1];
        r.stride[j + 1] = s, r.ext[j + 1] = e;
      }
  int64_t span = r.row;
  for (int i = 0; i < 3; ++i) {
    if (r.ext[i] <= 1) continue;
    if (r.stride[i] < span) return false;
    span += (r.ext[i] - 1) * r.stride[i];
  }
  return true;
}

// SPARGE_OK, SPARGE_EINVAL or SPARGE_EUNSUPPORTED for a cache's shape.
sparge_status_t check_kv4(const sparge_kv4_t* c) {
  if (c == nullptr || c->Hkv < 1 || c->d < 1 || c->group < 1 || c->page_size < 1 ||
      c->num_pages < 0)
    return SPARGE_EINVAL;
  if (c->page_size % 16 != 0) return SPARGE_EINVAL;
  if (c->d != 64 && c->d != 128) return SPARGE_EUNSUPPORTED;
  if (c->group != 32 && c->group != 64 && c->group != 128) return SPARGE_EUNSUPPORTED;
  if (c->group > c->d) return SPARGE_EINVAL;
  if (c->Hkv > 65535 || int64_t(c->num_pages) * c->page_size > INT32_MAX ||
      int64_t(c->num_pages) * c->page_size / 16 * c->Hkv > INT32_MAX)
    return SPARGE_EUNSUPPORTED;
  return SPARGE_OK;
}

// Token and head strides of a [T, Hkv, d] tensor, in bytes.
sparge_status_t row_strides(const int64_t* st, int64_t T, int64_t H, int64_t row, int64_t es,
                            Rows* r) {
  *r = Rows{{T, H, 1}, {0, 0, 0}, row};
  if (st == nullptr) return SPARGE_EINVAL;
  for (int i = 0; i < 2; ++i) {
    if (r->ext[i] <= 1) continue;
    if (st[i] < 0 || st[i] > (int64_t(1) << 58)) return SPARGE_EINVAL;
    r->stride[i] = st[i] * es;
    if (r->stride[i] % 16 != 0) return SPARGE_EUNSUPPORTED;
  }
  return extent(*r) < 0 ? SPARGE_EINVAL : SPARGE_OK;
}

sparge_status_t check_attn(const sparge_kv4_t* c, const sparge_kv4_attn_t* a) {
  const sparge_status_t st = check_kv4(c);
  if (st != SPARGE_OK) return st;
  if (a == nullptr || a->R < 0 || a->T < 0 || a->Hq < 1 || a->Hq % c->Hkv != 0 || a->max_q < 0 ||
      a->max_pages < 0 || a->max_len < 0 || (a->causal != 0 && a->causal != 1) ||
      !(a->scale > 0.f) || !(a->scale <= 0x1p100f) ||
      (a->dtype != SPARGE_F16 && a->dtype != SPARGE_BF16))
    return SPARGE_EINVAL;
  if (a->T > 1 && (a->q_stride < int64_t(a->Hq) * c->d || a->q_stride > (int64_t(1) << 58) / a->T))
    return SPARGE_EINVAL;
  if (a->T > 1 && a->q_stride % 8 != 0) return SPARGE_EUNSUPPORTED;
  if (a->R > 65535 || int64_t(a->T) * a->Hq > INT32_MAX ||
      int64_t(a->max_q) * a->Hq > INT32_MAX ||
      int64_t(a->max_pages) * c->page_size > INT32_MAX - 64)
    return SPARGE_EUNSUPPORTED;
  return SPARGE_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

}  // namespace

extern "C" {

static sparge_status_t rope_common(const sparge_rope_t* p, const void* src, void* dst,
                                   const int32_t* pos, const double* inv_freq,
                                   const int32_t* axis, const int32_t* perm, bool inverse,
                                   cudaStream_t stream) {
  if (p == nullptr) return SPARGE_EINVAL;
  if (p->B < 0 || p->H < 0 || p->N < 0 || p->d < 1 || p->axes < 1) return SPARGE_EINVAL;
  if (p->rot < 2 || p->rot > p->d || p->rot % 2 != 0) return SPARGE_EINVAL;
  if ((p->interleaved != 0 && p->interleaved != 1) || !is_dtype(p->dtype)) return SPARGE_EINVAL;
  if (p->pos_stride < 0 || p->pos_stride > (int64_t(1) << 40)) return SPARGE_EINVAL;
  const int64_t es = elem_size(p->dtype);
  if (p->d * es % 16 != 0 || p->rot * es % 32 != 0) return SPARGE_EUNSUPPORTED;
  Rows r[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t* st = (i == 0) != inverse ? p->x_stride : p->y_stride;  // r[0]: the source
    r[i] = Rows{{p->B, p->H, p->N}, {0, 0, 0}, p->d * es};
    for (int k = 0; k < 3; ++k) {
      if (r[i].ext[k] <= 1) continue;
      if (st[k] < 0 || st[k] > (int64_t(1) << 58)) return SPARGE_EINVAL;
      r[i].stride[k] = st[k] * es;
      if (r[i].stride[k] % 16 != 0) return SPARGE_EUNSUPPORTED;
    }
  }
  if (p->B == 0 || p->H == 0 || p->N == 0) return SPARGE_OK;
  if (int64_t(p->B) * p->H > INT32_MAX) return SPARGE_EUNSUPPORTED;
  if (src == nullptr || dst == nullptr || pos == nullptr || inv_freq == nullptr || axis == nullptr)
    return SPARGE_EINVAL;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(pos, 4) || !aligned(inv_freq, 8) ||
      !aligned(axis, 4) || !aligned(perm, 4))
    return SPARGE_EINVAL;
  const int64_t ns = extent(r[0]), nd = extent(r[1]);
  if (ns < 0 || nd < 0 || !disjoint(r[1])) return SPARGE_EINVAL;
  bool same = src == dst && perm == nullptr;
  for (int k = 0; k < 3; ++k) same = same && r[0].stride[k] == r[1].stride[k];
  if (!same && overlap(src, ns, dst, nd)) return SPARGE_EINVAL;
  DeviceScope dev;
  const sparge_status_t st = dev.enter(dst);
  if (st != SPARGE_OK) return st;
  int64_t ss[3], ds[3];
  for (int k = 0; k < 3; ++k) ss[k] = r[0].stride[k], ds[k] = r[1].stride[k];
  return from_cuda(
      launch_rope(*p, src, ss, dst, ds, pos, inv_freq, axis, perm, inverse, stream));
}

sparge_status_t sparge_rope_apply(const sparge_rope_t* p, const void* x, void* y,
                                  const int32_t* pos, const double* inv_freq,
                                  const int32_t* axis, const int32_t* perm, cudaStream_t stream) {
  return rope_common(p, x, y, pos, inv_freq, axis, perm, false, stream);
}

sparge_status_t sparge_rope_inverse(const sparge_rope_t* p, const void* y, void* x,
                                    const int32_t* pos, const double* inv_freq,
                                    const int32_t* axis, const int32_t* perm,
                                    cudaStream_t stream) {
  return rope_common(p, y, x, pos, inv_freq, axis, perm, true, stream);
}

sparge_status_t sparge_kv_plan(int32_t R, int32_t page_size, int32_t max_pages,
                               int32_t num_pages, int32_t max_tokens, const int32_t* new_len,
                               const int32_t* seq_len, int32_t* block_table,
                               int32_t* free_pages, const int32_t* free_count,
                               int32_t* seq_len_out, int32_t* free_count_out, int32_t* cu_new,
                               int32_t* slot_map, int32_t* admitted, cudaStream_t stream) {
  if (R < 0 || page_size < 1 || max_pages < 0 || num_pages < 0 || max_tokens < 0)
    return SPARGE_EINVAL;
  if (R > kMaxPlanRequests || int64_t(num_pages) * page_size > INT32_MAX ||
      int64_t(max_pages) * page_size > INT32_MAX || max_tokens > kMaxPlanTokens)
    return SPARGE_EUNSUPPORTED;
  // what has no elements may be NULL
  if (free_count == nullptr || free_count_out == nullptr || cu_new == nullptr) return SPARGE_EINVAL;
  if (R > 0 && (new_len == nullptr || seq_len == nullptr || seq_len_out == nullptr ||
                admitted == nullptr || (max_pages > 0 && block_table == nullptr)))
    return SPARGE_EINVAL;
  if ((num_pages > 0 && free_pages == nullptr) || (max_tokens > 0 && slot_map == nullptr))
    return SPARGE_EINVAL;
  const void* all[] = {new_len, seq_len, block_table, free_pages, free_count, seq_len_out,
                       free_count_out, cu_new, slot_map, admitted};
  for (const void* x : all)
    if (!aligned(x, 4)) return SPARGE_EINVAL;
  // what is written, apart from the two that may be their own inputs, meets nothing else
  const int64_t r4 = 4 * int64_t(R);
  const int64_t bytes[] = {r4, r4, r4 * max_pages, 4 * int64_t(num_pages), 4, r4, 4, r4 + 4,
                           4 * int64_t(max_tokens), r4};
  for (int i = 2; i < 10; ++i) {
    if (i == 4) continue;
    for (int j = 0; j < 10; ++j) {
      if (j == i || bytes[i] == 0 || bytes[j] == 0) continue;
      if (((i == 5 && j == 1) || (i == 6 && j == 4) || (i == 1 && j == 5) || (i == 4 && j == 6)) &&
          all[i] == all[j])
        continue;
      if (overlap(all[i], bytes[i], all[j], bytes[j])) return SPARGE_EINVAL;
    }
  }
  DeviceScope dev;
  const sparge_status_t st = dev.enter(cu_new);
  if (st != SPARGE_OK) return st;
  const KvPlanArgs a{R, page_size, max_pages, num_pages, max_tokens, new_len, seq_len,
                     block_table, free_pages, free_count, seq_len_out, free_count_out, cu_new,
                     slot_map, admitted};
  return from_cuda(launch_kv_plan(a, stream));
}

size_t sparge_kv4_bytes(const sparge_kv4_t* c) {
  if (check_kv4(c) != SPARGE_OK) return 0;
  return size_t(c->num_pages) * c->Hkv * c->page_size * (c->d + 4 * (c->d / c->group));
}

static sparge_status_t cache_common(bool read, const sparge_kv4_t* c, int32_t T, void* k,
                                    const int64_t* k_stride, void* v, const int64_t* v_stride,
                                    sparge_dtype_t dtype, const int32_t* slot_map, void* cache,
                                    int32_t* status, cudaStream_t stream) {
  sparge_status_t st = check_kv4(c);
  if (st != SPARGE_OK) return st;
  if (T < 0 || !is_dtype(dtype)) return SPARGE_EINVAL;
  if (!read && dtype == SPARGE_F32) return SPARGE_EUNSUPPORTED;
  if (T == 0 || c->num_pages == 0) return SPARGE_OK;
  if (slot_map == nullptr || cache == nullptr || !aligned(slot_map, 4) || !aligned(cache, 16) ||
      !aligned(status, 4) || !aligned(k, 16) || !aligned(v, 16))
    return SPARGE_EINVAL;
  if (!read && (k == nullptr || v == nullptr)) return SPARGE_EINVAL;
  if (k == nullptr && v == nullptr) return SPARGE_OK;
  const int64_t es = elem_size(dtype), row = c->d * es;
  const int64_t cache_bytes = int64_t(sparge_kv4_bytes(c));
  Rows r[2];
  void* const p[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    r[i] = Rows{{T, c->Hkv, 1}, {0, 0, 0}, row};
    if (p[i] == nullptr) continue;
    if ((st = row_strides(i == 0 ? k_stride : v_stride, T, c->Hkv, row, es, &r[i])) != SPARGE_OK)
      return st;
    if (overlap(p[i], extent(r[i]), cache, cache_bytes)) return SPARGE_EINVAL;
    if (read && (!disjoint(r[i]) || overlap(p[i], extent(r[i]), slot_map, 4 * int64_t(T))))
      return SPARGE_EINVAL;
  }
  if (!read && overlap(slot_map, 4 * int64_t(T), cache, cache_bytes)) return SPARGE_EINVAL;
  DeviceScope dev;
  if ((st = dev.enter(cache)) != SPARGE_OK) return st;
  return from_cuda(launch_kv4_cache(*c, read, T, k, r[0].stride, v, r[1].stride, dtype, slot_map,
                                    cache, status, stream));
}

sparge_status_t sparge_kv4_append(const sparge_kv4_t* c, int32_t T, const void* k,
                                  const int64_t k_stride[2], const void* v,
                                  const int64_t v_stride[2], sparge_dtype_t dtype,
                                  const int32_t* slot_map, void* cache, int32_t* status,
                                  cudaStream_t stream) {
  return cache_common(false, c, T, const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride,
                      dtype, slot_map, cache, status, stream);
}

sparge_status_t sparge_kv4_read(const sparge_kv4_t* c, int32_t T, const void* cache,
                                const int32_t* slot_map, void* k, const int64_t k_stride[2],
                                void* v, const int64_t v_stride[2], sparge_dtype_t dtype,
                                cudaStream_t stream) {
  return cache_common(true, c, T, k, k_stride, v, v_stride, dtype, slot_map,
                      const_cast<void*>(cache), nullptr, stream);
}

size_t sparge_kv4_workspace_bytes(const sparge_kv4_t* c, const sparge_kv4_attn_t* a) {
  if (check_attn(c, a) != SPARGE_OK) return 0;
  return kv4_attn_ws_bytes(*c, *a);
}

sparge_status_t sparge_kv4_attn(const sparge_kv4_t* c, const sparge_kv4_attn_t* a,
                                const void* q, const void* cache, const int32_t* block_table,
                                const int32_t* seq_len, const int32_t* cu_q, void* o,
                                float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  sparge_status_t st = check_attn(c, a);
  if (st != SPARGE_OK) return st;
  if (a->R == 0 || a->T == 0 || a->max_q == 0) return SPARGE_OK;
  if (q == nullptr || seq_len == nullptr || cu_q == nullptr || o == nullptr || ws == nullptr)
    return SPARGE_EINVAL;
  if ((a->max_pages > 0 && block_table == nullptr) || (c->num_pages > 0 && cache == nullptr))
    return SPARGE_EINVAL;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(o, 16) || !aligned(ws, 256) ||
      !aligned(block_table, 4) || !aligned(seq_len, 4) || !aligned(cu_q, 4) || !aligned(lse, 4))
    return SPARGE_EINVAL;
  if (ws_bytes < kv4_attn_ws_bytes(*c, *a)) return SPARGE_EWORKSPACE;
  // o, lse and ws are written: they meet nothing else
  const int64_t rows = int64_t(a->T) * a->Hq;
  const void* p[] = {o, lse, ws, q, cache, block_table, seq_len, cu_q};
  const int64_t n[] = {rows * c->d * 2, lse != nullptr ? rows * 4 : 0,
                       int64_t(kv4_attn_ws_bytes(*c, *a)),
                       ((a->T - 1) * a->q_stride + int64_t(a->Hq) * c->d) * 2,
                       int64_t(sparge_kv4_bytes(c)), 4 * int64_t(a->R) * a->max_pages,
                       4 * int64_t(a->R), 4 * int64_t(a->R) + 4};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (n[i] > 0 && n[j] > 0 && overlap(p[i], n[i], p[j], n[j])) return SPARGE_EINVAL;
  DeviceScope dev;
  if ((st = dev.enter(q)) != SPARGE_OK) return st;
  return from_cuda(launch_kv4_attn(*c, *a, q, cache, block_table, seq_len, cu_q, o, lse, ws, stream));
}

}  // extern "C"
