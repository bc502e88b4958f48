// C ABI of the paged cache's operators (declared in include/gdn.h): argument
// validation, plan and launches.  No allocation, no host sync.
#include "../../include/gdn.h"
#include "gdn_checks.h"
#include "gdn_paged.h"

#include <limits.h>

namespace {

using gdn::aligned;
using gdn::align_up;
using gdn::all_aligned;
using gdn::all_given;
using gdn::overlaps;
using gdn::Range;

constexpr int64_t kMaxRows = (1 << 26) - 64;   // tokens by query heads of one call
constexpr int64_t kMaxItems = (1 << 24) - 1;   // workgroups of 256 threads of one launch
constexpr int64_t kMaxKeys = 1 << 30;

// Elements that rows of D at these strides span, in up to four directions; -1 where
// two rows share elements.
struct Step {
  int64_t n, stride;
};
template <int N> int64_t span(int64_t D, Step (&s)[N]) {
  for (int i = 1; i < N; ++i)
    for (int j = i; j > 0 && s[j].stride < s[j - 1].stride; --j) {
      const Step t = s[j];
      s[j] = s[j - 1];
      s[j - 1] = t;
    }
  int64_t ext = D;
  for (const Step& x : s) {
    if (x.n < 2) continue;
    if (x.stride < ext) return -1;
    ext += (x.n - 1) * x.stride;
  }
  return ext;
}

int64_t size_of(const gdn_paged_dims* p) { return p->dtype == GDN_BF16 ? 2 : 4; }

// bytes: the span of the pool's keys (or values).
int check_paged(const gdn_paged_dims* p, gdn::PagePool* pool, size_t* bytes) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->N < 0 || p->S < 1 || p->Hq < 0 || p->Hk < 1 || p->D < 1 || p->pages < 1 || p->page < 1 || p->width < 1)
    return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (p->D % 8 || p->D > 256) return GDN_ERR_UNSUPPORTED;
  if (p->page > 4096 || (p->page & (p->page - 1))) return GDN_ERR_UNSUPPORTED;
  if (p->N > INT_MAX / 2 || p->S > INT_MAX / 2 || p->Hq > INT_MAX / 1024 || p->Hk > INT_MAX / 1024 || p->pages > INT_MAX ||
      p->width > INT_MAX || static_cast<double>(p->S) * p->width > 4.0e18)
    return GDN_ERR_UNSUPPORTED;
  const int64_t e = size_of(p), unit = 16 / e;
  for (int64_t s : {p->page_stride, p->head_stride, p->token_stride})
    if (s < 0 || s % unit || s > (int64_t{1} << 40)) return GDN_ERR_INVALID_ARG;
  // (the pool's addresses are formed in 64 bits)
  if (static_cast<double>(p->pages) * p->page_stride + static_cast<double>(p->Hk) * p->head_stride > 1.0e18)
    return GDN_ERR_UNSUPPORTED;
  Step s[] = {{p->pages, p->page_stride}, {p->Hk, p->head_stride}, {p->page, p->token_stride}};
  const int64_t ext = span(p->D, s);
  if (ext < 0) return GDN_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(ext) * e;
  pool->ps = p->page_stride * e;
  pool->hs = p->head_stride * e;
  pool->ts = p->token_stride * e;
  pool->pages = static_cast<int>(p->pages);
  pool->shift = 0;
  while ((int64_t{1} << pool->shift) < p->page) ++pool->shift;
  return GDN_OK;
}

// Whether keys and values share no element.
bool apart(const gdn_paged_dims* p, const void* k, const void* v) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(k), b = reinterpret_cast<uintptr_t>(v);
  Step s[] = {{p->pages, p->page_stride}, {p->Hk, p->head_stride}, {p->page, p->token_stride},
              {2, static_cast<int64_t>((a < b ? b - a : a - b) / size_of(p))}};
  return span(p->D, s) >= 0;
}

// The bytes of N rows of n elements, `stride` elements apart.
size_t rows_bytes(int64_t N, int64_t stride, int64_t n, int64_t e) {
  return N ? static_cast<size_t>((N - 1) * stride + n) * e : 0;
}

int check_attn(const gdn_paged_dims* d, int64_t prefix, int64_t max_q, int64_t max_len, bool uniform, gdn::AttnArgs* a,
               size_t* pool_bytes, size_t* part, size_t* ml) {
  *a = gdn::AttnArgs{};
  const int rc = check_paged(d, &a->pool, pool_bytes);
  if (rc) return rc;
  if (d->Hq < 1 || d->Hq % d->Hk || prefix < 0 || max_len < 0) return GDN_ERR_INVALID_ARG;
  if (uniform) {
    if (d->N % d->S) return GDN_ERR_INVALID_ARG;
    max_q = d->N / d->S;
  }
  if (d->N > 0 && (max_q < 1 || max_q > d->N)) return GDN_ERR_INVALID_ARG;
  if (max_len > d->width * d->page) return GDN_ERR_INVALID_ARG;
  if (prefix > kMaxKeys || max_len > kMaxKeys || d->N * d->Hq > kMaxRows) return GDN_ERR_UNSUPPORTED;
  a->N = static_cast<int>(d->N);
  a->S = static_cast<int>(d->S);
  a->per = static_cast<int>(d->N / d->S);
  a->Hq = static_cast<int>(d->Hq);
  a->Hk = static_cast<int>(d->Hk);
  a->G = static_cast<int>(d->Hq / d->Hk);
  a->D = static_cast<int>(d->D);
  a->width = d->width;
  a->prefix = static_cast<int>(prefix);
  a->max_q = static_cast<int>(max_q);
  a->max_len = static_cast<int>(max_len);
  *part = *ml = 0;
  if (d->N == 0) return GDN_OK;
  gdn::attn_plan(a, d->dtype == GDN_BF16, part, ml);
  const int64_t prefix_items = gdn::prefix_items(*a), own_items = gdn::own_items(*a);
  const bool one_launch = a->p_rows == a->o_rows;
  if ((one_launch ? prefix_items + own_items : prefix_items > own_items ? prefix_items : own_items) > kMaxItems)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_paged_append(const gdn_paged_dims* d, const gdn_turn* t, const void* q, const void* k,
                     const void* v, const float* wq, const float* wk, const float* rope,
                     const uint8_t* axis, const int32_t* pos, const int32_t* table,
                     const int32_t* past, const int32_t* cu, void* oq, void* k_pages, void* v_pages,
                     void* stream) {
  gdn::AppendArgs a{};
  size_t pool = 0;
  const int rc = check_paged(d, &a.pool, &pool);
  if (rc) return rc;
  if (!t || t->R < 0 || t->P < 0 || t->A < 1 || t->R > d->D || !(t->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (t->R % 16 || t->A > 4 || t->P > INT_MAX) return GDN_ERR_UNSUPPORTED;
  if (t->first < -kMaxKeys || t->first > kMaxKeys) return GDN_ERR_UNSUPPORTED;
  const int64_t e = size_of(d), unit = 16 / e, N = d->N;
  const int64_t qs = t->q_stride ? t->q_stride : d->Hq * d->D, ks = t->k_stride ? t->k_stride : d->Hk * d->D;
  const int64_t vs = t->v_stride ? t->v_stride : d->Hk * d->D;
  if (qs < d->Hq * d->D || ks < d->Hk * d->D || vs < d->Hk * d->D || qs % unit || ks % unit || vs % unit || qs > INT_MAX ||
      ks > INT_MAX || vs > INT_MAX)
    return GDN_ERR_INVALID_ARG;
  const bool queries = d->Hq > 0;
  if (!queries && (q || oq || wq)) return GDN_ERR_INVALID_ARG;
  if (queries && (wq == nullptr) != (wk == nullptr)) return GDN_ERR_INVALID_ARG;
  if (!cu && N % d->S) return GDN_ERR_INVALID_ARG;
  if (t->R > 0 && !rope) return GDN_ERR_INVALID_ARG;
  if (!all_given(table, past)) return GDN_ERR_INVALID_ARG;
  if (N > 0 && (!all_given(k, v, k_pages, v_pages) || (queries && !all_given(q, oq)))) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, wq, wk, rope, oq, k_pages, v_pages)) return GDN_ERR_INVALID_ARG;
  const size_t w = static_cast<size_t>(d->D) * 4;
  const Range in[] = {{q, rows_bytes(N, qs, d->Hq * d->D, e)}, {k, rows_bytes(N, ks, d->Hk * d->D, e)},
                      {v, rows_bytes(N, vs, d->Hk * d->D, e)}, {wq, w}, {wk, w},
                      {rope, static_cast<size_t>(t->P) * t->R * 4}, {axis, static_cast<size_t>(t->R / 2)},
                      {pos, static_cast<size_t>(N) * t->A * 4}, {table, static_cast<size_t>(d->S) * d->width * 4},
                      {past, static_cast<size_t>(d->S) * 4}, {cu, static_cast<size_t>(d->S + 1) * 4}};
  const Range oqr{oq, rows_bytes(N, d->Hq * d->D, d->Hq * d->D, e)};
  const Range outk[] = {oqr, {k_pages, pool}}, outv[] = {oqr, {v_pages, pool}};
  if (overlaps(outk, in) || overlaps(outv, in)) return GDN_ERR_INVALID_ARG;
  if (N > 0 && !apart(d, k_pages, v_pages)) return GDN_ERR_INVALID_ARG;
  a.BT = N;
  a.S = static_cast<int>(d->S);
  a.per = static_cast<int>(N / d->S);
  a.Hq = static_cast<int>(d->Hq);
  a.Hk = static_cast<int>(d->Hk);
  a.D = static_cast<int>(d->D);
  a.R = static_cast<int>(t->R);
  a.P = static_cast<int>(t->P);
  a.A = t->A;
  a.qs = qs;
  a.ks = ks;
  a.vs = vs;
  a.interleaved = t->interleaved != 0;
  a.eps = t->eps;
  a.w_offset = t->w_offset;
  a.q = q;
  a.k = k;
  a.v = v;
  a.wq = wq;
  a.wk = wk;
  a.rope = rope;
  a.axis = axis;
  a.pos = pos;
  a.first = t->first;
  a.table = table;
  a.past = past;
  a.cu = cu;
  a.width = d->width;
  a.oq = oq;
  a.kp = k_pages;
  a.vp = v_pages;
  return gdn::launch_append(a, d->dtype == GDN_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_prefix_attention_workspace_bytes(const gdn_paged_dims* d, int64_t prefix, int64_t max_q,
                                         int64_t max_len, size_t* out) {
  gdn::AttnArgs a;
  size_t pool, part, ml;
  const int rc = check_attn(d, prefix, max_q, max_len, false, &a, &pool, &part, &ml);
  if (rc) return rc;
  if (!out) return GDN_ERR_INVALID_ARG;
  *out = align_up(part) + align_up(ml);
  return GDN_OK;
}

int gdn_prefix_attention(const gdn_paged_dims* d, const void* q, const void* k_pages,
                         const void* v_pages, const int32_t* table, const int32_t* lens,
                         const int32_t* prefix_pages, int64_t prefix, const int32_t* cu,
                         int64_t max_q, int64_t max_len, float scale, void* o, float* lse, void* ws,
                         size_t ws_bytes, void* stream) {
  gdn::AttnArgs a;
  size_t pool, part, ml;
  const int rc = check_attn(d, prefix, max_q, max_len, cu == nullptr, &a, &pool, &part, &ml);
  if (rc) return rc;
  if (!all_given(table, lens) || (prefix > 0 && !prefix_pages)) return GDN_ERR_INVALID_ARG;
  if (d->N > 0 && !all_given(q, k_pages, v_pages, o)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k_pages, v_pages, o)) return GDN_ERR_INVALID_ARG;
  const size_t need = align_up(part) + align_up(ml);
  if (need > ws_bytes || (need > 0 && !ws)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws)) return GDN_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(d->N) * d->Hq * d->D * size_of(d);
  const Range out[] = {{o, rows}, {lse, static_cast<size_t>(d->N) * d->Hq * 4}, {ws, need}};
  const Range in[] = {{q, rows}, {k_pages, pool}, {v_pages, pool}, {table, static_cast<size_t>(d->S) * d->width * 4},
                      {lens, static_cast<size_t>(d->S) * 4},
                      {prefix_pages, static_cast<size_t>((prefix + d->page - 1) / d->page) * 4},
                      {cu, static_cast<size_t>(d->S + 1) * 4}};
  if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.kp = k_pages;
  a.vp = v_pages;
  a.table = table;
  a.lens = lens;
  a.prefix_pages = prefix_pages;
  a.cu = cu;
  a.scale = scale * 1.4426950408889634f;  // the statistics are in base 2
  a.o = o;
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + align_up(part));
  return gdn::launch_attn(a, d->dtype == GDN_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
