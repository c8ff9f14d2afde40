// FiX decode over a paged cache: one new query per sequence against the
// pages of its keys, values and log forget gates.  With t = L - 1,
//   S_s = scale q.k_s,  m = max S,  D_s[c] = exp(sum_{r=s+1..t} g_r[c]),
//   o[c] = sum_s exp(S_s - m) D_s[c] v_s[c],
// followed by the norm (or division by l = sum_s exp(S_s - m)) and the output
// gate.  The cache is walked from the newest token back, so that the decay is
// a running suffix sum of the stored gates.
//
// First form: one CTA per (sequence, q head), 32 keys at a time, thread c on
// value channel c.  Bound by latency (one CTA walks a whole sequence).
#include "fix_internal.h"

#define FIX_PAGED_TRY(expr)           \
  do {                                \
    fix_status _s = (expr);           \
    if (_s != FIX_OK) return _s;      \
  } while (0)

namespace fix {

struct PagedArgs {
  int B, Hq, Hkv, Dk, Dv, grp, scalar, no_norm, y_f32;
  float scale, eps;
  int page_size, num_pages, max_pages;
  const int *table, *seqlens;
  const __nv_bfloat16 *q, *k, *v, *w, *z;
  const float* g;
  void* y;
  int* status;
};

constexpr int kPagedKeys = 32;

__global__ void __launch_bounds__(128) paged_decode_kernel(PagedArgs a) {
  __shared__ float sq[128], sp[kPagedKeys], red[4];
  __shared__ long long srow[kPagedKeys];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, kv = h / a.grp;
  const int c = threadIdx.x, lane = c & 31, warp = c >> 5;
  const long long cap = (long long)a.max_pages * a.page_size;
  long long L = a.seqlens[b] > 0 ? a.seqlens[b] : 0;
  if (L > cap) {
    L = cap;
    if (a.status && c == 0) *a.status = FIX_ERR_PAGE;
  }
  if (c < a.Dk) sq[c] = bf2f(a.q[((size_t)b * a.Hq + h) * a.Dk + c]) * a.scale;
  float m = -INFINITY, l = 0.f, o = 0.f, suf = 0.f;
  for (long long te = L; te > 0; te -= kPagedKeys) {
    const long long tb = te > kPagedKeys ? te - kPagedKeys : 0;
    const int nk = (int)(te - tb);
    __syncthreads();
    if (c < kPagedKeys) {
      long long row = -1;
      if (c < nk) {
        const long long s = tb + c;
        const int page = a.table[(long long)b * a.max_pages + s / a.page_size];
        if (page >= 0 && page < a.num_pages)
          row = ((long long)page * a.page_size + s % a.page_size) * a.Hkv + kv;
        else if (a.status)
          *a.status = FIX_ERR_PAGE;
      }
      srow[c] = row;
    }
    __syncthreads();
    for (int s = warp; s < kPagedKeys; s += 4) {
      float x = -INFINITY;
      if (srow[s] >= 0) {
        x = 0.f;
        for (int e = lane; e < a.Dk; e += 32) x += sq[e] * bf2f(a.k[srow[s] * a.Dk + e]);
        x = warp_sum(x);
      }
      if (lane == 0) sp[s] = x;
    }
    __syncthreads();
    float mt = m;
    for (int s = 0; s < nk; ++s) mt = fmaxf(mt, sp[s]);
    const float mu = mt == -INFINITY ? 0.f : mt;
    const float alpha = __expf(m - mu);
    o *= alpha;
    l *= alpha;
    m = mt;
    for (int s = nk - 1; s >= 0; --s) {
      if (srow[s] < 0) continue;
      const float p = __expf(sp[s] - mu);
      l += p;
      if (c < a.Dv) {
        o += p * __expf(suf) * bf2f(a.v[srow[s] * a.Dv + c]);
        suf += a.scalar ? a.g[srow[s]] : a.g[srow[s] * a.Dv + c];
      }
    }
  }
  float sq2 = c < a.Dv ? o * o : 0.f;
  sq2 = warp_sum(sq2);
  if (lane == 0) red[warp] = sq2;
  __syncthreads();
  const float tot = red[0] + red[1] + red[2] + red[3];
  if (c >= a.Dv) return;
  float y = a.no_norm ? o / l : o / sqrtf(tot / (float)a.Dv + a.eps) * bf2f(a.w[c]);
  if (m == -INFINITY) y = 0.f;
  const size_t at = ((size_t)b * a.Hq + h) * a.Dv + c;
  if (a.z) y *= swish(bf2f(a.z[at]));
  if (a.y_f32) reinterpret_cast<float*>(a.y)[at] = y;
  else reinterpret_cast<__nv_bfloat16*>(a.y)[at] = f2bf(y);
}

static fix_status paged_dims(const fix_attn_problem* p, const fix_attn_page_cache* c, Dims* d) {
  FIX_PAGED_TRY(validate_problem(p, d));
  if (p->cu_seqlens || p->num_seqs) return FIX_ERR_CU_SEQLENS;   // lengths come with the cache
  if (p->seqlen != 1) return FIX_ERR_SHAPE;
  return validate_cache(c, *d);
}

}  // namespace fix

using namespace fix;

extern "C" size_t fix_attn_decode_paged_workspace_bytes(const fix_attn_problem* p,
                                                        const fix_attn_page_cache* c) {
  Dims d;
  if (paged_dims(p, c, &d) != FIX_OK) return 0;
  return 256;
}

extern "C" fix_status fix_attn_decode_paged(const fix_attn_problem* p, const fix_attn_page_cache* c,
                                            const void* q, const void* o_norm_weight,
                                            const void* o_gate, void* y, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  Dims d;
  FIX_PAGED_TRY(paged_dims(p, c, &d));
  if (!q || (!o_norm_weight && !d.no_norm) || !y || !workspace) return FIX_ERR_NULL;
  for (const void* x : {q, o_norm_weight, o_gate, (const void*)y, (const void*)workspace})
    if (reinterpret_cast<uintptr_t>(x) & 15u) return FIX_ERR_ALIGN;
  if (workspace_bytes < 256) return FIX_ERR_WORKSPACE;
  FIX_PAGED_TRY(check_device());
  PagedArgs a{};
  a.B = d.B; a.Hq = d.Hq; a.Hkv = d.Hkv; a.Dk = d.Dk; a.Dv = d.Dv; a.grp = d.grp;
  a.scalar = d.scalar_gate; a.no_norm = d.no_norm; a.y_f32 = p->y_dtype == FIX_DTYPE_F32;
  a.scale = d.scale; a.eps = d.eps;
  a.page_size = c->page_size; a.num_pages = c->num_pages; a.max_pages = c->max_pages;
  a.table = c->page_table; a.seqlens = c->seqlens;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(c->k_pages);
  a.v = static_cast<const __nv_bfloat16*>(c->v_pages);
  a.g = c->g_pages;
  a.w = static_cast<const __nv_bfloat16*>(o_norm_weight);
  a.z = static_cast<const __nv_bfloat16*>(o_gate);
  a.y = y;
  a.status = c->status;
  paged_decode_kernel<<<d.B * d.Hq, 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launch_status();
}
