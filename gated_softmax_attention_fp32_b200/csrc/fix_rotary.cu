// Rotation of q and k by position, alone (fix_attn_rotary) or while new
// tokens are appended to a paged cache (fix_attn_append_paged).
//
// A pair (a, b) at position p turns by t = p f:  a' = a cos t - b sin t,
// b' = a sin t + b cos t.  p f is formed in double and loses its whole turns
// there, so that positions of any size keep an angle error near 1e-7; the
// products and sums are float, rounded to bf16 once.
//
// Memory bound: a token's heads are read once and written once.  One CTA per
// token computes the token's rot_dim/2 sines and cosines into shared memory
// once, for all its heads; a thread then moves 16 channels of a head (two
// 16-byte loads and stores): the 8 + 8 channels that eight pairs span.
#include "fix_internal.h"

#define FIX_ROT_TRY(expr)             \
  do {                                \
    fix_status _s = (expr);           \
    if (_s != FIX_OK) return _s;      \
  } while (0)

namespace fix {

constexpr int kTokThreads = 128;

struct TokenArgs {
  long long N;                    // tokens
  int T;                          // tokens per sequence when not packed
  int nseq;
  const int64_t* cu;              // packed lengths or NULL
  const int* positions;           // given positions or NULL
  const int* seqlens;             // append: lengths in the cache, else NULL
  int Hq, Hkv, Dk, Dv, scalar;
  int rot, interleaved, inverse;  // rot = 0: nothing is rotated
  const float* inv_freq;
  const __nv_bfloat16 *q, *k, *v;
  const float* g;
  long long qs, ks, vs, gs;       // elements between tokens
  __nv_bfloat16 *q_out, *k_out;
  // paged cache (append only)
  const int* table;
  int page_size, num_pages, max_pages;
  __nv_bfloat16 *k_pages, *v_pages;
  float* g_pages;
  int* status;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Sequence b of token n and its index in it; false behind the last sequence.
__device__ __forceinline__ bool find_seq(const TokenArgs& a, long long n, int* b, long long* t,
                                         long long* len) {
  if (!a.cu) {
    *b = (int)(n / a.T);
    *t = n - (long long)*b * a.T;
    *len = a.T;
    return true;
  }
  int lo = 0, hi = a.nseq;            // the first b with cu[b + 1] > n
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid + 1] > n) hi = mid; else lo = mid + 1;
  }
  if (lo >= a.nseq) return false;
  *b = lo;
  *t = n - a.cu[lo];
  *len = a.cu[lo + 1] - a.cu[lo];
  return *t >= 0;
}

// Rotates (or, with cs == NULL, copies) the 16 channels of unit u of one head
// row and stores them to dst and, where given, dst2.
__device__ __forceinline__ void rotate_unit(const TokenArgs& a, const float2* cs, int u,
                                            const __nv_bfloat16* src, __nv_bfloat16* dst,
                                            __nv_bfloat16* dst2) {
  const bool turn = u * 16 < a.rot;
  const int e0 = (turn && !a.interleaved) ? 8 * u : 16 * u;
  const int e1 = (turn && !a.interleaved) ? a.rot / 2 + 8 * u : 16 * u + 8;
  uint4 x = *reinterpret_cast<const uint4*>(src + e0);
  uint4 y = *reinterpret_cast<const uint4*>(src + e1);
  if (turn && cs) {
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
    const float2* f = cs + 8 * u;
    if (!a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c0 = f[2 * i], c1 = f[2 * i + 1];
        const float a0 = lo_f(xw[i]), a1 = hi_f(xw[i]), b0 = lo_f(yw[i]), b1 = hi_f(yw[i]);
        xw[i] = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
        yw[i] = pack_bf16(a0 * c0.y + b0 * c0.x, a1 * c1.y + b1 * c1.x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c0 = f[i], c1 = f[4 + i];
        const float a0 = lo_f(xw[i]), b0 = hi_f(xw[i]), a1 = lo_f(yw[i]), b1 = hi_f(yw[i]);
        xw[i] = pack_bf16(a0 * c0.x - b0 * c0.y, a0 * c0.y + b0 * c0.x);
        yw[i] = pack_bf16(a1 * c1.x - b1 * c1.y, a1 * c1.y + b1 * c1.x);
      }
    }
  }
  if (dst) {
    *reinterpret_cast<uint4*>(dst + e0) = x;
    *reinterpret_cast<uint4*>(dst + e1) = y;
  }
  if (dst2) {
    *reinterpret_cast<uint4*>(dst2 + e0) = x;
    *reinterpret_cast<uint4*>(dst2 + e1) = y;
  }
}

// grid N, block kTokThreads
__global__ void __launch_bounds__(kTokThreads) token_kernel(TokenArgs a) {
  __shared__ float2 cs[64];
  __shared__ long long s_pos, s_row;
  const int tid = threadIdx.x;
  const long long n = blockIdx.x;
  if (tid == 0) {
    int b = 0;
    long long t = 0, len = 0, pos = -1, row = -1;
    if (a.positions) {
      pos = a.positions[n];
    } else if (find_seq(a, n, &b, &t, &len)) {
      pos = a.seqlens ? (long long)a.seqlens[b] - len + t : t;
      if (a.seqlens && pos >= 0) {
        const long long col = pos / a.page_size;
        int page = -1;
        if (col < a.max_pages) page = a.table[(long long)b * a.max_pages + col];
        if (page >= 0 && page < a.num_pages)
          row = (long long)page * a.page_size + pos % a.page_size;
        else if (a.status)
          *a.status = FIX_ERR_PAGE;
      }
    }
    s_pos = pos;
    s_row = row;
  }
  __syncthreads();
  const long long pos = s_pos, row = s_row;
  const bool turn = a.rot && (pos >= 0 || a.positions);
  if (turn && tid < a.rot / 2) {
    // the angle less its whole turns, 2 pi in two doubles
    const double t = (double)pos * (double)a.inv_freq[tid];
    const double turns = rint(t * 0.15915494309189534);
    const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, t));
    float s, c;
    sincosf((float)r, &s, &c);
    cs[tid] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  const float2* f = turn ? cs : nullptr;
  const int uk = a.Dk / 16;
  if (a.q_out)
    for (int i = tid; i < a.Hq * uk; i += kTokThreads) {
      const int h = i / uk, u = i % uk;
      rotate_unit(a, f, u, a.q + n * a.qs + h * a.Dk, a.q_out + (n * a.Hq + h) * a.Dk, nullptr);
    }
  if (a.k && (a.k_out || row >= 0))
    for (int i = tid; i < a.Hkv * uk; i += kTokThreads) {
      const int h = i / uk, u = i % uk;
      rotate_unit(a, f, u, a.k + n * a.ks + h * a.Dk,
                  a.k_out ? a.k_out + (n * a.Hkv + h) * a.Dk : nullptr,
                  row >= 0 ? a.k_pages + (row * a.Hkv + h) * a.Dk : nullptr);
    }
  if (row < 0) return;
  const int nv = a.Hkv * a.Dv;
  for (int i = tid * 8; i < nv; i += kTokThreads * 8)
    *reinterpret_cast<uint4*>(a.v_pages + row * nv + i) =
        *reinterpret_cast<const uint4*>(a.v + n * a.vs + i);
  if (a.scalar) {
    for (int i = tid; i < a.Hkv; i += kTokThreads) a.g_pages[row * a.Hkv + i] = a.g[n * a.gs + i];
  } else {
    for (int i = tid * 4; i < nv; i += kTokThreads * 4)
      *reinterpret_cast<float4*>(a.g_pages + row * nv + i) =
          *reinterpret_cast<const float4*>(a.g + n * a.gs + i);
  }
}

static bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A token stride in elements: 0 selects the dense one.
static fix_status token_stride(int64_t given, long long dense, int multiple, long long* out) {
  if (given == 0) given = dense;
  if (given < dense || given % multiple || given > (1LL << 40)) return FIX_ERR_SHAPE;
  *out = given;
  return FIX_OK;
}

// Dims of a problem whose packed lengths are read on the device only.
static fix_status token_dims(const fix_attn_problem* p, Dims* d) {
  if (!p) return FIX_ERR_NULL;
  fix_attn_problem dense = *p;
  dense.cu_seqlens = nullptr;
  dense.cu_seqlens_host = nullptr;
  dense.num_seqs = 0;
  FIX_ROT_TRY(validate_problem(&dense, d));
  if (!p->cu_seqlens) return p->num_seqs || p->cu_seqlens_host ? FIX_ERR_CU_SEQLENS : FIX_OK;
  if (p->batch != 1) return FIX_ERR_SHAPE;
  if (p->num_seqs < 1) return FIX_ERR_CU_SEQLENS;
  d->nseq = p->num_seqs;
  return FIX_OK;
}

static fix_status check_rotation(const fix_attn_rotation* r, const Dims& d) {
  if (!r->inv_freq) return FIX_ERR_NULL;
  if (misaligned(r->inv_freq)) return FIX_ERR_ALIGN;
  if (r->rot_dim < 16 || r->rot_dim > d.Dk || r->rot_dim % 16) return FIX_ERR_SHAPE;
  return FIX_OK;
}

fix_status validate_cache(const fix_attn_page_cache* c, const Dims& d) {
  if (!c) return FIX_ERR_NULL;
  if (c->page_size < 1 || c->num_pages < 1 || c->max_pages < 1) return FIX_ERR_SHAPE;
  if ((unsigned long long)c->num_pages * c->page_size >= (1ULL << 32) / d.Hkv) return FIX_ERR_SHAPE;
  if (!c->page_table || !c->seqlens || !c->k_pages || !c->v_pages || !c->g_pages) return FIX_ERR_NULL;
  for (const void* x : {(const void*)c->page_table, (const void*)c->seqlens, (const void*)c->k_pages,
                        (const void*)c->v_pages, (const void*)c->g_pages})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(c->status) & 3u) return FIX_ERR_ALIGN;
  return FIX_OK;
}

static fix_status launch_tokens(const TokenArgs& a, cudaStream_t st) {
  FIX_ROT_TRY(check_device());
  token_kernel<<<(unsigned)a.N, kTokThreads, 0, st>>>(a);
  return launch_status();
}

}  // namespace fix

using namespace fix;

extern "C" fix_status fix_attn_rotary(const fix_attn_problem* p, const fix_attn_rotation* r,
                                      const int32_t* positions, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, void* q_out, void* k_out,
                                      int inverse, void* stream) {
  Dims d;
  FIX_ROT_TRY(token_dims(p, &d));
  if (d.N == 0) return FIX_OK;
  if (!r || !q || !q_out || (!k) != (!k_out)) return FIX_ERR_NULL;
  FIX_ROT_TRY(check_rotation(r, d));
  for (const void* x : {q, k, (const void*)q_out, (const void*)k_out, (const void*)p->cu_seqlens})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return FIX_ERR_ALIGN;
  TokenArgs a{};
  FIX_ROT_TRY(token_stride(q_stride, (long long)d.Hq * d.Dk, 8, &a.qs));
  FIX_ROT_TRY(token_stride(k_stride, (long long)d.Hkv * d.Dk, 8, &a.ks));
  a.N = d.N; a.T = d.T; a.nseq = d.nseq; a.cu = p->cu_seqlens;
  a.positions = positions;
  a.Hq = d.Hq; a.Hkv = d.Hkv; a.Dk = d.Dk; a.Dv = d.Dv; a.scalar = d.scalar_gate;
  a.rot = r->rot_dim; a.interleaved = r->interleaved; a.inverse = inverse;
  a.inv_freq = r->inv_freq;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  return launch_tokens(a, static_cast<cudaStream_t>(stream));
}

extern "C" fix_status fix_attn_append_paged(const fix_attn_problem* p, const fix_attn_page_cache* c,
                                            const fix_attn_rotation* r, const void* q,
                                            int64_t q_stride, const void* k, int64_t k_stride,
                                            const void* v, int64_t v_stride, const float* g,
                                            int64_t g_stride, void* q_out, void* k_out,
                                            void* stream) {
  Dims d;
  FIX_ROT_TRY(token_dims(p, &d));
  if (d.N == 0) return FIX_OK;
  FIX_ROT_TRY(validate_cache(c, d));
  if (!k || !v || !g || (!q) != (!q_out) || (!r && (q || k_out))) return FIX_ERR_NULL;
  if (r) FIX_ROT_TRY(check_rotation(r, d));
  for (const void* x : {q, k, v, (const void*)q_out, (const void*)k_out, (const void*)p->cu_seqlens})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(g) & (d.scalar_gate ? 3u : 15u)) return FIX_ERR_ALIGN;
  TokenArgs a{};
  FIX_ROT_TRY(token_stride(q_stride, (long long)d.Hq * d.Dk, 8, &a.qs));
  FIX_ROT_TRY(token_stride(k_stride, (long long)d.Hkv * d.Dk, 8, &a.ks));
  FIX_ROT_TRY(token_stride(v_stride, (long long)d.Hkv * d.Dv, 8, &a.vs));
  FIX_ROT_TRY(token_stride(g_stride, (long long)d.Hkv * (d.scalar_gate ? 1 : d.Dv),
                           d.scalar_gate ? 1 : 4, &a.gs));
  a.N = d.N; a.T = d.T; a.nseq = d.nseq; a.cu = p->cu_seqlens;
  a.seqlens = c->seqlens;
  a.Hq = d.Hq; a.Hkv = d.Hkv; a.Dk = d.Dk; a.Dv = d.Dv; a.scalar = d.scalar_gate;
  if (r) {
    a.rot = r->rot_dim; a.interleaved = r->interleaved;
    a.inv_freq = r->inv_freq;
  }
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.g = g;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.table = c->page_table;
  a.page_size = c->page_size; a.num_pages = c->num_pages; a.max_pages = c->max_pages;
  a.k_pages = static_cast<__nv_bfloat16*>(c->k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(c->v_pages);
  a.g_pages = c->g_pages;
  a.status = c->status;
  return launch_tokens(a, static_cast<cudaStream_t>(stream));
}
