// Rotation of q and k by position, alone (fix_attn_rotary) or while new
// tokens are appended to a paged cache (fix_attn_append_paged).
//
// A pair (a, b) at position p turns by t = p f:  a' = a cos t - b sin t,
// b' = a sin t + b cos t.  p f is formed in double and loses its whole turns
// there, so that positions of any size keep an angle error near 1e-7; the
// products and sums are float, rounded to bf16 once.
//
// Memory bound: a token's heads are read once and written once.  A token is a
// list of 32-byte units: eight pairs of a rotated head (8 + 8 channels), or 32
// consecutive bytes that are copied.  A warp takes up to kItems units per lane
// of one token, and works alone: it issues all its loads first, then finds the
// token's position, then the sines and cosines (two angles per lane, shared
// within the warp; a lane's units all have the same pairs, as the units of a
// head divide 32), then rotates and stores.
//
// Measured (B200, copy rate 6568 GB/s): 16,384 tokens of 16 + 4 heads of 128
// in 29.0 us, 5.8 TB/s; 4,859 prompt tokens of 16 + 4 heads into pages of 16
// in 18.4 us, 4.6 TB/s; one token of 32 + 8 heads in 2.8 us.
#include "fix_internal.h"

#define FIX_ROT_TRY(expr)             \
  do {                                \
    fix_status _s = (expr);           \
    if (_s != FIX_OK) return _s;      \
  } while (0)

namespace fix {

constexpr int kTokWarps = 4;      // warps per CTA: four tokens

struct TokenArgs {
  int N;                          // tokens
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
  int nq, nk, nv, ng;             // units of a token's q, k, v, g
  int items;                      // units per lane of a warp
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

// Sequence b of token n and its index in it; false behind the last sequence
// (whole warp).
__device__ __forceinline__ bool find_seq(const TokenArgs& a, int n, int* b, long long* t,
                                         long long* len) {
  if (!a.cu) {
    *b = n / a.T;
    *t = n - *b * a.T;
    *len = a.T;
    return true;
  }
  // how many sequences end at or before n: 32 probes a round
  const int lane = threadIdx.x & 31;
  int base = 0, left = a.nseq;
  while (left > 0) {
    const int step = (left + 31) / 32, at = (lane + 1) * step - 1;
    const bool before = at < left && a.cu[base + at + 1] <= n;
    const int skip = __popc(__ballot_sync(0xffffffffu, before)) * step;
    base += skip;
    left = min(step - 1, left - skip);
  }
  if (base >= a.nseq) return false;
  *b = base;
  *t = n - a.cu[base];
  *len = a.cu[base + 1] - a.cu[base];
  return *t >= 0;
}

// Rotates the eight pairs of a unit in place.
__device__ __forceinline__ void rotate_pairs(uint4& x, uint4& y, const float2* f, int interleaved) {
  uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
  uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
  if (!interleaved) {
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

// grid (tokens / 4, runs of 32 a.items units), a warp per token and run
template <int kItems>
__global__ void __launch_bounds__(kTokWarps * 32) token_kernel(const __grid_constant__ TokenArgs a) {
  __shared__ float4 cs[kTokWarps][4][8];        // (cos, sin) of pairs 8 u + 2 i, + 1 at [i][u]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x * kTokWarps + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n >= a.N) return;
  const int uk = a.Dk / 16, u = lane & (uk - 1);
  const int first = blockIdx.y * a.items * 32 + lane;
  const int qk = a.nq + a.nk, qkv = qk + a.nv, all = qkv + a.ng;
  const bool turning = u * 16 < a.rot;
  // Unit id of a token's q starts 32 (id - u) bytes into it, at its head's
  // row, and has its halves e0 and e1 bytes into the row; likewise k.  Units
  // of v and g are 32 bytes after one another.
  const bool apart = turning && !a.interleaved;
  const long long e0 = apart ? -16 * u : 0, step = apart ? a.rot : 16;
  auto unit_of = [&](const void* q, const void* k, const void* v, const void* g, int id) {
    const char* p = static_cast<const char*>(id < a.nq ? q : id < qk ? k : id < qkv ? v : g);
    const int from = id < a.nq ? 0 : id < qk ? a.nq : id < qkv ? qk : qkv;
    return p + (id < qk ? e0 : 0) + (long long)(id - from) * 32;
  };

  uint4 x[kItems], y[kItems];
  const void *qs = a.q + n * a.qs, *ks = a.k + n * a.ks, *vs = a.v + n * a.vs, *gs = a.g + n * a.gs;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int id = first + i * 32;
    if (i < a.items && id < all) {
      const char* p = unit_of(qs, ks, vs, gs, id);
      x[i] = *reinterpret_cast<const uint4*>(p);
      y[i] = *reinterpret_cast<const uint4*>(p + (id < qk ? step : 16));
    }
  }

  const bool gates = a.scalar && blockIdx.y == 0;   // one float per kv head
  const float* gn = a.g + (long long)n * a.gs;
  const float g0 = gates && lane < a.Hkv ? gn[lane] : 0.f;

  // the token's position, and its row in the pools
  int b = 0;
  long long t = 0, len = 0, pos = -1, row = -1;
  bool placed = false;
  if (a.positions) {
    pos = a.positions[n];
    placed = true;
  } else if (find_seq(a, n, &b, &t, &len)) {
    pos = a.seqlens ? (long long)a.seqlens[b] - len + t : t;
    placed = pos >= 0;
  }
  if (a.seqlens && placed) {
    int page = -1;
    unsigned slot = 0;
    if (pos <= INT32_MAX) {                     // not so only for lengths in cu that are none
      const unsigned col = (unsigned)pos / (unsigned)a.page_size;
      slot = (unsigned)pos - col * a.page_size;
      if (col < (unsigned)a.max_pages) page = a.table[(long long)b * a.max_pages + col];
    }
    if ((unsigned)page < (unsigned)a.num_pages) row = (long long)page * a.page_size + slot;
    else if (a.status && lane == 0) *a.status = FIX_ERR_PAGE;
  }

  const bool turn = a.rot && placed;
  float4 f[4];
  if (turn && blockIdx.y * a.items * 32 < qk) {
    float c[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pair = 2 * lane + i;
      // the angle less its whole turns, 2 pi in two doubles
      const double w = pair < a.rot / 2 ? (double)pos * (double)a.inv_freq[pair] : 0.0;
      const double turns = rint(w * 0.15915494309189534);
      const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, w));
      sincospif((float)(r * 0.31830988618379067), &s[i], &c[i]);
      if (a.inverse) s[i] = -s[i];
    }
    cs[warp][lane & 3][lane >> 2] = make_float4(c[0], s[0], c[1], s[1]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = cs[warp][i][u];
  }

  void *qo = a.q_out + (long long)n * a.Hq * a.Dk, *ko = a.k_out + (long long)n * a.Hkv * a.Dk;
  void *kp = a.k_pages + row * a.Hkv * a.Dk, *vp = a.v_pages + row * a.Hkv * a.Dv,
       *gp = a.g_pages + row * a.Hkv * a.Dv;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int id = first + i * 32;
    if (i >= a.items || id >= all) break;
    if (id < qk && turn && turning)
      rotate_pairs(x[i], y[i], reinterpret_cast<const float2*>(f), a.interleaved);
    const long long to1 = id < qk ? step : 16;
    if (id < a.nq || row >= 0) {
      char* d = const_cast<char*>(unit_of(qo, kp, vp, gp, id));
      *reinterpret_cast<uint4*>(d) = x[i];
      *reinterpret_cast<uint4*>(d + to1) = y[i];
    }
    if (a.k_out && id >= a.nq && id < qk) {
      char* d = const_cast<char*>(unit_of(qo, ko, vp, gp, id));
      *reinterpret_cast<uint4*>(d) = x[i];
      *reinterpret_cast<uint4*>(d + to1) = y[i];
    }
  }
  if (gates && row >= 0) {
    float* to = a.g_pages + row * a.Hkv;
    if (lane < a.Hkv) to[lane] = g0;
    for (int h = lane + 32; h < a.Hkv; h += 32) to[h] = gn[h];
  }
}

static bool misaligned(const void* p, unsigned bytes = 16) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

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
  // a token's runs of units fit a grid's y (below 65,536)
  if ((long long)d->Hq * (d->Dk > d->Dv ? d->Dk : d->Dv) > (1 << 25)) return FIX_ERR_SHAPE;
  if (!p->cu_seqlens) return p->num_seqs || p->cu_seqlens_host ? FIX_ERR_CU_SEQLENS : FIX_OK;
  if (p->batch != 1) return FIX_ERR_SHAPE;
  if (p->num_seqs < 1) return FIX_ERR_CU_SEQLENS;
  d->nseq = p->num_seqs;
  return FIX_OK;
}

static fix_status check_rotation(const fix_attn_rotation* r, const Dims& d) {
  if (!r->inv_freq) return FIX_ERR_NULL;
  if (misaligned(r->inv_freq, 4)) return FIX_ERR_ALIGN;
  if (r->rot_dim < 16 || r->rot_dim > d.Dk || r->rot_dim % 16) return FIX_ERR_SHAPE;
  return FIX_OK;
}

fix_status validate_cache(const fix_attn_page_cache* c, const Dims& d) {
  if (!c) return FIX_ERR_NULL;
  if (c->page_size < 1 || c->num_pages < 1 || c->max_pages < 1) return FIX_ERR_SHAPE;
  if ((unsigned long long)c->num_pages * c->page_size >= (1ULL << 32) / d.Hkv) return FIX_ERR_SHAPE;
  if (!c->page_table || !c->seqlens || !c->k_pages || !c->v_pages || !c->g_pages) return FIX_ERR_NULL;
  for (const void* x : {(const void*)c->k_pages, (const void*)c->v_pages, (const void*)c->g_pages})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  for (const void* x : {(const void*)c->page_table, (const void*)c->seqlens, (const void*)c->status})
    if (misaligned(x, 4)) return FIX_ERR_ALIGN;
  return FIX_OK;
}

// Units per lane: eight keep enough loads in flight with few warps; fewer
// where the tokens are too few to fill the SMs (eight warps on each of the
// B200's 148) otherwise.
static fix_status launch_tokens(TokenArgs& a, cudaStream_t st) {
  FIX_ROT_TRY(check_device());
  const long long units = (long long)a.nq + a.nk + a.nv + a.ng;
  const long long per_lane = units > 32 ? (units + 31) / 32 : 1;
  int most = 8;
  while (most > 1 && (long long)a.N * ((per_lane + most - 1) / most) < 148 * 8) most /= 2;
  const long long runs = (per_lane + most - 1) / most;
  a.items = (int)((per_lane + runs - 1) / runs);
  const OverlappedLaunch launch(dim3((a.N + kTokWarps - 1) / kTokWarps, (unsigned)runs),
                                kTokWarps * 32, 0, st);
  switch (most) {
    case 1: return launch.run(token_kernel<1>, a);
    case 2: return launch.run(token_kernel<2>, a);
    case 4: return launch.run(token_kernel<4>, a);
    default: return launch.run(token_kernel<8>, a);
  }
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
  for (const void* x : {q, k, (const void*)q_out, (const void*)k_out})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  if (misaligned(positions, 4) || misaligned(p->cu_seqlens, 8)) return FIX_ERR_ALIGN;
  TokenArgs a{};
  FIX_ROT_TRY(token_stride(q_stride, (long long)d.Hq * d.Dk, 8, &a.qs));
  FIX_ROT_TRY(token_stride(k_stride, (long long)d.Hkv * d.Dk, 8, &a.ks));
  a.N = d.N; a.T = d.T; a.nseq = d.nseq; a.cu = p->cu_seqlens;
  a.positions = positions;
  a.Hq = d.Hq; a.Hkv = d.Hkv; a.Dk = d.Dk; a.Dv = d.Dv;
  a.rot = r->rot_dim; a.interleaved = r->interleaved; a.inverse = inverse;
  a.inv_freq = r->inv_freq;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.nq = d.Hq * (d.Dk / 16);
  a.nk = k ? d.Hkv * (d.Dk / 16) : 0;
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
  for (const void* x : {q, k, v, (const void*)q_out, (const void*)k_out})
    if (misaligned(x)) return FIX_ERR_ALIGN;
  if (misaligned(g, d.scalar_gate ? 4 : 16) || misaligned(p->cu_seqlens, 8)) return FIX_ERR_ALIGN;
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
  a.nq = q ? d.Hq * (d.Dk / 16) : 0;
  a.nk = d.Hkv * (d.Dk / 16);
  a.nv = d.Hkv * (d.Dv / 16);
  a.ng = d.scalar_gate ? 0 : d.Hkv * (d.Dv / 8);
  return launch_tokens(a, static_cast<cudaStream_t>(stream));
}
