// FiX decode over a paged cache: one new query per sequence against the
// pages of its keys, values and log forget gates.  With t = L - 1,
//   S_s = scale q.k_s,  m = max S,  D_s[c] = exp(sum_{r=s+1..t} g_r[c]),
//   o[c] = sum_s exp(S_s - m) D_s[c] v_s[c],
// followed by the norm (or division by l = sum_s exp(S_s - m)) and the output
// gate.
//
// Measured (B200, copy rate 6568 GB/s), Hq 32, Hkv 8, D 128, element-wise
// gate: one sequence of 131,071 tokens in 170 to 175 us, 6.2 TB/s; 64 of 1 to
// 8,191 in 104 to 110 us, 5.7 TB/s; one of 257 in 9.6 us.
//
// What bounds it: every cached byte is read once (1 KB per key and kv head at
// D 128 with the element-wise gate), against 4 flops per q head and channel
// and one exponential per channel, so it runs at memory speed as long as a
// key costs each SM fewer than about 40 cycles.  Around that a call pays some
// 10 us: two launches, the dependent reads lengths -> page table -> tile, and
// the join.
//
// Work split (paged_decode_kernel).  A unit is one (sequence, kv head, block
// of up to 8 NT q heads of its group); its keys are cut into tiles of 16.
// All units form one line, a unit taking a position per tile and kUnitCost
// more for what a warp spends on starting and finishing it; the line is cut
// into equal spans, one per warp of the grid, so that unequal lengths balance
// (they are read on the device).  A warp works alone (own ring of tiles in
// shared memory, no block barriers), newest tile first, so that the decay is
// a running suffix sum of the gates and no factor exceeds 1 for g <= 0.  A
// unit that lies in one span is finished by its warp; the pieces of the
// others leave (m, l, o, total gate) in the workspace, and paged_join_kernel
// joins them: the decay from a piece's last key to t is exp(the later pieces'
// gate totals).
//
// Matrix products (mma.sync: a tile has 16 keys and 8 heads, far too few rows
// for tcgen05 to pay).  Keys take the 16-row side in S^T = K q^T, value
// channels in O^T = V'^T P^T, heads the 8 columns.
// Precision: q k products are exact in the bf16 product and summed in fp32.
// Element-wise gate: V' = D v and P are fp32 values, split into two tf32
// parts each (11 bits and more), three products: about 2^-21.  Scalar gate:
// V stays bf16, D goes to P, which is split into three bf16 parts (24 bits).
// Exponentials are ex2.approx, off by 2 ulp; below 2^-126 they are 0.
// The tensor cores' own fp32 sums truncate, always towards zero, so that a sum
// kept in them drifts (no gates, 32,768 keys in one warp: 2.8e-4 of y): they
// add up one tile's products, from zero, and the running sums are added to
// outside, rounding to nearest.
// Gate sums are kept in units of log 2: a tile's gates are summed by
// themselves, and the tile's sum is added to a compensated total (likewise
// the pieces' totals in the join).  One running fp32 sum over all keys rounds
// the same way at every step where the gates are steady (all of -1e-4, 32,768
// keys in one warp: 9e-5 of y; now 1e-6).  The sum of the weights is
// compensated for the same reason.  The values' running sums are not, for want
// of registers: equal weights and equal values in 32,768 keys, no norm, 2e-5.
// All this costs 4 to 6% where spans are short (256 sequences of 90 to 900
// tokens, 16 q heads per kv head: 51.4 -> 53.3 us; 24 with the scalar gate,
// D 64: 20.4 -> 21.6) and 1% or nothing where the memory sets the pace.
#include <type_traits>

#include "fix_internal.h"

#define FIX_PAGED_TRY(expr)           \
  do {                                \
    fix_status _s = (expr);           \
    if (_s != FIX_OK) return _s;      \
  } while (0)

namespace fix {

constexpr int kTileKeys = 16;
constexpr int kPagedWarps = 4;         // warps per CTA of the split kernel
constexpr int kJoinWarps = 16;         // at most, per CTA
constexpr int kSMs = 148;              // B200
// Line positions of a unit beside its tiles.  0 leaves whole spans of one-tile
// units to single warps (64 unequal sequences: 161 us instead of 105); 1 to 4
// differ by 2 to 4%.
constexpr int kUnitCost = 3;

struct PagedArgs {
  int B, Hq, Hkv, Dk, grp, no_norm, y_f32;
  int nhb, hpb;                        // head blocks per group, heads per block
  float scale_log2, eps;
  int page_size, num_pages, max_pages;
  int page_shift;                      // log2 of the page size, or -1
  const int *table, *seqlens;
  const __nv_bfloat16 *q, *k, *v, *w, *z;
  const float* g;
  void* y;
  int* status;
  int nworkers;
  long long slot_floats;               // floats per slot: hpb (DV + 2) + DV
  float* slots;                        // two per worker
  int4* jobs;                          // the join's work: (pieces, first worker, unit)
  int join_by_unit, heads_per_cta, warps_per_head, heads_per_warp;   // shape of the join
};

__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
  const long long cap = (long long)a.max_pages * a.page_size;
  const int L = a.seqlens[b];
  return L <= 0 ? 0 : (L > cap ? (int)cap : L);
}
__device__ __forceinline__ int tiles_of(int len) {
  return (int)(((unsigned)len + kTileKeys - 1) / kTileKeys);
}
__device__ __forceinline__ int paged_tiles(const PagedArgs& a, int b) {
  return tiles_of(paged_len(a, b));
}
// Line positions of one unit of n tiles.
__device__ __forceinline__ int paged_cost(int n) { return n ? n + kUnitCost : 0; }

__device__ __forceinline__ int warp_upto(int x) {      // sum over this lane and those below
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The line over all sequences, for a whole warp: lane i sums a run of K
// sequences.  (The host refuses sizes whose line could pass 2^31 positions.)
struct Line {
  int K, len;            // sequences per lane; the length of the lane's last one
  int mine, upto;        // positions of this lane's run; of the runs up to it
  __device__ __forceinline__ Line(const PagedArgs& a, int upb) {
    const int lane = threadIdx.x & 31;
    K = (a.B + 31) / 32;
    len = mine = 0;
#pragma unroll 8
    for (int i = lane * K; i < min(a.B, (lane + 1) * K); ++i) {
      len = paged_len(a, i);
      mine += paged_cost(tiles_of(len));
    }
    mine *= upb;
    upto = warp_upto(mine);
  }
  __device__ __forceinline__ int total() const { return __shfl_sync(0xffffffffu, upto, 31); }
  // The sequence b that holds position pos < total(), its length L and where it
  // starts.
  __device__ __forceinline__ void find(const PagedArgs& a, int pos, int upb, int* b, int* L,
                                       int* start) const {
    const int lane = threadIdx.x & 31;
    const int src = __ffs(__ballot_sync(0xffffffffu, upto > pos)) - 1;
    *start = __shfl_sync(0xffffffffu, upto - mine, src);
    if (K == 1) {
      *b = src;
      *L = __shfl_sync(0xffffffffu, len, src);
      return;
    }
    for (int i0 = src * K;; i0 += 32) {                  // within the run, 32 at a time
      const int i = i0 + lane;
      const int l = i < min(a.B, (src + 1) * K) ? paged_len(a, i) : 0;
      const int t = paged_cost(tiles_of(l)) * upb, sum = warp_upto(t);
      const uint32_t in = __ballot_sync(0xffffffffu, *start + sum > pos);
      if (in) {
        const int f = __ffs(in) - 1;
        *b = i0 + f;
        *L = __shfl_sync(0xffffffffu, l, f);
        *start += __shfl_sync(0xffffffffu, sum - t, f);
        return;
      }
      *start += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// x += y and x += y c for N floats, two at a time where N is even.
__device__ __forceinline__ void add_pair(float* x, const float* y) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x[0]), "+f"(x[1])
      : "f"(y[0]), "f"(y[1]));
}
__device__ __forceinline__ void fma_pair(float* x, const float* y, float c) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " mov.b64 c, {%4, %4};\n fma.rn.f32x2 a, b, c, a;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(x[0]), "+f"(x[1])
      : "f"(y[0]), "f"(y[1]), "f"(c));
}
template <int N>
__device__ __forceinline__ void add_n(float* x, const float* y) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 2) add_pair(x + e, y + e);
  } else {
    x[0] += y[0];
  }
}
template <int N>
__device__ __forceinline__ void fma_n(float* x, const float* y, float c) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 2) fma_pair(x + e, y + e, c);
  } else {
    x[0] = fmaf(y[0], c, x[0]);
  }
}
// Adds x, which has the sum's `lost` in it already, and notes what that
// rounds off (compensated summation); a sum that is not finite loses nothing.
__device__ __forceinline__ void add_exactly(float& sum, float& lost, float x) {
  const float s = sum + x;
  lost = fabsf(s) < INFINITY ? x - (s - sum) : 0.f;
  sum = s;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, hi rounded to tf32; the product takes lo's leading 11 bits.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

template <int N>
__device__ __forceinline__ void lds_n(uint32_t addr, float* x) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                 : "r"(addr)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[0]) : "r"(addr) : "memory");
}
template <int N>
__device__ __forceinline__ void sts_n(uint32_t addr, const float* x) {
  if constexpr (N == 4)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3])
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(x[0]), "f"(x[1]) : "memory");
  else
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x[0]) : "memory");
}

// Tiles lie in rows of keys (pitch a multiple of 128 bytes), 16-byte chunk c of
// key s at chunk c ^ (s % 8), so that matrix loads and the gates' reads meet no
// bank conflicts.  With `addr` that of chunk c0 in its row, the chunk c0 + c
// (c0 and c without a bit in common) is at chunk_at(addr, c): one xor with a
// constant for what lies within 128 bytes, the rest a constant offset.
__device__ __forceinline__ constexpr uint32_t chunk_at(uint32_t addr, int c) {
  return (addr ^ ((c & 7) << 4)) + (c >> 3) * 128;
}

// Bytes of one warp's shared memory.
__host__ __device__ constexpr int row_pitch(int bytes) { return bytes < 128 ? 128 : bytes; }
template <int DV, bool SCALAR>
struct Ring {
  static constexpr int kStages = SCALAR || DV <= 64 ? 2 : 1;
  static constexpr int kVPitch = row_pitch(DV * 2);
  static constexpr int kGPitch = row_pitch(DV * 4);
  static constexpr int kV = kTileKeys * kVPitch;
  static constexpr int kG = SCALAR ? 128 : kTileKeys * kGPitch;
  __host__ __device__ static int stage(int Dk) { return kTileKeys * row_pitch(Dk * 2) + kV + kG; }
  __host__ __device__ static int warp_bytes(int Dk, int nt) {
    return (kStages * stage(Dk) + nt * 8 * (Dk * 2 + 16) + 127) / 128 * 128;
  }
};

// The N channels of one lane of a finished row, y = o f [w] [swish(z)]; w and z
// are read when the object is made.
template <int N>
struct Finish {
  float by[N];
  __device__ __forceinline__ Finish(const PagedArgs& a, size_t row0, int c0, bool read) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      by[e] = 1.f;
      if (read && !a.no_norm) by[e] = bf2f(a.w[c0 + e]);
      if (read && a.z) by[e] *= swish(bf2f(a.z[row0 + c0 + e]));
    }
  }
  __device__ __forceinline__ void store(const PagedArgs& a, size_t row0, int c0, const float* o,
                                        float f, bool none) const {
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = none ? 0.f : o[e] * f * by[e];
    if (a.y_f32) {
      float* d = reinterpret_cast<float*>(a.y) + row0 + c0;
      if constexpr (N == 4) *reinterpret_cast<float4*>(d) = make_float4(y[0], y[1], y[2], y[3]);
      else if constexpr (N == 2) *reinterpret_cast<float2*>(d) = make_float2(y[0], y[1]);
      else *d = y[0];
    } else {
      __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(a.y) + row0 + c0;
      if constexpr (N == 4)
        *reinterpret_cast<uint2*>(d) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
      else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(d) = pack2(y[0], y[1]);
      else *d = f2bf(y[0]);
    }
  }
};
template <int N>
__device__ __forceinline__ void load_n(const float* p, float* x) {
  if constexpr (N == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  } else if constexpr (N == 2) {
    const float2 u = *reinterpret_cast<const float2*>(p);
    x[0] = u.x; x[1] = u.y;
  } else {
    x[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float* x) {
  if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  else *p = x[0];
}
// The factor that finishes a row: 1 / rms of its channels, or 1 / l.
template <int N>
__device__ __forceinline__ float row_factor(const PagedArgs& a, const float* o, float l, int DV) {
  if (a.no_norm) return 1.f / l;
  float sq = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) sq += o[e] * o[e];
  return 1.f / sqrtf(warp_sum(sq) / (float)DV + a.eps);
}

// SAME: Dk == DV, known at compile time.
template <int DV, int NT, bool SCALAR, bool SAME>
__global__ void __launch_bounds__(kPagedWarps * 32, NT == 1 ? 3 : 2)
    paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  using R = Ring<DV, SCALAR>;
  constexpr int ST = R::kStages;
  constexpr int MT = DV / 16;
  constexpr int VPL = DV >= 32 ? DV / 32 : 1;      // channels per lane where lanes span a row
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Dk = SAME ? DV : a.Dk;
  const int kpitch = row_pitch(Dk * 2), qpitch = Dk * 2 + 16;
  char* mine = smem + (size_t)warp * R::warp_bytes(Dk, NT);
  const uint32_t ring = smem_addr(mine);
  const int stage_bytes = R::stage(Dk);
  char* sq = mine + ST * stage_bytes;
  const int upb = a.Hkv * a.nhb;

  // this kernel's inputs are there when the one before it has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Line line(a, upb);
  const int total = line.total();
  const int worker = warp * gridDim.x + blockIdx.x;
  // Spans of `less` positions, one more for the first `longer` workers (long
  // ones are evened out so, 64 unequal sequences: 105.1 -> 103.4 us); short
  // ones are all rounded up, for fewer pieces (one sequence of 6,249 tokens:
  // 15.2 us instead of 18.0).
  int less = total / a.nworkers, longer = total - less * a.nworkers;
  if (less < 8) {
    less += longer > 0;
    longer = 0;
  }
  const int first = min(total, less * worker + min(worker, longer));
  const int last = min(total, first + less + (worker < longer));
  int4 job = make_int4(0, 0, 0, 0);      // the unit that begins here and ends beyond
  int b = 0, L = 0, base = 0;            // sequence, its length and line position
  if (first < last) line.find(a, first, upb, &b, &L, &base);

  // lane roles
  const int j = lane & 3, r8 = lane & 7;
  const uint32_t kaddr = (r8 + ((lane >> 3) & 1) * 8) * kpitch + (((lane >> 4) ^ r8) << 4);
  const uint32_t vaddr =
      (r8 + (lane >> 4) * 8) * R::kVPitch + ((((lane >> 3) & 1) ^ r8) << 4);
  const uint32_t qaddr = smem_addr(sq) + r8 * qpitch + (lane >> 3) * 16;
  const int key0 = lane >> 2;                               // and key0 + 8: the S rows
  // gates: of key 2 j and key 2 j + 1, chunk lane / 16, where V' is formed; a
  // lane's own channels of key 0 where the decays are
  const uint32_t gpair0 = 2 * j * R::kGPitch + ((lane >> 2) & 3) * 4 + (((lane >> 4) ^ (2 * j)) << 4);
  const uint32_t gpair1 =
      (2 * j + 1) * R::kGPitch + ((lane >> 2) & 3) * 4 + (((lane >> 4) ^ (2 * j + 1)) << 4);
  const uint32_t gmine = lane * VPL * 4;
  const int kshift = 31 - __clz(Dk / 8);
  const bool whole_pages = a.page_size % kTileKeys == 0;    // a tile lies in one page

  for (int pos = first; pos < last;) {
    const int nb = tiles_of(L), cost = paged_cost(nb);
    if (pos - base >= cost * upb) {                         // next sequence
      base += cost * upb;
      L = paged_len(a, ++b);
      continue;
    }
    const int u = (int)((unsigned)(pos - base) / (unsigned)cost);   // unit of the sequence
    const int live = base + u * cost + kUnitCost;         // position of its tile 0
    const int t0 = max(0, pos - live), t1 = min(nb, last - live);
    if (t1 <= t0) break;                                    // only its start lies in this span
    pos = live + t1;
    const int kv = a.nhb == 1 ? u : u / a.nhb, hb = u - kv * a.nhb;
    const int h0 = kv * a.grp + hb * a.hpb;                 // first q head
    const int nh = min(a.hpb, a.grp - hb * a.hpb);          // q heads
    const int n = t1 - t0;
    const int* table = a.table + (long long)b * a.max_pages;

    // Where the keys of two tiles are: lane i has key i of the pair of tiles
    // 2 p and 2 p + 1.  fetch() starts the read of the page table, a pair ahead
    // of its use; rows() ends it: the key's row in the pools, and which keys
    // are there.
    auto fetch = [&](int pair) {
      const unsigned s = (unsigned)pair * 32 + lane;
      if (pair < 0 || s >= (unsigned)L) return -1;
      return table[a.page_shift >= 0 ? s >> a.page_shift : s / (unsigned)a.page_size];
    };
    uint32_t row = 0, mask = 0;
    auto rows = [&](int pair, int page) {
      const unsigned s = (unsigned)pair * 32 + lane;
      const unsigned slot =
          a.page_shift >= 0 ? s & (a.page_size - 1) : s % (unsigned)a.page_size;
      const bool there = (unsigned)page < (unsigned)a.num_pages;
      if (!there && s < (unsigned)L && a.status) *a.status = FIX_ERR_PAGE;
      row = there ? ((uint32_t)page * a.page_size + slot) * a.Hkv + kv : 0u;
      mask = __ballot_sync(0xffffffffu, there);
    };
    int page = -1;                         // of the pair below the current one
    auto step = [&](int tile) {            // before a tile is copied; tiles go down
      if (tile & 1) {
        rows(tile >> 1, page);
        page = fetch((tile >> 1) - 1);
      }
    };
    // Copies N rows of a tile, CPR 16-byte chunks each, from a pool.  A full tile
    // of one page has evenly spaced rows; keys that are not there are filled
    // with zeros.
    auto copy_rows = [&](uint32_t dst, const void* pool, int tile, auto cpr_, int pitch) {
      constexpr int kFixed = decltype(cpr_)::value;         // chunks per row, 0: Dk / 8
      const int from = (tile & 1) * 16;                     // lane of the tile's first key
      const uint32_t there = mask >> from & 0xffffu;
      const int shift = kFixed ? 0 : kshift;
      const int cpr = kFixed ? kFixed : 1 << shift, per = 32 / cpr;
      const int key = lane / cpr, c = lane % cpr;           // and keys per, 2 per, .. further
      const uint32_t d = dst + key * pitch + ((c ^ (key & 7)) << 4);
      if (whole_pages && there == 0xffffu) {
        const uint32_t r0 = __shfl_sync(0xffffffffu, row, from) + key * a.Hkv;
        const char* src = static_cast<const char*>(pool) + (size_t)r0 * (cpr * 16) + c * 16;
        const uint32_t stride = a.Hkv * cpr * 16;
#pragma unroll
        for (int it = 0; it < (kFixed ? kFixed / 2 : 8); ++it) {
          if (!kFixed && it >= cpr / 2) break;
          copy16(chunk_at(d, (it * per) & 7) + it * per * pitch,
                 src + (size_t)stride * (uint32_t)(it * per), true);
        }
      } else {
#pragma unroll 4
        for (int it = 0; it < cpr / 2; ++it) {
          const int k = key + it * per;
          const uint32_t rr = __shfl_sync(0xffffffffu, row, from + k);
          copy16(chunk_at(d, (it * per) & 7) + it * per * pitch,
                 static_cast<const char*>(pool) + (size_t)rr * (cpr * 16) + c * 16, there >> k & 1);
        }
      }
    };
    auto copy_k = [&](int stage, int tile) {
      copy_rows(ring + stage * stage_bytes, a.k, tile,
                std::integral_constant<int, SAME ? DV / 8 : 0>{}, kpitch);
    };
    auto copy_vg = [&](int stage, int tile) {
      const uint32_t dst = ring + stage * stage_bytes + kTileKeys * kpitch;
      copy_rows(dst, a.v, tile, std::integral_constant<int, DV / 8>{}, R::kVPitch);
      if constexpr (SCALAR) {
        if ((lane & 16) == (tile & 1) * 16)
          copy4(dst + R::kV + (lane & 15) * 4, a.g + row, mask >> lane & 1);
      } else {
        copy_rows(dst + R::kV, a.g, tile, std::integral_constant<int, DV / 4>{}, R::kGPitch);
      }
    };

    uint32_t masks[ST];
    const int page0 = fetch((t1 - 1) >> 1);
    page = fetch(((t1 - 1) >> 1) - 1);
    // the block's queries, rows of 8 NT heads (zero beyond nh)
    for (int i = lane; i < NT * 8 << kshift; i += 32) {
      const int h = i >> kshift, c = i & ((1 << kshift) - 1);
      copy16(smem_addr(sq + h * qpitch + c * 16),
             a.q + ((size_t)b * a.Hq + h0 + min(h, nh - 1)) * Dk + c * 8, h < nh);
    }
    rows((t1 - 1) >> 1, page0);
    int tile = t1 - 1;                     // the next one to copy
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      if (s < n) {
        if (s) step(tile);
        masks[s] = mask >> (tile & 1) * 16 & 0xffffu;
        copy_k(s, tile);
      }
      cp_async_commit();
      if (s < n) copy_vg(s, tile--);
      cp_async_commit();
    }

    float acc[MT][NT][4];
    // of the gates after a tile: their sum and what its roundings lost
    float m[NT][2], l[NT][2], llost[NT][2], suf[VPL], lost[VPL];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = -INFINITY;
        l[t][e] = llost[t][e] = 0.f;
      }
#pragma unroll
    for (int e = 0; e < VPL; ++e) suf[e] = lost[e] = 0.f;

    for (int i = 0; i < n; ++i) {
      const int stage = ST == 1 ? 0 : (i & 1);
      const uint32_t at = ring + stage * stage_bytes;
      const uint32_t vm = masks[0];
      cp_async_wait<2 * ST - 1>();
      __syncwarp();
      // S^T = K q^T
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < (SAME ? (DV + 31) / 32 : 4); ++ks) {       // 32 channels at a time
        if (!SAME && ks * 32 >= Dk) break;
        uint32_t ka[2][4], qf[NT][4];
        ldsm4(chunk_at(at + kaddr, 4 * ks), ka[0]);
        if (Dk > 16) ldsm4(chunk_at(at + kaddr, 4 * ks + 2), ka[1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t qp = qaddr + t * 8 * qpitch + ks * 64;
          if (Dk > 16) ldsm4(qp, qf[t]);
          else ldsm2(qp, qf[t]);
          mma_bf16(s[t], ka[0], qf[t][0], qf[t][1]);
          if (Dk > 16) mma_bf16(s[t], ka[1], qf[t][2], qf[t][3]);
        }
      }
      __syncwarp();
      const bool more = i + ST < n;
      if (more) {
        step(tile);
        copy_k(stage, tile);
      }
      cp_async_commit();

      // softmax of the tile against the running maximum
      float p[NT][4];
      bool moved = false;
      float al[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] *= a.scale_log2;
        if (vm != 0xffffu) {
          if (!((vm >> key0) & 1)) s[t][0] = s[t][1] = -INFINITY;
          if (!((vm >> (key0 + 8)) & 1)) s[t][2] = s[t][3] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[t][e], s[t][2 + e]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[t][e]);
          const float ref = x == -INFINITY ? 0.f : x;
          al[t][e] = ex2(m[t][e] - ref);
          moved |= x != m[t][e];
          m[t][e] = x;
          p[t][e] = ex2(s[t][e] - ref);
          p[t][2 + e] = ex2(s[t][2 + e] - ref);
          // (compensated: nearly equal weights round the same way at every tile)
          const float l0 = l[t][e] * al[t][e], x2 = fmaf(llost[t][e], al[t][e], p[t][e] + p[t][2 + e]);
          l[t][e] = l0 + x2;
          llost[t][e] = x2 - (l[t][e] - l0);
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[x][t][e] *= al[t][e & 1];
      }

      cp_async_wait<2 * ST - 1>();
      __syncwarp();
      const uint32_t vat = at + kTileKeys * kpitch, gat = vat + R::kV;
      if constexpr (SCALAR) {
        // the decay of key (lane & 15), exp of the gates after it, goes to P
        float x;
        lds_n<1>(gat + (lane & 15) * 4, &x);
        x *= kLog2e;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          const float z = __shfl_down_sync(0xffffffffu, x, o, 16);
          if ((lane & 15) + o < 16) x += z;
        }
        float after = __shfl_down_sync(0xffffffffu, x, 1, 16);
        if ((lane & 15) == 15) after = 0.f;
        const float d = ex2(suf[0] + (after + lost[0]));
        add_exactly(suf[0], lost[0], __shfl_sync(0xffffffffu, x, 0, 16) + lost[0]);
        const float d0 = __shfl_sync(0xffffffffu, d, key0), d1 = __shfl_sync(0xffffffffu, d, key0 + 8);
        uint32_t pb[NT][3][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float dd = hf ? d1 : d0;
            float x0 = p[t][2 * hf] * dd, x1 = p[t][2 * hf + 1] * dd;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint32_t w = pack2(x0, x1);
              const float2 f = unpack2(w);
              x0 -= f.x;
              x1 -= f.y;
              pb[t][part][hf] = transpose8(w);
            }
          }
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          uint32_t va[4];
          ldsm4t(chunk_at(vat + vaddr, 2 * x), va);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = 2; part >= 0; --part)
              mma_bf16(sum, va, pb[t][part][0], pb[t][part][1]);
            add_n<4>(acc[x][t], sum);
          }
        }
      } else {
        // gates -> decays in place, a lane on its channels from the newest key
        // back
        if (DV >= 32 || lane < DV) {
          float own[VPL];                    // the tile's sum, with what the total has lost
#pragma unroll
          for (int e = 0; e < VPL; ++e) own[e] = lost[e];
#pragma unroll
          for (int key = kTileKeys - 1; key >= 0; --key) {
            const uint32_t gp = chunk_at(gat + gmine, key & 7) + key * R::kGPitch;
            float x[VPL], d[VPL];
            lds_n<VPL>(gp, x);
#pragma unroll
            for (int e = 0; e < VPL; ++e) d[e] = suf[e];
            add_n<VPL>(d, own);
#pragma unroll
            for (int e = 0; e < VPL; ++e) d[e] = ex2(d[e]);
            fma_n<VPL>(own, x, kLog2e);
            sts_n<VPL>(gp, d);
          }
#pragma unroll
          for (int e = 0; e < VPL; ++e) add_exactly(suf[e], lost[e], own[e]);
        }
        // P^T: the exact fp32 values, transposed as two 16-bit halves
        uint32_t ph[NT][4], pl[NT][4];                       // keys 2j, 2j + 1, 2j + 8, 2j + 9
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t x0 = __float_as_uint(p[t][2 * hf]), x1 = __float_as_uint(p[t][2 * hf + 1]);
            const uint32_t lo = transpose8(__byte_perm(x0, x1, 0x5410));
            const uint32_t hi = transpose8(__byte_perm(x0, x1, 0x7632));
            split_tf32(__uint_as_float(__byte_perm(lo, hi, 0x5410)), ph[t][2 * hf], pl[t][2 * hf]);
            split_tf32(__uint_as_float(__byte_perm(lo, hi, 0x7632)), ph[t][2 * hf + 1],
                       pl[t][2 * hf + 1]);
          }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          uint32_t va[4];
          ldsm4t(chunk_at(vat + vaddr, 2 * x), va);
          uint32_t vh[8], vl[8];            // [2 key + channel half]
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t g0 = chunk_at(gat + gpair0, 4 * x + 2 * ch);
            const uint32_t g1 = chunk_at(gat + gpair1, 4 * x + 2 * ch);
            const float2 v01 = unpack2(va[ch]), v23 = unpack2(va[2 + ch]);
            float d0, d1, d2, d3;
            lds_n<1>(g0, &d0);
            lds_n<1>(g1, &d1);
            lds_n<1>(g0 + 8 * R::kGPitch, &d2);
            lds_n<1>(g1 + 8 * R::kGPitch, &d3);
            split_tf32(v01.x * d0, vh[ch], vl[ch]);
            split_tf32(v01.y * d1, vh[2 + ch], vl[2 + ch]);
            split_tf32(v23.x * d2, vh[4 + ch], vl[4 + ch]);
            split_tf32(v23.y * d3, vh[6 + ch], vl[6 + ch]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              mma_tf32(sum, vl + 4 * ks, ph[t][2 * ks], ph[t][2 * ks + 1]);
              mma_tf32(sum, vh + 4 * ks, pl[t][2 * ks], pl[t][2 * ks + 1]);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              mma_tf32(sum, vh + 4 * ks, ph[t][2 * ks], ph[t][2 * ks + 1]);
            add_n<4>(acc[x][t], sum);
          }
        }
      }
      __syncwarp();
      if constexpr (ST == 2) masks[0] = masks[1];
      if (more) {
        masks[ST - 1] = mask >> (tile & 1) * 16 & 0xffffu;
        copy_vg(stage, tile--);
      }
      cp_async_commit();
    }

    // The piece's rows go through the ring (its tiles are used up), so that
    // lanes span a row: o [heads][DV + 4], then m and l.
    constexpr int OP = DV + 4;
    float* so = reinterpret_cast<float*>(mine);
    float* sml = so + NT * 8 * OP;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = t * 8 + 2 * j + e;
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
        if (lane < 4) {
          sml[2 * h] = m[t][e];
          sml[2 * h + 1] = l[t][e];
        }
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
            so[h * OP + x * 16 + ch * 8 + (lane >> 2)] = acc[x][t][2 * ch + e];
      }
    __syncwarp();
    const int c0 = lane * VPL;
    const bool in_row = c0 < DV;
    if (n == nb) {
      // the whole unit: finish its rows
#pragma unroll 1
      for (int h = 0; h < nh; ++h) {
        float o[VPL];
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[e] = 0.f;
        if (in_row) load_n<VPL>(so + h * OP + c0, o);
        const float lh = sml[2 * h + 1];
        const float f = row_factor<VPL>(a, o, lh, DV);
        const size_t row0 = ((size_t)b * a.Hq + h0 + h) * DV;
        if (in_row) Finish<VPL>(a, row0, c0, true).store(a, row0, c0, o, f, lh == 0.f);
      }
      if (a.join_by_unit && lane == 0) a.jobs[b * upb + u] = make_int4(0, 0, 0, 0);
    } else {
      // slot 1: the unit begins here; slot 0: it began before
      float* slot = a.slots + (2LL * worker + (t0 == 0)) * a.slot_floats;
#pragma unroll 1
      for (int h = 0; h < nh; ++h) {
        float o[VPL];
        if (in_row) {
          load_n<VPL>(so + h * OP + c0, o);
          store_n<VPL>(slot + h * DV + c0, o);
        }
      }
      float* tail = slot + a.hpb * DV;
      if constexpr (SCALAR)
#pragma unroll
        for (int e = 1; e < VPL; ++e) suf[e] = suf[0];      // one gate for all channels
      if (in_row) store_n<VPL>(tail + c0, suf);
      if (lane < 2 * nh) tail[DV + lane] = sml[lane];
      if (t0 == 0) {
        const int end = live + nb - 1, big = longer * (less + 1);
        const int wl = end < big ? end / (less + 1) : longer + (end - big) / less;
        job = make_int4(wl - worker + 1, worker, b * upb + u, 0);
        if (a.join_by_unit && lane == 0) a.jobs[b * upb + u] = job;
      }
    }
    __syncwarp();
  }
  if (!a.join_by_unit && lane == 0) a.jobs[worker] = job;

  // sequences without a token
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int L = a.seqlens[b];
    if (L > 0) {
      if (a.status && threadIdx.x == 0 && L > (long long)a.max_pages * a.page_size)
        *a.status = FIX_ERR_PAGE;
      continue;
    }
    for (long long e = threadIdx.x; e < (long long)a.Hq * DV; e += blockDim.x) {
      const size_t at = (size_t)b * a.Hq * DV + e;
      if (a.y_f32) reinterpret_cast<float*>(a.y)[at] = 0.f;
      else reinterpret_cast<__nv_bfloat16*>(a.y)[at] = f2bf(0.f);
    }
    if (a.join_by_unit)
      for (int u = threadIdx.x; u < upb; u += blockDim.x)
        a.jobs[b * upb + u] = make_int4(0, 0, 0, 0);
  }
}

// Joins the pieces of the units that were cut.  grid.x: the units, or (where
// there are more units than workers) the workers, each for the cut unit that
// begins in its span; grid.y: the head block's heads, heads_per_cta at a time.
// What it costs is the latency of its loads and, with many rows, their number:
//   HPW = 1: a head has warps_per_head warps, each for a run of its pieces,
//     four pieces at a time;
//   HPW = 4: a warp has four heads, which share the reads of the pieces' gate
//     totals, two pieces at a time.
// Pieces are taken newest first; channels lie over the lanes.
template <int DV, int HPW>
__global__ void __launch_bounds__(kJoinWarps * 32 / HPW)
    paged_join_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int VPL = DV >= 32 ? DV / 32 : 1;
  constexpr int kDeep = HPW == 1 ? 4 : 2;      // 8 is no faster, and slower for few pieces
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int upb = a.Hkv * a.nhb;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 job = a.jobs[blockIdx.x];
  const int np = job.x;
  // (the bounds hold unless the workspace or the lengths were written meanwhile)
  if (np < 2 || job.y < 0 || np > a.nworkers - job.y || (unsigned)job.z >= (unsigned)(a.B * upb))
    return;
  const int b = job.z / upb, u = job.z % upb;
  const int kv = u / a.nhb, hb = u % a.nhb;
  const int nh = min(a.hpb, a.grp - hb * a.hpb);
  const int wph = HPW == 1 ? a.warps_per_head : 1;
  const int h = blockIdx.y * a.heads_per_cta + warp / wph * HPW, run = warp % wph;   // and HPW - 1 more
  if (blockIdx.y * a.heads_per_cta >= nh) return;
  const int c0 = lane * VPL;
  const bool live = h < nh && c0 < DV;
  const size_t row0 = ((size_t)b * a.Hq + kv * a.grp + hb * a.hpb + h) * DV;
  const Finish<VPL> finish(a, row0, c0, live && run == 0 && HPW == 1);
  const int runs = min(wph, (np + kDeep - 1) / kDeep);      // warps that have pieces
  const int i0 = run < runs ? np * run / runs : 0, i1 = run < runs ? np * (run + 1) / runs : 0;
  const int tail = a.hpb * DV;
  float M[HPW], l[HPW], o[HPW][VPL], after[VPL], lost[VPL];
#pragma unroll
  for (int k = 0; k < HPW; ++k) {
    M[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < VPL; ++e) o[k][e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < VPL; ++e) after[e] = lost[e] = 0.f;
  if (live) {
    for (int i = i1 - 1; i >= i0; i -= kDeep) {
      float pm[kDeep][HPW], pl[kDeep][HPW], x[kDeep][HPW][VPL], t[kDeep][VPL];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        // a run's last batch may be short: its missing pieces count nothing
        const bool there = i - d >= i0;
        const float* s = a.slots + (2LL * (job.y + i - d) + (i == d)) * a.slot_floats;
#pragma unroll
        for (int k = 0; k < HPW; ++k) {
          const bool head = there && h + k < nh;
          pm[d][k] = head ? s[tail + DV + 2 * (h + k)] : -INFINITY;
          pl[d][k] = head ? s[tail + DV + 2 * (h + k) + 1] : 0.f;
#pragma unroll
          for (int e = 0; e < VPL; ++e) x[d][k][e] = 0.f;
          if (head) load_n<VPL>(s + (h + k) * DV + c0, x[d][k]);
        }
#pragma unroll
        for (int e = 0; e < VPL; ++e) t[d][e] = 0.f;
        if (there) load_n<VPL>(s + tail + c0, t[d]);
      }
      float ref[HPW];
#pragma unroll
      for (int k = 0; k < HPW; ++k) {
        float mx = M[k];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) mx = fmaxf(mx, pm[d][k]);
        ref[k] = mx == -INFINITY ? 0.f : mx;
        const float f0 = ex2(M[k] - ref[k]);
        M[k] = mx;
        l[k] *= f0;
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[k][e] *= f0;
      }
      float own[VPL];                    // the batch's sum, with what the total has lost
#pragma unroll
      for (int e = 0; e < VPL; ++e) own[e] = lost[e];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        float decay[VPL];
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          decay[e] = ex2(after[e] + own[e]);
          own[e] += t[d][e];
        }
#pragma unroll
        for (int k = 0; k < HPW; ++k) {
          // a piece without weight adds nothing, whatever the gates: that of the
          // sequence's first token, which no decay uses, is in `after` by then
          const float f = ex2(pm[d][k] - ref[k]);
          l[k] += f * pl[d][k];
#pragma unroll
          for (int e = 0; e < VPL; ++e)
            if (pl[d][k] != 0.f) o[k][e] += f * x[d][k][e] * decay[e];
        }
      }
#pragma unroll
      for (int e = 0; e < VPL; ++e) add_exactly(after[e], lost[e], own[e]);
    }
  }
  if constexpr (HPW > 1) {
#pragma unroll
    for (int k = 0; k < HPW; ++k) {
      if (h + k >= nh) break;
      const size_t row = row0 + k * DV;
      const float f = row_factor<VPL>(a, o[k], l[k], DV);
      if (live) Finish<VPL>(a, row, c0, true).store(a, row, c0, o[k], f, l[k] == 0.f);
    }
  } else {
    __shared__ float so[kJoinWarps][DV], stot[kJoinWarps][DV], sml[kJoinWarps][2];
    if (live) {
      store_n<VPL>(&so[warp][c0], o[0]);
      store_n<VPL>(&stot[warp][c0], after);
      if (lane == 0) {
        sml[warp][0] = M[0];
        sml[warp][1] = l[0];
      }
    }
    __syncthreads();
    if (run != 0 || h >= nh) return;
    // this head's runs, newest first
    float top = -INFINITY, sum = 0.f, y[VPL];
    for (int i = 0; i < runs; ++i) top = fmaxf(top, sml[warp + i][0]);
    if (top == -INFINITY) top = 0.f;
#pragma unroll
    for (int e = 0; e < VPL; ++e) y[e] = after[e] = 0.f;
#pragma unroll 4
    for (int i = runs - 1; i >= 0; --i) {
      const float f = ex2(sml[warp + i][0] - top), li = sml[warp + i][1];
      sum += f * li;
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        if (li != 0.f) y[e] += f * so[warp + i][c0 + e] * ex2(after[e]);
        after[e] += stot[warp + i][c0 + e];
      }
    }
    const float f = row_factor<VPL>(a, y, sum, DV);
    if (live) finish.store(a, row0, c0, y, f, sum == 0.f);
  }
}

// ---------------------------------------------------------------- host side

// Heads per block: 8 columns of one product, or 16 for groups above 8.
static int paged_nt(const Dims& d) { return d.grp > 8 ? 2 : 1; }

template <int DV, bool SCALAR>
static int paged_smem(int Dk, int nt) {
  return kPagedWarps * Ring<DV, SCALAR>::warp_bytes(Dk, nt);
}
static int paged_smem_bytes(const Dims& d) {
  const int nt = paged_nt(d), Dk = d.Dk;
  switch (d.Dv) {
    case 16: return d.scalar_gate ? paged_smem<16, true>(Dk, nt) : paged_smem<16, false>(Dk, nt);
    case 32: return d.scalar_gate ? paged_smem<32, true>(Dk, nt) : paged_smem<32, false>(Dk, nt);
    case 64: return d.scalar_gate ? paged_smem<64, true>(Dk, nt) : paged_smem<64, false>(Dk, nt);
    default: return d.scalar_gate ? paged_smem<128, true>(Dk, nt) : paged_smem<128, false>(Dk, nt);
  }
}

struct PagedPlan {
  int nt, hpb, nhb, ctas, workers, smem, jobs;
  long long units, slot_floats;
  size_t job_bytes, bytes;
};

// Grid: as many CTAs as the SMs hold at once (three of them by registers with
// one column block, two with two; fewer where their shared memory, of 228 KB
// an SM with 1 KB taken per CTA, does not allow it), but no more than there
// can be tiles.  Planned with the B200's 148 SMs whatever the device, so that
// the workspace size agrees between sizing and calling.
static PagedPlan paged_plan(const Dims& d, const fix_attn_page_cache* c) {
  PagedPlan p{};
  p.nt = paged_nt(d);
  p.hpb = d.grp < 8 * p.nt ? d.grp : 8 * p.nt;
  p.nhb = (d.grp + p.hpb - 1) / p.hpb;
  p.units = (long long)d.B * d.Hkv * p.nhb;
  p.smem = paged_smem_bytes(d);
  const int fit = 228 * 1024 / (p.smem + 1024);
  const int per_sm = fit < (p.nt == 1 ? 3 : 2) ? fit : (p.nt == 1 ? 3 : 2);
  long long cap = (long long)c->max_pages * c->page_size;
  if (cap > INT32_MAX) cap = INT32_MAX;
  const long long tiles = (cap + kTileKeys - 1) / kTileKeys * p.units;
  p.ctas = tiles < (long long)kSMs * per_sm ? (int)tiles : kSMs * per_sm;
  p.workers = p.ctas * kPagedWarps;
  p.slot_floats = ((long long)p.hpb * (d.Dv + 2) + d.Dv + 31) / 32 * 32;
  p.jobs = p.units < p.workers ? (int)p.units : p.workers;
  p.job_bytes = ((size_t)p.jobs * sizeof(int4) + 255) / 256 * 256;
  p.bytes = p.job_bytes + (size_t)p.workers * 2 * p.slot_floats * 4;
  return p;
}

static fix_status paged_dims(const fix_attn_problem* p, const fix_attn_page_cache* c, Dims* d) {
  FIX_PAGED_TRY(validate_problem(p, d));
  if (p->cu_seqlens || p->num_seqs) return FIX_ERR_CU_SEQLENS;   // lengths come with the cache
  if (p->seqlen != 1) return FIX_ERR_SHAPE;
  if ((long long)d->B * d->Hq > (1 << 28)) return FIX_ERR_SHAPE;
  FIX_PAGED_TRY(validate_cache(c, *d));
  // the line of tiles is counted in 32 bits
  long long cap = (long long)c->max_pages * c->page_size;
  if (cap > INT32_MAX) cap = INT32_MAX;
  const PagedPlan pl = paged_plan(*d, c);
  const long long line = ((cap + kTileKeys - 1) / kTileKeys + kUnitCost) * pl.units;
  return line < INT32_MAX - (1 << 16) ? FIX_OK : FIX_ERR_SHAPE;
}

template <int DV, int NT, bool SCALAR, bool SAME>
static fix_status paged_launch(const PagedArgs& a, const PagedPlan& pl, cudaStream_t st) {
  auto* kernel = paged_decode_kernel<DV, NT, SCALAR, SAME>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kernel), pl.smem)) return FIX_ERR_CUDA;
  FIX_PAGED_TRY(OverlappedLaunch(dim3(pl.ctas), kPagedWarps * 32, pl.smem, st).run(kernel, a));
  const OverlappedLaunch join(dim3(pl.jobs, (a.hpb + a.heads_per_cta - 1) / a.heads_per_cta),
                              a.heads_per_cta / a.heads_per_warp * a.warps_per_head * 32, 0, st);
  return a.heads_per_warp == 4 ? join.run(paged_join_kernel<DV, 4>, a)
                               : join.run(paged_join_kernel<DV, 1>, a);
}

template <int DV, bool SCALAR>
static fix_status paged_launch_dv(const PagedArgs& a, const PagedPlan& pl, cudaStream_t st) {
  const bool same = a.Dk == DV;
  if (pl.nt == 1)
    return same ? paged_launch<DV, 1, SCALAR, true>(a, pl, st)
                : paged_launch<DV, 1, SCALAR, false>(a, pl, st);
  return same ? paged_launch<DV, 2, SCALAR, true>(a, pl, st)
              : paged_launch<DV, 2, SCALAR, false>(a, pl, st);
}

}  // namespace fix

using namespace fix;

extern "C" size_t fix_attn_decode_paged_workspace_bytes(const fix_attn_problem* p,
                                                        const fix_attn_page_cache* c) {
  Dims d;
  if (paged_dims(p, c, &d) != FIX_OK) return 0;
  return paged_plan(d, c).bytes;
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
  const PagedPlan pl = paged_plan(d, c);
  if (workspace_bytes < pl.bytes) return FIX_ERR_WORKSPACE;
  FIX_PAGED_TRY(check_device());
  PagedArgs a{};
  a.B = d.B; a.Hq = d.Hq; a.Hkv = d.Hkv; a.Dk = d.Dk; a.grp = d.grp;
  a.no_norm = d.no_norm; a.y_f32 = p->y_dtype == FIX_DTYPE_F32;
  a.nhb = pl.nhb; a.hpb = pl.hpb;
  a.scale_log2 = d.scale * kLog2e; a.eps = d.eps;
  a.page_size = c->page_size; a.num_pages = c->num_pages; a.max_pages = c->max_pages;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c->page_size == 1 << i) a.page_shift = i;
  a.table = c->page_table; a.seqlens = c->seqlens;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(c->k_pages);
  a.v = static_cast<const __nv_bfloat16*>(c->v_pages);
  a.g = c->g_pages;
  a.w = static_cast<const __nv_bfloat16*>(o_norm_weight);
  a.z = static_cast<const __nv_bfloat16*>(o_gate);
  a.y = y;
  a.status = c->status;
  a.nworkers = pl.workers;
  a.slot_floats = pl.slot_floats;
  a.jobs = static_cast<int4*>(workspace);
  a.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.job_bytes);
  // warps per head: about one per piece that a unit of average length has, up
  // to some 4096 in all (28 per SM), and four heads per warp where the rows are
  // more (256 sequences, 2 kv heads, 16 q heads each: 52.9 -> 51.7 us); CTAs of four
  // warps where there are heads enough
  a.join_by_unit = pl.units <= pl.workers;
  const int pieces = pl.workers / pl.jobs;
  const long long rows = (long long)pl.jobs * pl.hpb;
  a.warps_per_head = 1;
  while (a.warps_per_head < kJoinWarps && 2 * a.warps_per_head <= pieces &&
         rows * 2 * a.warps_per_head <= 4096)
    a.warps_per_head *= 2;
  a.heads_per_cta = a.heads_per_warp = rows > 4096 && pl.hpb >= 4 ? 4 : 1;
  while (a.heads_per_cta / a.heads_per_warp * a.warps_per_head < 4 && a.heads_per_cta < pl.hpb)
    a.heads_per_cta *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d.Dv) {
    case 16: return d.scalar_gate ? paged_launch_dv<16, true>(a, pl, st) : paged_launch_dv<16, false>(a, pl, st);
    case 32: return d.scalar_gate ? paged_launch_dv<32, true>(a, pl, st) : paged_launch_dv<32, false>(a, pl, st);
    case 64: return d.scalar_gate ? paged_launch_dv<64, true>(a, pl, st) : paged_launch_dv<64, false>(a, pl, st);
    default: return d.scalar_gate ? paged_launch_dv<128, true>(a, pl, st) : paged_launch_dv<128, false>(a, pl, st);
  }
}
