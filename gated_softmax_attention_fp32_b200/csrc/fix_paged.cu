// FiX decode over a paged cache: one new query per sequence against the
// pages of its keys, values and log forget gates.  With t = L - 1,
//   S_s = scale q.k_s,  m = max S,  D_s[c] = exp(sum_{r=s+1..t} g_r[c]),
//   o[c] = sum_s exp(S_s - m) D_s[c] v_s[c],
// followed by the norm (or division by l = sum_s exp(S_s - m)) and the output
// gate.
//
// What bounds it: every cached byte is read once (1 KB per key and kv head at
// D 128 with the element-wise gate), against 2 flops per q head and channel
// and one exponential per channel, so it should run at memory speed as long
// as a key costs each SM fewer than about 40 cycles.
//
// Work split (paged_decode_kernel).  A unit is one (sequence, kv head, block
// of up to 8 NT q heads of its group); its keys are cut into tiles of 16.
// All units' tiles form one line, cut into equal spans, one per warp of the
// grid: unequal lengths balance, and the lengths are read on the device.  A
// warp works alone (own ring of tiles in shared memory, no block barriers),
// newest tile first, so that the decay is a running suffix sum of the gates
// and no factor exceeds 1 for g <= 0.  A piece that is a whole unit is
// finished by its warp; the others leave (m, l, o, total gate) in a slot of
// the workspace and paged_join_kernel joins a unit's pieces: the decay from a
// piece's last key to t is exp(the later pieces' gate totals).
//
// Matrix products (mma.sync: a tile has 16 keys and 8 heads, far too few rows
// for tcgen05 to pay).  Keys take the 16-row side in S^T = K q^T and the
// reduced side in O^T = V'^T P^T, heads the 8 columns.  The reduced side may
// be permuted freely: lane j of four takes keys 4j..4j+3, so that a suffix sum
// over the tile's gates is three additions in a lane and a scan over four
// lanes.  Row r of the S product is therefore key 4 (r / 2) + r % 2, and + 2
// for r >= 8.
// Precision: q k products are exact in the bf16 product and summed in fp32.
// Element-wise gate: V' = D v and P are fp32 values, split into two tf32
// parts each (11 bits and more), three products: about 2^-21.  Scalar gate:
// V stays bf16, D goes to P, which is split into three bf16 parts (24 bits).
#include "fix_internal.h"

#define FIX_PAGED_TRY(expr)           \
  do {                                \
    fix_status _s = (expr);           \
    if (_s != FIX_OK) return _s;      \
  } while (0)

namespace fix {

constexpr int kTileKeys = 16;
constexpr int kPagedWarps = 4;         // warps per CTA of the split kernel
constexpr int kJoinThreads = 256;
constexpr int kSMs = 148;              // B200

struct PagedArgs {
  int B, Hq, Hkv, Dk, grp, no_norm, y_f32;
  int nhb, hpb;                        // head blocks per group, heads per block
  float scale_log2, eps;
  int page_size, num_pages, max_pages;
  const int *table, *seqlens;
  const __nv_bfloat16 *q, *k, *v, *w, *z;
  const float* g;
  void* y;
  int* status;
  int nworkers;
  long long slot_floats;               // floats per slot: hpb (DV + 2) + DV
  float* slots;                        // two per worker
  int units;                           // B * Hkv * nhb
  int join_by_unit, heads_per_cta;     // shape of the join
};

__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
  const long long cap = (long long)a.max_pages * a.page_size;
  const int L = a.seqlens[b];
  return L <= 0 ? 0 : (L > cap ? (int)cap : L);
}
__device__ __forceinline__ int paged_tiles(const PagedArgs& a, int b) {
  return (int)(((unsigned)paged_len(a, b) + kTileKeys - 1) / kTileKeys);
}
__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Tiles of one head block over all sequences (whole warp).
__device__ __forceinline__ long long tiles_total(const PagedArgs& a) {
  long long n = 0;
#pragma unroll 8
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += paged_tiles(a, b);
  return warp_sum_ll(n);
}
// Tiles of one head block before sequence b (whole warp).
__device__ __forceinline__ long long tiles_before(const PagedArgs& a, int b) {
  long long n = 0;
#pragma unroll 8
  for (int i = threadIdx.x & 31; i < b; i += 32) n += paged_tiles(a, i);
  return warp_sum_ll(n);
}
// The sequence that holds tile `pos` of the line (pos below its length, a
// line of `upb` units per sequence) and the line position where it starts
// (whole warp).
__device__ __forceinline__ void find_tile(const PagedArgs& a, long long pos, int upb, int* b,
                                          long long* start) {
  const int lane = threadIdx.x & 31;
  const int K = (a.B + 31) / 32;                  // sequences per lane
  long long n = 0;
#pragma unroll 8
  for (int i = lane * K; i < min(a.B, (lane + 1) * K); ++i) n += paged_tiles(a, i);
  n *= upb;
  long long incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, incl > pos)) - 1;
  long long at = __shfl_sync(0xffffffffu, incl - n, src);
  int i = src * K;
  for (;;) {
    const long long t = (long long)paged_tiles(a, i) * upb;
    if (pos < at + t || i + 1 >= a.B) break;
    at += t;
    ++i;
  }
  *b = i;
  *start = at;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

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

// Bytes of one warp's shared memory.
__host__ __device__ constexpr int row_pitch(int bytes) { return bytes < 128 ? 128 : bytes; }
template <int DV, bool SCALAR>
struct Ring {
  static constexpr int kStages = SCALAR || DV <= 64 ? 2 : 1;
  static constexpr int kVPitch = row_pitch(DV * 2);
  static constexpr int kGPitch = row_pitch(DV * 4);
  static constexpr int kV = kTileKeys * kVPitch;
  static constexpr int kG = SCALAR ? 64 : kTileKeys * kGPitch;
  __host__ __device__ static int stage(int Dk) { return kTileKeys * row_pitch(Dk * 2) + kV + kG; }
  __host__ __device__ static int warp_bytes(int Dk, int nt) {
    return (kStages * stage(Dk) + nt * 8 * (Dk * 2 + 16) + 127) / 128 * 128;
  }
};

// Finishes one row's channel value.
__device__ __forceinline__ void store_y(const PagedArgs& a, size_t at, float y) {
  if (a.z) y *= swish(bf2f(a.z[at]));
  if (a.y_f32) reinterpret_cast<float*>(a.y)[at] = y;
  else reinterpret_cast<__nv_bfloat16*>(a.y)[at] = f2bf(y);
}

template <int DV, int NT, bool SCALAR>
__global__ void __launch_bounds__(kPagedWarps * 32, NT == 1 ? 3 : 2)
    paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  using R = Ring<DV, SCALAR>;
  constexpr int ST = R::kStages;
  constexpr int MT = DV / 16;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Dk = a.Dk;
  const int kpitch = row_pitch(Dk * 2), qpitch = Dk * 2 + 16;
  char* mine = smem + (size_t)warp * R::warp_bytes(Dk, NT);
  const uint32_t ring = smem_addr(mine);
  const int stage_bytes = R::stage(Dk);
  char* sq = mine + ST * stage_bytes;

  // sequences without a token
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (a.seqlens[b] > 0) {
      if (a.status && threadIdx.x == 0 && a.seqlens[b] > (long long)a.max_pages * a.page_size)
        *a.status = FIX_ERR_PAGE;
      continue;
    }
    for (int e = threadIdx.x; e < a.Hq * DV; e += blockDim.x) {
      const size_t at = (size_t)b * a.Hq * DV + e;
      if (a.y_f32) reinterpret_cast<float*>(a.y)[at] = 0.f;
      else reinterpret_cast<__nv_bfloat16*>(a.y)[at] = f2bf(0.f);
    }
  }

  const int upb = a.Hkv * a.nhb;
  const long long total = tiles_total(a) * upb;
  const int worker = warp * gridDim.x + blockIdx.x;
  const long long span = (total + a.nworkers - 1) / a.nworkers;
  const long long first = span * worker, last = min(total, first + span);
  if (first >= last) return;
  int b;
  long long base;                     // line position of sequence b
  find_tile(a, first, upb, &b, &base);

  // lane roles
  const int j = lane & 3, r8 = lane & 7;
  const int ldkey = ((r8 >> 1) << 2) | (r8 & 1);            // key of matrix row r8
  const uint32_t kaddr = (uint32_t)(ldkey + ((lane >> 3) & 1) * 2) * kpitch;
  const int kchunk = lane >> 4;
  const uint32_t vaddr = (uint32_t)(ldkey + (lane >> 4) * 2) * R::kVPitch;
  const int vchunk = (lane >> 3) & 1;
  const int key0 = ((lane >> 3) << 2) | ((lane >> 2) & 1);  // keys of this lane's two S rows
  const int kshift = 31 - __clz(Dk / 8);

  for (long long pos = first; pos < last;) {
    const int L = paged_len(a, b);
    const int nb = (int)(((unsigned)L + kTileKeys - 1) / kTileKeys);
    if (pos >= base + (long long)nb * upb) {                // next sequence
      base += (long long)nb * upb;
      ++b;
      continue;
    }
    const int u = (int)((pos - base) / nb);                 // unit of the sequence
    const int t0 = (int)((pos - base) - (long long)u * nb);
    const int t1 = (int)min((long long)nb, t0 + (last - pos));
    const int kv = u / a.nhb, hb = u - kv * a.nhb;
    const int h0 = kv * a.grp + hb * a.hpb;                 // first q head
    const int nh = min(a.hpb, a.grp - hb * a.hpb);          // q heads
    const int n = t1 - t0;
    const int* table = a.table + (long long)b * a.max_pages;

    // row of key (lane & 15) of a tile in the pools, and which keys are there
    auto lookup = [&](int tile, uint32_t& row, uint32_t& mask) {
      const unsigned s = (unsigned)tile * kTileKeys + (lane & 15);
      int page = -1;
      unsigned slot = 0;
      if (s < (unsigned)L) {
        const unsigned col = s / (unsigned)a.page_size;
        slot = s - col * a.page_size;
        page = table[col];
        if ((unsigned)page >= (unsigned)a.num_pages) {
          page = -1;
          if (a.status) *a.status = FIX_ERR_PAGE;
        }
      }
      row = page < 0 ? 0u : ((uint32_t)page * a.page_size + slot) * a.Hkv + kv;
      mask = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    };
    auto copy_k = [&](int stage, uint32_t row, uint32_t mask) {
      const uint32_t dst = ring + stage * stage_bytes;
#pragma unroll 8
      for (int it = 0; it < Dk / 16; ++it) {
        const int idx = it * 32 + lane, key = idx >> kshift, c = idx & ((1 << kshift) - 1);
        const uint32_t rr = __shfl_sync(0xffffffffu, row, key);
        const int f = ((key >> 2) << 1) | (key & 1);
        copy16(dst + key * kpitch + ((c ^ f) << 4), a.k + (size_t)rr * Dk + c * 8,
               (mask >> key) & 1);
      }
    };
    auto copy_vg = [&](int stage, uint32_t row, uint32_t mask) {
      const uint32_t dst = ring + stage * stage_bytes + kTileKeys * kpitch;
#pragma unroll
      for (int it = 0; it < DV / 16; ++it) {
        const int idx = it * 32 + lane, key = idx / (DV / 8), c = idx % (DV / 8);
        const uint32_t rr = __shfl_sync(0xffffffffu, row, key);
        const int f = ((key >> 2) << 1) | (key & 1);
        copy16(dst + key * R::kVPitch + ((c ^ f) << 4), a.v + (size_t)rr * DV + c * 8,
               (mask >> key) & 1);
      }
      const uint32_t gdst = dst + R::kV;
      if (SCALAR) {
        if (lane < kTileKeys) copy4(gdst + lane * 4, a.g + row, (mask >> lane) & 1);
      } else {
#pragma unroll
        for (int it = 0; it < DV / 8; ++it) {
          const int idx = it * 32 + lane, key = idx / (DV / 4), c = idx % (DV / 4);
          const uint32_t rr = __shfl_sync(0xffffffffu, row, key);
          copy16(gdst + key * R::kGPitch + ((c ^ ((key >> 2) << 1)) << 4),
                 a.g + (size_t)rr * DV + c * 4, (mask >> key) & 1);
        }
      }
    };

    uint32_t row, mask, masks[ST];
    lookup(t1 - 1, row, mask);
    // the block's queries, rows of 8 NT heads (zero beyond nh)
    __syncwarp();
    for (int i = lane; i < NT * 8 << kshift; i += 32) {
      const int h = i >> kshift, c = i & ((1 << kshift) - 1);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (h < nh)
        x = *reinterpret_cast<const uint4*>(a.q + ((size_t)b * a.Hq + h0 + h) * Dk + c * 8);
      *reinterpret_cast<uint4*>(sq + h * qpitch + c * 16) = x;
    }
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      masks[s] = mask;
      if (s < n) copy_k(s, row, mask);
      cp_async_commit();
      if (s < n) copy_vg(s, row, mask);
      cp_async_commit();
      if (s + 1 < n) lookup(t1 - 2 - s, row, mask);
    }

    float acc[MT][NT][4];
    float m[NT][2], l[NT][2];
    float suf[SCALAR ? 1 : MT][2];
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
        l[t][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < (SCALAR ? 1 : MT); ++i) suf[i][0] = suf[i][1] = 0.f;

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
#pragma unroll 8
      for (int ks = 0; ks < Dk / 16; ++ks) {
        uint32_t ka[4];
        ldsm4(at + kaddr + (((ks * 2 + kchunk) ^ r8) << 4), ka);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const char* qp = sq + (t * 8 + (lane >> 2)) * qpitch + ks * 32 + j * 4;
          mma_bf16(s[t], ka, *reinterpret_cast<const uint32_t*>(qp),
                   *reinterpret_cast<const uint32_t*>(qp + 16));
        }
      }
      __syncwarp();
      if (i + ST < n) copy_k(stage, row, mask);
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
          if (!((vm >> (key0 + 2)) & 1)) s[t][2] = s[t][3] = -INFINITY;
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
          l[t][e] = l[t][e] * al[t][e] + p[t][e] + p[t][2 + e];
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
      const uint32_t vat = at + kTileKeys * kpitch;
      const char* gat = mine + stage * stage_bytes + kTileKeys * kpitch + R::kV;
      if constexpr (SCALAR) {
        // the decay of key (lane & 15), exp of the gates after it, goes to P
        float x = reinterpret_cast<const float*>(gat)[lane & 15];
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          const float z = __shfl_down_sync(0xffffffffu, x, o, 16);
          if ((lane & 15) + o < 16) x += z;
        }
        float after = __shfl_down_sync(0xffffffffu, x, 1, 16);
        if ((lane & 15) == 15) after = 0.f;
        const float d = ex2((suf[0][0] + after) * kLog2e);
        suf[0][0] += __shfl_sync(0xffffffffu, x, 0, 16);
        const float d0 = __shfl_sync(0xffffffffu, d, key0), d1 = __shfl_sync(0xffffffffu, d, key0 + 2);
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
          ldsm4t(vat + vaddr + (((x * 2 + vchunk) ^ r8) << 4), va);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int part = 0; part < 3; ++part)
              mma_bf16(acc[x][t], va, pb[t][part][0], pb[t][part][1]);
        }
      } else {
        // P^T: the exact fp32 values, transposed as two 16-bit halves
        uint32_t ph[NT][4], pl[NT][4];                       // keys 4j .. 4j + 3
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
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          uint32_t va[4];
          ldsm4t(vat + vaddr + (((x * 2 + vchunk) ^ r8) << 4), va);
          uint32_t vh[8], vl[8];            // [2 key + channel half]
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const char* gp = gat + 4 * j * R::kGPitch +
                             (((x * 4 + (lane >> 4) + 2 * ch) ^ (2 * j)) << 4) + ((lane >> 2) & 3) * 4;
            float gk[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) gk[y] = *reinterpret_cast<const float*>(gp + y * R::kGPitch);
            const float e2 = gk[3], e1 = e2 + gk[2], e0 = e1 + gk[1];
            float z, sum = e0 + gk[0];
            z = __shfl_down_sync(0xffffffffu, sum, 1, 4);
            if (j < 3) sum += z;
            z = __shfl_down_sync(0xffffffffu, sum, 2, 4);
            if (j < 2) sum += z;
            float after = __shfl_down_sync(0xffffffffu, sum, 1, 4);
            if (j == 3) after = 0.f;
            after = (after + suf[x][ch]) * kLog2e;
            suf[x][ch] += __shfl_sync(0xffffffffu, sum, 0, 4);
            const float2 v01 = unpack2(va[ch]), v23 = unpack2(va[2 + ch]);
            split_tf32(v01.x * ex2(fmaf(e0, kLog2e, after)), vh[ch], vl[ch]);
            split_tf32(v01.y * ex2(fmaf(e1, kLog2e, after)), vh[2 + ch], vl[2 + ch]);
            split_tf32(v23.x * ex2(fmaf(e2, kLog2e, after)), vh[4 + ch], vl[4 + ch]);
            split_tf32(v23.y * ex2(after), vh[6 + ch], vl[6 + ch]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              mma_tf32(acc[x][t], vl + 4 * ks, ph[t][2 * ks], ph[t][2 * ks + 1]);
              mma_tf32(acc[x][t], vh + 4 * ks, pl[t][2 * ks], pl[t][2 * ks + 1]);
              mma_tf32(acc[x][t], vh + 4 * ks, ph[t][2 * ks], ph[t][2 * ks + 1]);
            }
        }
      }
      __syncwarp();
      if (i + ST < n) copy_vg(stage, row, mask);
      cp_async_commit();
      if constexpr (ST == 2) masks[0] = masks[1];
      masks[ST - 1] = mask;
      if (i + ST + 1 < n) lookup(t1 - 2 - ST - i, row, mask);
    }

#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
        l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
      }
    if (n == nb) {
      // the whole unit: finish its rows
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = t * 8 + 2 * j + e;
          float f;
          if (a.no_norm) {
            f = 1.f / l[t][e];
          } else {
            float sq2 = 0.f;
#pragma unroll
            for (int x = 0; x < MT; ++x)
              sq2 += acc[x][t][e] * acc[x][t][e] + acc[x][t][2 + e] * acc[x][t][2 + e];
            sq2 += __shfl_xor_sync(0xffffffffu, sq2, 4);
            sq2 += __shfl_xor_sync(0xffffffffu, sq2, 8);
            sq2 += __shfl_xor_sync(0xffffffffu, sq2, 16);
            f = 1.f / sqrtf(sq2 / (float)DV + a.eps);
          }
          if (h >= nh) continue;
          const bool none = l[t][e] == 0.f;          // no finite logit
          const size_t row0 = ((size_t)b * a.Hq + h0 + h) * DV;
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              const int c = x * 16 + ch * 8 + (lane >> 2);
              float y = acc[x][t][2 * ch + e] * f;
              if (!a.no_norm) y *= bf2f(a.w[c]);
              store_y(a, row0 + c, none ? 0.f : y);
            }
        }
    } else {
      float* slot = a.slots + (2LL * worker + (pos == first ? 0 : 1)) * a.slot_floats;
      float* sm = slot + a.hpb * DV;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = t * 8 + 2 * j + e;
          if (h >= nh) continue;
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
              slot[h * DV + x * 16 + ch * 8 + (lane >> 2)] = acc[x][t][2 * ch + e];
          if (lane < 4) {
            sm[h] = m[t][e];
            sm[a.hpb + h] = l[t][e];
          }
        }
      float* tot = sm + 2 * a.hpb;
      if constexpr (SCALAR) {
        if (lane == 0) tot[0] = suf[0][0];
      } else {
        if (j == 0) {
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) tot[x * 16 + ch * 8 + (lane >> 2)] = suf[x][ch];
        }
      }
    }
    pos += n;
  }
}

// Joins the pieces of the units that were cut.  grid.x: the units, or (where
// there are more units than workers) the workers, each for the cut unit that
// begins in its span; grid.y: the head blocks' heads, heads_per_cta at a time.
// A head has 8 / heads_per_cta warps, each for a run of its pieces; channels
// lie over the lanes.  Launched so that it may start while the split kernel
// still runs: what it reads before the wait are that kernel's inputs.
template <int DV, bool SCALAR>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int VPL = DV >= 32 ? DV / 32 : 1;
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float so[kWarps][DV], stot[kWarps][DV], sml[kWarps][2];
  __shared__ int s_unit, s_np, s_w0, s_slot1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int upb = a.Hkv * a.nhb;
  if (warp == 0) {
    const long long total = tiles_total(a) * upb;
    const long long span = (total + a.nworkers - 1) / a.nworkers;
    int b = 0, u = 0;
    long long start = 0;
    int nb = 0;
    if (a.join_by_unit) {
      b = blockIdx.x / upb;
      u = blockIdx.x % upb;
      nb = paged_tiles(a, b);
      start = tiles_before(a, b) * upb + (long long)u * nb;
    } else {
      const long long e = span * (blockIdx.x + 1);          // where the worker's span ends
      if (e < total) {
        long long base;
        find_tile(a, e, upb, &b, &base);
        nb = paged_tiles(a, b);
        u = (int)((e - base) / nb);
        start = base + (long long)u * nb;
        if (start == e || start < span * blockIdx.x) nb = 0;   // not cut here, or begun before
      }
    }
    if (lane == 0) {
      int np = 0, w0 = 0;
      if (nb > 0) {
        w0 = (int)(start / span);
        np = (int)((start + nb - 1) / span) - w0 + 1;
      }
      s_np = np;
      s_w0 = w0;
      s_unit = b * upb + u;
      s_slot1 = start != (long long)w0 * span;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int np = s_np;
  if (np < 2) return;
  const int b = s_unit / upb, u = s_unit % upb;
  const int kv = u / a.nhb, hb = u % a.nhb;
  const int nh = min(a.hpb, a.grp - hb * a.hpb);
  const int wph = kWarps / a.heads_per_cta;                 // warps per head
  const int h = blockIdx.y * a.heads_per_cta + warp / wph, run = warp % wph;
  if (blockIdx.y * a.heads_per_cta >= nh) return;
  const bool live = h < nh && lane * VPL < DV;
  auto slot_of = [&](int i) {
    return a.slots + (2LL * (s_w0 + i) + (i == 0 ? s_slot1 : 0)) * a.slot_floats;
  };
  const int i0 = (int)((long long)np * run / wph), i1 = (int)((long long)np * (run + 1) / wph);
  const int c0 = lane * VPL;
  float M = -INFINITY, l = 0.f, o[VPL], after[VPL];
#pragma unroll
  for (int e = 0; e < VPL; ++e) o[e] = after[e] = 0.f;
  if (h < nh) {
    for (int i = i0 + lane; i < i1; i += 32) M = fmaxf(M, slot_of(i)[a.hpb * DV + h]);
    M = warp_max(M);
  }
  const float ref = M == -INFINITY ? 0.f : M;
  if (live) {
#pragma unroll 4
    for (int i = i1 - 1; i >= i0; --i) {
      const float* s = slot_of(i);
      const float f = ex2(s[a.hpb * DV + h] - ref);
      l += f * s[a.hpb * (DV + 1) + h];
      const float* tot = s + a.hpb * (DV + 2);
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        o[e] += f * s[h * DV + c0 + e] * ex2(after[e] * kLog2e);
        after[e] += SCALAR ? tot[0] : tot[c0 + e];
      }
    }
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
      so[warp][c0 + e] = o[e];
      stot[warp][c0 + e] = after[e];
    }
    if (lane == 0) {
      sml[warp][0] = M;
      sml[warp][1] = l;
    }
  }
  __syncthreads();
  if (run != 0 || h >= nh) return;
  // this head's runs, newest first
  M = -INFINITY;
  for (int i = 0; i < wph; ++i) M = fmaxf(M, sml[warp + i][0]);
  if (M == -INFINITY) M = 0.f;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < VPL; ++e) o[e] = after[e] = 0.f;
  for (int i = wph - 1; i >= 0; --i) {
    const float f = ex2(sml[warp + i][0] - M);
    l += f * sml[warp + i][1];
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
      o[e] += f * so[warp + i][c0 + e] * ex2(after[e] * kLog2e);
      after[e] += stot[warp + i][c0 + e];
    }
  }
  const bool none = l == 0.f;                               // no finite logit
  float f;
  if (a.no_norm) {
    f = 1.f / l;
  } else {
    float sq2 = 0.f;
#pragma unroll
    for (int e = 0; e < VPL; ++e) sq2 += o[e] * o[e];
    f = 1.f / sqrtf(warp_sum(sq2) / (float)DV + a.eps);
  }
  if (!live) return;
  const size_t at = ((size_t)b * a.Hq + kv * a.grp + hb * a.hpb + h) * DV + c0;
#pragma unroll
  for (int e = 0; e < VPL; ++e) {
    float y = o[e] * f;
    if (!a.no_norm) y *= bf2f(a.w[c0 + e]);
    store_y(a, at + e, none ? 0.f : y);
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
  int nt, hpb, nhb, units, ctas, workers, smem;
  long long slot_floats;
  size_t bytes;
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
  p.units = d.B * d.Hkv * p.nhb;
  p.smem = paged_smem_bytes(d);
  const int fit = 228 * 1024 / (p.smem + 1024);
  const int per_sm = fit < (p.nt == 1 ? 3 : 2) ? fit : (p.nt == 1 ? 3 : 2);
  long long cap = (long long)c->max_pages * c->page_size;
  if (cap > INT32_MAX) cap = INT32_MAX;
  const long long tiles = (cap + kTileKeys - 1) / kTileKeys * p.units;
  p.ctas = tiles < (long long)kSMs * per_sm ? (int)tiles : kSMs * per_sm;
  p.workers = p.ctas * kPagedWarps;
  p.slot_floats = ((long long)p.hpb * (d.Dv + 2) + d.Dv + 31) / 32 * 32;
  p.bytes = (size_t)p.workers * 2 * p.slot_floats * 4;
  return p;
}

static fix_status paged_dims(const fix_attn_problem* p, const fix_attn_page_cache* c, Dims* d) {
  FIX_PAGED_TRY(validate_problem(p, d));
  if (p->cu_seqlens || p->num_seqs) return FIX_ERR_CU_SEQLENS;   // lengths come with the cache
  if (p->seqlen != 1) return FIX_ERR_SHAPE;
  if ((long long)d->B * d->Hq > (1 << 28)) return FIX_ERR_SHAPE;
  return validate_cache(c, *d);
}

template <int DV, int NT, bool SCALAR>
static fix_status paged_launch(const PagedArgs& a, const PagedPlan& pl, cudaStream_t st) {
  auto* kernel = paged_decode_kernel<DV, NT, SCALAR>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kernel), pl.smem)) return FIX_ERR_CUDA;
  kernel<<<pl.ctas, kPagedWarps * 32, pl.smem, st>>>(a);
  FIX_PAGED_TRY(launch_status());
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.join_by_unit ? a.units : a.nworkers,
                     (a.hpb + a.heads_per_cta - 1) / a.heads_per_cta);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, paged_join_kernel<DV, SCALAR>, a);
  return launch_status();
}

template <int DV>
static fix_status paged_launch_dv(const PagedArgs& a, const PagedPlan& pl, bool scalar,
                                  cudaStream_t st) {
  if (scalar)
    return pl.nt == 1 ? paged_launch<DV, 1, true>(a, pl, st) : paged_launch<DV, 2, true>(a, pl, st);
  return pl.nt == 1 ? paged_launch<DV, 1, false>(a, pl, st) : paged_launch<DV, 2, false>(a, pl, st);
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
  a.slots = static_cast<float*>(workspace);
  a.units = pl.units;
  // few units: a CTA per unit and head, all its warps on the head's pieces;
  // many: each unit has few pieces, a CTA's warps take a head each
  a.join_by_unit = pl.units <= pl.workers;
  a.heads_per_cta = a.join_by_unit ? 1 : pl.hpb > 4 ? 8 : pl.hpb > 2 ? 4 : pl.hpb;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (d.Dv) {
    case 16: return paged_launch_dv<16>(a, pl, d.scalar_gate, st);
    case 32: return paged_launch_dv<32>(a, pl, d.scalar_gate, st);
    case 64: return paged_launch_dv<64>(a, pl, d.scalar_gate, st);
    default: return paged_launch_dv<128>(a, pl, d.scalar_gate, st);
  }
}
