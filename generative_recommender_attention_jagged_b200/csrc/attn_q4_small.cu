// HSTU attention of a few new rows a user over the 4-bit paged cache.
//
//   s_ij = alpha ks_j sum_e q_ie (c_je - kz_j) + rab_pos[..] + rab_ts[..]
//   o_i  = sum_j SiLU(s_ij) vs_j (c'_j - vz_j)
//
// with ks, kz (vs, vz) the scale and zero point of key (value) row j and c its
// codes.  Incremental serving: one or a few new actions of each user against a
// history of thousands of cached tokens, so every cached byte is read once for
// a handful of rows (136 bytes a token and head at d = 128).  With a quarter of
// bf16's bytes to read, widening the codes counts as much as reading them: 64
// users of 1000 to 8192 keys, 4 heads of 128, one row each take 80 us (2.2 TB/s),
// with 45% of the issue slots used.  What follows from that:
//
//   - A CTA takes one (user, head, part of the cached keys); its warps walk
//     tiles of 32 keys by themselves, with no block-wide barrier.  Each warp
//     keeps a ring of tiles in shared memory filled by cp.async (codes, scale
//     words and timestamps), so that about 10 KB a warp are in flight while it
//     computes.
//   - The products run on mma.sync with the keys as M and the rows as N (8
//     rows, or 16 in two N tiles): S^T = K Q^T, then O^T = V^T P^T.  With few
//     rows the 128-row tiles of tcgen05 would be mostly empty, and the codes
//     would have to be widened into shared memory; here they are widened in
//     registers, in the layout the instruction wants: a thread reads 16 bytes
//     of a key row as they lie (32 codes), and (w >> 4 i) & 0x000F000F with the
//     exponent of 128 in front is already the bf16 pair 128 + code of two
//     neighbouring dimensions.  For V^T the pair has to be two keys of one
//     dimension: one byte permute of two keys' words makes four such pairs.
//   - The order of the dimensions (of the keys) inside a product is free as
//     long as both operands agree, so every load is contiguous and no operand
//     is shuffled.
//   - Between the products the scores go through shared memory once, to one key
//     a lane: the key's scale, time and position are then one load each and only
//     the rows there are cost anything (a request with one new action has one of
//     eight); the weights come back by a transposing ldmatrix.
//   - For K the 128 + kz of each element is taken off after the product, as
//     (128 + kz) sum_e q_ie in fp32.  What cancels is of the size of 128 sum_e |q_ie|,
//     whatever s is, so the error of s is absolute: up to 2^-11 alpha ks_j sum_e |q_ie|
//     (D / 16 sums of 16 products, each to 2^-22 of them).  fp32 calls, which need
//     more, subtract first.  For V it is taken off before the product (the sum runs
//     over thousands of keys), one packed subtraction.
//   - Weights: SiLU in fp32, sums in fp32.  a_ij vs_j goes into the second product in
//     fp16, with codes - vz (integers) in fp16 too: a power of two for each row and
//     tile of 32 keys brings its largest weight to 2^14 .. 2^15, so that fp16's range is
//     no limit, and is taken back where the tile's O^T joins the running sum.  The
//     rounding of 2^-11 is not seen in y (1.64e-3 of it with one head, where 1.63e-3 is
//     its own rounding).  One bf16 term, 2^-8, is: what LayerNorm leaves of o is as
//     noisy as the weights however many keys there are (up to 3.2e-3), and only means
//     that differ from head to head hide it.  64 users of 1000 to 8192 keys, 1 row: 80 us
//     in fp16, 77 with one bf16 term, 90 with two.
//   - fp32 calls split each row element and each weight into three bf16 terms
//     (8 + 8 + 8 bits: what is left is below 2^-24 of it) and run each product
//     three times, smallest terms first; code - zero is exact as it is, and every
//     tile's O^T is summed from zero and added to the running sum in fp32, since
//     the tensor core's own sums are not rounded to nearest.
//
// Users with more rows than a pass takes (fp32, or a head size that the tcgen05 kernel
// does not take, or one such user among others) have a CTA for each 8 or 16 of them.
//
// The new rows' own keys are a few: each warp takes rows and does the allowed
// pairs in fp32 FMAs, so that what a mask hides is never touched.  The CTA that
// finishes a tile of rows last (a counter in the workspace) adds the parts in order,
// normalises and gates: one launch behind the plan (plan_q4_kernel), which lists the tiles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cfloat>

#include "device_common.cuh"
#include "hstu_internal.h"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 2;       // key tiles a warp has in shared memory
constexpr int kKeys = 32;      // keys of a tile
constexpr int kMinPart = 256;  // keys below which a part is not split further

template <int D>
struct Stage {
  static constexpr int kRowBytes = D / 2;
  static constexpr int kVRow = D / 2 + 16;  // padded: the V reads of a warp then hit 32 different banks
  uint8_t k[kKeys * kRowBytes];
  uint8_t v[kKeys * kVRow];
  uint32_t km[kKeys];
  uint32_t vm[kKeys];
  long long ts[kKeys];
};

// Bytes of a key's row in the exchange buffer: fp32 scores, then over them the
// weights in bf16 (three terms of 16 bytes per 8 rows for fp32 calls).
template <typename T, int NQ>
constexpr int kXRow = (sizeof(T) == 4 ? 48 : 32) * NQ;

template <typename T, int D, int NQ>
struct __align__(16) SmallSmem {
  union {
    Stage<D> ring[kWarps][kRing];
    float red[kWarps][8 * NQ][D];
  };
  float self[8 * NQ][D];  // the new rows' sums over the new keys
  uint8_t xs[kWarps][kKeys][kXRow<T, NQ>];
  float qsum[8 * NQ];     // sum_e q_ie
  long long t_i[8 * NQ];
  int rp[8 * NQ];         // rab_pos index of key position 0
  long long thr[kMaxBuckets];
  float rts[kMaxBuckets];
  uint4 oct[32];
  int last;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// (zero where off)
__device__ __forceinline__ void cp4(void* dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with fp16 operands
__device__ __forceinline__ void mma16816_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// fp16 pair 1024 + nibble i of each 16-bit half
__device__ __forceinline__ uint32_t widen_half(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
}

// The power of two that brings a row's largest weight of a tile to 2^14 .. 2^15 (fp16 holds 65504; smaller weights keep
// their 11 bits down to 2^-28 of it), and its inverse, both normal numbers.  NaN weights do not count.
__device__ __forceinline__ float half_scale(float weight) {
  float m;
  asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(weight));
  const uint32_t e = __float_as_uint(m) & 0x7F800000u;
  return __uint_as_float(min(max(0x7F000000u + (14u << 23) - e, 0x00800000u), 0x7E800000u));
}
__device__ __forceinline__ float inverse_scale(float scale) {
  return __uint_as_float(0x7F000000u - __float_as_uint(scale));
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t add_bf16x2_(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// bf16 pair 128 + nibble i of each 16-bit half
__device__ __forceinline__ uint32_t widen(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u; }

template <typename T>
__device__ __forceinline__ float silu_of(float s) {
  if constexpr (sizeof(T) == 4) return s / (1.f + expf(-s));
  else return __fdividef(s, 1.f + __expf(-s));  // a few ulp, far below the weight's rounding to bf16
}

__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// x as N bf16 terms, largest first; their sum is x to 2^(-8 N) |x| (each term takes 8 bits)
template <int N>
__device__ __forceinline__ void split_bf16(float x, float (&y)[N]) {
#pragma unroll
  for (int p = 0; p < N; ++p) {
    y[p] = __bfloat162float(__float2bfloat16_rn(x));
    // an infinity or NaN (or what rounds to one) stays in the first term
    x = fabsf(y[p]) <= FLT_MAX ? x - y[p] : 0.f;
  }
}

__device__ __noinline__ int bucket_slow(const long long* thr, long long dt) { return bucket_of_dt(thr, dt); }

// rab_ts of the bucket of t_i - t_j: the octave table for differences of 0 .. 2^32 - 2 (the search
// stays out of line, it would be unrolled at every score)
__device__ __forceinline__ float time_bias(const long long* thr, const float* rts, const uint4* oct, long long dt) {
  const unsigned long long x = (unsigned long long)dt + 1;
  return rts[(x >> 32) == 0 && x != 0 ? bucket_oct(oct, (unsigned int)x) : bucket_slow(thr, dt)];
}

__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Keys of one part of a user with L cached tokens, and how many parts it has.
__device__ __forceinline__ int part_keys(int L, int splits) {
  return max(kMinPart, ((L + splits - 1) / splits + kKeys - 1) / kKeys * kKeys);
}

// (four CTAs an SM for one N tile of bf16 rows: 128 registers; three otherwise)
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && NQ == 1 ? 4 : 3)
    attn_q4_small_kernel(const AttnArgs a, const BucketTable tab, int32_t* counters, const int2* row_tiles) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kTerms = kF32 ? 3 : 1;  // terms of a row element, and of a weight (bf16 calls: one, in fp16)
  constexpr int kWords = D / 32;   // words of a K row a thread reads (its quarter of the dimensions)
  constexpr int kSteps = D / 16;   // products of 16 dimensions
  constexpr int kTilesM = D / 16;  // 16-dimension tiles of O^T
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SmallSmem<T, D, NQ>& sm = *reinterpret_cast<SmallSmem<T, D, NQ>*>(smem_raw);
  const int split = blockIdx.x % a.num_splits, head = (int)(blockIdx.x / a.num_splits) % a.H;
  const int tile = (int)(blockIdx.x / a.num_splits) / a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  grid_dependency_wait();
  const int valid = a.hdr->pad[0];
  const int2 item = row_tiles[tile];
  const int u = item.x, r0 = 8 * NQ * item.y;
  if (valid != 1 || u < 0) return;  // a user's lengths do not hold, or no tile
  const int q0 = a.q_offsets[u], rows = a.q_offsets[u + 1] - q0;
  const int L = a.cached_lens[u], n = L + rows;
  const int part = part_keys(L, a.num_splits);
  const int parts = max(1, (L + part - 1) / part);
  if (split >= parts) return;
  const int k_lo = split * part, k_hi = min(L, k_lo + part);
  const int hist = n - (a.num_cand ? a.num_cand[u] : 0);
  const int32_t* table = a.page_table + (size_t)u * a.max_pages;
  const int64_t* ts = a.ts + a.ts_offsets[u];

  // this part's page ids and timestamps (the first part also has the new tokens')
  auto check_keys = [&] {
    for (int x = k_lo / a.page_size + threadIdx.x; x < (k_hi + a.page_size - 1) / a.page_size; x += kThreads) {
      const int pid = table[x];
      if (pid < 0 || pid >= a.num_pages) report_error(a.hdr, kErrPage, u);
    }
    for (int x = threadIdx.x; x < k_hi - k_lo + (split == 0 ? n - L : 0); x += kThreads) {
      const int j = x < k_hi - k_lo ? k_lo + x : L + x - (k_hi - k_lo);
      const long long t = ts[j];
      if (t > kTsLimit || t < -kTsLimit || (j > 0 && t < ts[j - 1])) report_error(a.hdr, kErrUnsorted, u);
    }
  };
  const bool checks = head == 0 && r0 == 0;
  if (rows == 0) {
    if (checks) check_keys();
    return;
  }

  for (int x = threadIdx.x; x < kMaxBuckets; x += kThreads) {
    sm.thr[x] = tab.thr[x];
    sm.rts[x] = x < a.nb ? a.rab_ts[x] : 0.f;
  }
  if (threadIdx.x < 32)
    sm.oct[threadIdx.x] = make_uint4(tab.oct[threadIdx.x][0], tab.oct[threadIdx.x][1], tab.oct[threadIdx.x][2],
                                     tab.oct[threadIdx.x][3]);
  __syncthreads();

  const T* q = static_cast<const T*>(a.q);
  const T* kn = static_cast<const T*>(a.k);
  const T* vn = static_cast<const T*>(a.v);
  const uint8_t* kp = static_cast<const uint8_t*>(a.k_pool);
  const uint8_t* vp = static_cast<const uint8_t*>(a.v_pool);
  Stage<D>* ring = sm.ring[warp];
  const int tiles = (k_hi - k_lo + kKeys - 1) / kKeys;
  const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;  // tiles warp, warp + 4, ...

  const int nr = min(8 * NQ, rows - r0);
  // ---- the rows: fragments of Q^T, their sums, times and positions
  uint32_t qf[NQ][kSteps][2][kTerms];
#pragma unroll
  for (int w = 0; w < NQ; ++w) {
    const int r = 8 * w + g;
    const T* qr = q + (size_t)(q0 + r0 + min(r, nr - 1)) * a.qkv_stride + head * D + (D / 4) * t;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float x[4];
      if constexpr (kF32) {
        const float4 f = *reinterpret_cast<const float4*>(qr + 4 * k);
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
      } else {
        const uint2 f = *reinterpret_cast<const uint2*>(qr + 4 * k);
        x[0] = __uint_as_float(f.x << 16), x[1] = __uint_as_float(f.x & 0xFFFF0000u);
        x[2] = __uint_as_float(f.y << 16), x[3] = __uint_as_float(f.y & 0xFFFF0000u);
      }
      s += (x[0] + x[1]) + (x[2] + x[3]);
      if constexpr (kF32) {
        float y[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16(x[e], y[e]);
#pragma unroll
        for (int p = 0; p < kTerms; ++p) {
          qf[w][k][0][p] = pack_bf16x2(y[0][p], y[1][p]);
          qf[w][k][1][p] = pack_bf16x2(y[2][p], y[3][p]);
        }
      } else {
        qf[w][k][0][0] = pack_bf16x2(x[0], x[1]);
        qf[w][k][1][0] = pack_bf16x2(x[2], x[3]);
      }
    }
    s += __shfl_xor_sync(~0u, s, 1);
    s += __shfl_xor_sync(~0u, s, 2);
    if (warp == 0 && t == 0) {  // what the weights need of row r
      const int i = L + r0 + min(r, nr - 1);
      sm.qsum[r] = s;
      sm.t_i[r] = ts[i];
      sm.rp[r] = min(i, hist) + a.n_max - 1;
    }
  }
  __syncthreads();
  float o[NQ][kTilesM][4];
#pragma unroll
  for (int w = 0; w < NQ; ++w)
#pragma unroll
    for (int m = 0; m < kTilesM; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[w][m][e] = 0.f;

  // page id of this lane's key of the warp's m-th tile (loaded one tile ahead of its copy)
  auto page_of = [&](int m) -> int {
    const int j = k_lo + (warp + m * kWarps) * kKeys + lane;
    return m < mine && j < k_hi ? table[page_index(a, j)] : 0;
  };
  auto fetch = [&](int m, int pid) {
    if (m < mine) {
      const int j = k_lo + (warp + m * kWarps) * kKeys + lane;
      // past the part's end and for a page id out of range (reported by check_keys) the codes are those of
      // the pool's first row, under scales and zero points of 0
      const bool on = j < k_hi && (unsigned)pid < (unsigned)a.num_pages;
      Stage<D>& st = ring[m % kRing];
      // (the pool has fewer than 2^32 rows: attn_q4_small_supported)
      const uint32_t slot =
          on ? ((uint32_t)pid * a.H + head) * a.page_size + (j - page_index(a, j) * a.page_size) : 0;
      constexpr int kPieces = D / 32;  // 16-byte pieces of a row
      const uint32_t k_to = smem_u32(st.k), v_to = smem_u32(st.v);
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        const int c = 32 * x + lane, row = c / kPieces, piece = c % kPieces;
        const uint32_t s = __shfl_sync(~0u, slot, row);
        cp16(k_to + row * (D / 2) + piece * 16, kp + piece * 16 + (size_t)s * (D / 2));
        cp16(v_to + row * Stage<D>::kVRow + piece * 16, vp + piece * 16 + (size_t)s * (D / 2));
      }
      cp4(&st.km[lane], a.k_scales + slot, on);
      cp4(&st.vm[lane], a.v_scales + slot, on);
      cp8(&st.ts[lane], ts + min(j, n - 1));
    }
    cp_commit();
  };

  int pid = page_of(0);
#pragma unroll
  for (int m = 0; m < kRing - 1; ++m) {
    const int next = page_of(m + 1);
    fetch(m, pid);
    pid = next;
  }
  for (int m = 0; m < mine; ++m) {
    {
      const int next = page_of(m + kRing);
      fetch(m + kRing - 1, pid);
      pid = next;
    }
    cp_wait<kRing - 1>();
    __syncwarp();
    const Stage<D>& st = ring[m % kRing];
    const int j0 = k_lo + (warp + m * kWarps) * kKeys;
    uint8_t(&xs)[kKeys][kXRow<T, NQ>] = sm.xs[warp];
    // ---- S^T = (128 + codes) Q^T (fp32: (codes - kz) Q^T), 16 keys at a time
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float s[NQ][4];
#pragma unroll
      for (int w = 0; w < NQ; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[w][e] = 0.f;
      uint32_t ka[kWords], kb[kWords];
      const uint8_t* krow = st.k + (16 * half + g) * (D / 2) + t * (D / 8);
      if constexpr (D == 128) {
        *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(krow);
        *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(krow + 8 * (D / 2));
      } else {
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
          ka[c] = reinterpret_cast<const uint32_t*>(krow)[c];
          kb[c] = reinterpret_cast<const uint32_t*>(krow + 8 * (D / 2))[c];
        }
      }
      uint32_t za = 0, zb = 0;
      if constexpr (kF32) {
        const uint32_t ma = st.km[16 * half + g], mb = st.km[16 * half + g + 8];
        za = add_bf16x2_(__byte_perm(ma, ma, 0x3232), 0x43004300u);
        zb = add_bf16x2_(__byte_perm(mb, mb, 0x3232), 0x43004300u);
      }
#pragma unroll
      for (int p = kTerms - 1; p >= 0; --p)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int i = 2 * (k & 1);
          uint32_t a0 = widen(ka[k >> 1], i), a1 = widen(kb[k >> 1], i), a2 = widen(ka[k >> 1], i + 1),
                   a3 = widen(kb[k >> 1], i + 1);
          if constexpr (kF32) {
            a0 = sub_bf16x2(a0, za), a1 = sub_bf16x2(a1, zb), a2 = sub_bf16x2(a2, za), a3 = sub_bf16x2(a3, zb);
          }
#pragma unroll
          for (int w = 0; w < NQ; ++w) mma16816(s[w], a0, a1, a2, a3, qf[w][k][0][p], qf[w][k][1][p]);
        }
#pragma unroll
      for (int w = 0; w < NQ; ++w)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float2*>(xs[16 * half + 8 * x + g] + 4 * (8 * w + 2 * t)) =
              make_float2(s[w][2 * x], s[w][2 * x + 1]);
    }
    __syncwarp();
    // ---- weights: lane = key, only the rows there are
    uint32_t p[kTerms][NQ][4];  // B fragments of P^T: keys 8 x .. 8 x + 7 against rows 8 w .. 8 w + 7
    float back[NQ][2];          // fp16 weights: what undoes the scales of rows 8 w + 2 t, 8 w + 2 t + 1
#pragma unroll
    for (int w = 0; w < NQ; ++w) back[w][0] = back[w][1] = 0.f;
    {
      const int j = j0 + lane;
      const uint32_t km = st.km[lane], vm = st.vm[lane];
      const float ks = a.alpha * meta_scale(km), kz = kF32 ? 0.f : -(128.f + meta_zero(km));
      const float vs = meta_scale(vm);
      const long long tj = st.ts[lane];
      const float* bias_of = a.rab_pos - min(j, L);
      const float* sc_of = reinterpret_cast<const float*>(xs[lane]);
      float pos_bias[8 * NQ];  // all rows' loads on the way before the first is used
#pragma unroll
      for (int r = 0; r < 8 * NQ; ++r) {
        if (r >= nr) break;
        pos_bias[r] = __ldg(bias_of + sm.rp[r]);
      }
      uint32_t pk[kTerms][4 * NQ];
#pragma unroll
      for (int r = 0; r < 8 * NQ; r += 2) {
        float wt[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (r + e < nr) {
            const float bias = pos_bias[r + e] + time_bias(sm.thr, sm.rts, sm.oct, sm.t_i[r + e] - tj);
            const float raw = kF32 ? sc_of[r + e] : fmaf(kz, sm.qsum[r + e], sc_of[r + e]);
            wt[e] = j < k_hi ? silu_of<T>(fmaf(ks, raw, bias)) * vs : 0.f;
            if constexpr (!kF32) {
              const float scale = half_scale(wt[e]);
              wt[e] *= scale;
              if (t == ((r / 2) & 3)) back[r / 8][e] = inverse_scale(scale);
            }
          }
        if constexpr (kF32) {
          float y[2][kTerms];
          split_bf16(wt[0], y[0]);
          split_bf16(wt[1], y[1]);
#pragma unroll
          for (int x = 0; x < kTerms; ++x) pk[x][r / 2] = pack_bf16x2(y[0][x], y[1][x]);
        } else {
          pk[0][r / 2] = pack_half2(wt[0], wt[1]);
        }
      }
      // the lane's weights over its own scores, then transposed by ldmatrix
#pragma unroll
      for (int x = 0; x < kTerms; ++x)
#pragma unroll
        for (int w = 0; w < NQ; ++w)
          *reinterpret_cast<uint4*>(xs[lane] + 16 * (NQ * x + w)) =
              make_uint4(pk[x][4 * w], pk[x][4 * w + 1], pk[x][4 * w + 2], pk[x][4 * w + 3]);
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kTerms; ++x)
#pragma unroll
        for (int w = 0; w < NQ; ++w)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(p[x][w][0]), "=r"(p[x][w][1]), "=r"(p[x][w][2]), "=r"(p[x][w][3])
                       : "r"(smem_u32(xs[lane] + 16 * (NQ * x + w)))
                       : "memory");
    }
    // ---- O^T += (codes' - vz) P^T
    // 16-bit pieces (4 codes) of a V row a thread reads: its eighth of the dimensions
    constexpr int kHalves = D / 32;
    // [16 keys][lo, hi]: keys 2 t, 2 t + 1 (lo) or 2 t + 8, 2 t + 9 (hi) side by side
    uint32_t vh[2][2][kHalves];
    uint32_t vz[2][2];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = 16 * half + 8 * x + 2 * t;
        const uint8_t* va = st.v + key * Stage<D>::kVRow + g * (D / 16);
        const uint8_t* vb = va + Stage<D>::kVRow;
        if constexpr (kHalves % 2 == 0) {
          uint32_t wa[kHalves / 2], wb[kHalves / 2];
          if constexpr (D == 128) {
            *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(va);
            *reinterpret_cast<uint2*>(wb) = *reinterpret_cast<const uint2*>(vb);
          } else {
            wa[0] = *reinterpret_cast<const uint32_t*>(va);
            wb[0] = *reinterpret_cast<const uint32_t*>(vb);
          }
#pragma unroll
          for (int c = 0; c < kHalves / 2; ++c) {
            vh[half][x][2 * c] = __byte_perm(wa[c], wb[c], 0x5410);
            vh[half][x][2 * c + 1] = __byte_perm(wa[c], wb[c], 0x7632);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kHalves; ++c)
            vh[half][x][c] = (uint32_t)reinterpret_cast<const uint16_t*>(va)[c] |
                             ((uint32_t)reinterpret_cast<const uint16_t*>(vb)[c] << 16);
        }
        vz[half][x] = add_bf16x2_(__byte_perm(st.vm[key], st.vm[key + 1], 0x7632), 0x43004300u);
        if constexpr (!kF32) vz[half][x] = (vz[half][x] & 0x000F000Fu) | 0x64006400u;  // 128 + zero -> 1024 + zero
      }
    // row g of tile m is the thread's nibble m of its D / 8, row g + 8 its nibble m + D / 16
#pragma unroll
    for (int m2 = 0; m2 < kTilesM; ++m2) {
      constexpr int kSecond = D / 16;
      float f[NQ][4];
#pragma unroll
      for (int w = 0; w < NQ; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[w][e] = 0.f;  // a tile is summed by itself
      uint32_t av[2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        auto value = [&](int x, int m) {
          return kF32 ? sub_bf16x2(widen(vh[half][x][m >> 2], m & 3), vz[half][x])
                      : sub_half2(widen_half(vh[half][x][m >> 2], m & 3), vz[half][x]);
        };
        av[half][0] = value(0, m2);
        av[half][1] = value(0, m2 + kSecond);
        av[half][2] = value(1, m2);
        av[half][3] = value(1, m2 + kSecond);
      }
#pragma unroll
      for (int x = kTerms - 1; x >= 0; --x)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int w = 0; w < NQ; ++w)
            (kF32 ? mma16816 : mma16816_half)(f[w], av[half][0], av[half][1], av[half][2], av[half][3],
                                               p[x][w][2 * half], p[x][w][2 * half + 1]);
#pragma unroll
      for (int w = 0; w < NQ; ++w) {
        if constexpr (!kF32) {
          const uint64_t back2 = pack_pair(back[w][0], back[w][1]);
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            unpack_pair(fma_pair(pack_pair(f[w][e], f[w][e + 1]), back2, pack_pair(o[w][m2][e], o[w][m2][e + 1])),
                        o[w][m2][e], o[w][m2][e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[w][m2][e] += f[w][e];
        }
      }
    }
    __syncwarp();  // the tile's slot may be filled again
  }
  cp_wait<0>();

  // ---- the new rows' own keys: row r by worker r of the user's parts x warps, fp32
  for (int x = threadIdx.x; x < 8 * NQ * D; x += kThreads) (&sm.self[0][0])[x] = 0.f;
  __syncthreads();
  for (int r = split + parts * warp; r < nr; r += parts * kWarps) {
    constexpr int kPer = D / 32;
    const int i = L + r0 + r;
    const size_t row = (size_t)(q0 + r0 + r) * a.qkv_stride + head * D + kPer * lane;
    float qv[kPer], acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      qv[e] = as_f(q[row + e]);
      acc[e] = 0.f;
    }
    const bool cand = i >= hist;
    const int j_end = cand ? hist : i + 1;
    const long long ti = ts[i];
    // its keys L .. j_end - 1, and a candidate's own; four at a time, so that their loads overlap
    const int count = j_end - L + (cand ? 1 : 0);
#pragma unroll 1
    for (int c0 = 0; c0 < count; c0 += 4) {
      float dot[4], bias[4], vv[4][kPer];
      long long tj[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int x = min(c0 + c, count - 1), j = L + x < j_end ? L + x : i;
        const size_t at = (size_t)(q0 + j - L) * a.qkv_stride + head * D + kPer * lane;
        dot[c] = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          dot[c] = fmaf(qv[e], as_f(kn[at + e]), dot[c]);
          vv[c][e] = as_f(vn[at + e]);
        }
        bias[c] = a.rab_pos[min(i, hist) - min(j, hist) + a.n_max - 1];
        tj[c] = ts[j];
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) dot[c] += __shfl_xor_sync(~0u, dot[c], o);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c0 + c < count) {  // (nothing of a key past the last is used)
          const float wt =
              silu_of<T>(a.alpha * dot[c] + bias[c] + time_bias(sm.thr, sm.rts, sm.oct, ti - tj[c]));
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(wt, vv[c][e], acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) sm.self[r][kPer * lane + e] = acc[e];
  }
  // ---- the warps' sums meet in shared memory (the ring is idle) and go out in order
#pragma unroll
  for (int w = 0; w < NQ; ++w)
#pragma unroll
    for (int m = 0; m < kTilesM; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int idx = m + (e >> 1) * (D / 16), half = idx >> 2, nib = idx & 3;
        // 16-bit piece (D / 32) g + half of the row: elements 0, 2, 4, 6 of its word, or 1, 3, 5, 7
        const int piece = (D / 32) * g + half, dim = 8 * (piece >> 1) + 2 * nib + (piece & 1);
        sm.red[warp][8 * w + 2 * t + (e & 1)][dim] = o[w][m][e];
      }
  __syncthreads();
  float* out = a.o_ws + (((size_t)split * a.T_q + q0 + r0) * a.H + head) * D;
  for (int x = threadIdx.x; x < nr * D; x += kThreads) {
    const int r = x / D, e = x % D;
    float s = sm.self[r][e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sm.red[w][r][e];
    out[(size_t)r * a.H * D + e] = s;
  }
  __syncthreads();

  if (checks) check_keys();  // (the keys' own loads have them in the caches by now)

  // ---- the last CTA of these rows adds the parts, normalises and gates
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) sm.last = atomicAdd(&counters[tile], 1) == a.H * parts - 1;
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  const int HD = a.H * D;  // a multiple of 32, at most 1024
  const float inv_n = 1.f / (float)a.n_max;
  static_assert(sizeof(sm.ring) >= kWarps * 1024 * sizeof(float));
  float* sums = reinterpret_cast<float*>(sm.ring);  // [kWarps][HD]
  // four rows at a time: all threads add their parts (eight loads each on the way), then a warp finishes a row
#pragma unroll 1
  for (int first = r0; first < r0 + nr; first += kWarps) {
    const int there = min(kWarps, r0 + nr - first);
    const size_t row = q0 + first + min(warp, there - 1);
    float2 x[16], uv[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      uv[k] = make_float2(0.f, 0.f);
      if (!a.out_raw && 64 * k + 2 * lane < HD) {  // the gate on its way with the sums
        const T* uu = static_cast<const T*>(a.u) + row * a.u_stride + 64 * k + 2 * lane;
        uv[k] = make_float2(as_f(uu[0]), as_f(uu[1]));
      }
    }
#pragma unroll 1
    for (int e = 4 * threadIdx.x; e < there * HD; e += 4 * kThreads) {
      const float* src = a.o_ws + (size_t)(q0 + first) * HD + e;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int part0 = 0; part0 < parts; part0 += 8) {
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = part0 + i < parts ? __ldcg(reinterpret_cast<const float4*>(src + (size_t)(part0 + i) * a.T_q * HD))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s.x += y[i].x;
          s.y += y[i].y;
          s.z += y[i].z;
          s.w += y[i].w;
        }
      }
      *reinterpret_cast<float4*>(sums + e) = make_float4(s.x * inv_n, s.y * inv_n, s.z * inv_n, s.w * inv_n);
    }
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float* src = sums + min(warp, there - 1) * HD + 64 * k + 2 * lane;
      x[k] = 64 * k + 2 * lane < HD ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
      sum += x[k].x + x[k].y;
    }
    __syncthreads();  // (the next rows' sums go over these)
    if (warp >= there) continue;
    if (a.out_raw) {
      float* out = static_cast<float*>(a.out) + row * HD + 2 * lane;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (64 * k + 2 * lane < HD) *reinterpret_cast<float2*>(out + 64 * k) = x[k];
      continue;
    }
    const float mean = warp_add(sum) / (float)HD;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (64 * k + 2 * lane < HD) {
        const float c0 = x[k].x - mean, c1 = x[k].y - mean;
        sq = fmaf(c0, c0, fmaf(c1, c1, sq));
      }
    const float rstd = rsqrtf(warp_add(sq) / (float)HD + a.ln_eps);
    T* out = static_cast<T*>(a.out) + row * HD + 2 * lane;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (64 * k + 2 * lane < HD) {
        const int e = 64 * k + 2 * lane;
        const float2 ga = a.ln_gamma ? *reinterpret_cast<const float2*>(a.ln_gamma + e) : make_float2(1.f, 1.f);
        const float2 be = a.ln_beta ? *reinterpret_cast<const float2*>(a.ln_beta + e) : make_float2(0.f, 0.f);
        const float y0 = ((x[k].x - mean) * rstd * ga.x + be.x) * uv[k].x;
        const float y1 = ((x[k].y - mean) * rstd * ga.y + be.y) * uv[k].y;
        if constexpr (kF32) *reinterpret_cast<float2*>(out + 64 * k) = make_float2(y0, y1);
        else *reinterpret_cast<__nv_bfloat162*>(out + 64 * k) = __floats2bfloat162_rn(y0, y1);
      }
  }
}

template <typename T, int D, int NQ>
cudaError_t launch(const AttnArgs& a, const BucketTable& thr, int32_t* counters, const int2* tiles, int n_tiles,
                   cudaStream_t s) {
  constexpr size_t smem = sizeof(SmallSmem<T, D, NQ>);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    const cudaError_t e = cudaFuncSetAttribute(attn_q4_small_kernel<T, D, NQ>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  const long long ctas = (long long)n_tiles * a.H * a.num_splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_dependent(attn_q4_small_kernel<T, D, NQ>, dim3((unsigned)ctas), dim3(kThreads), smem, s, a, thr,
                          counters, tiles);
}

template <typename T, int NQ>
cudaError_t launch_d(const AttnArgs& a, const BucketTable& thr, int32_t* counters, const int2* tiles, int n_tiles,
                     cudaStream_t s) {
  switch (a.d) {
    case 32: return launch<T, 32, NQ>(a, thr, counters, tiles, n_tiles, s);
    case 64: return launch<T, 64, NQ>(a, thr, counters, tiles, n_tiles, s);
    case 96: return launch<T, 96, sizeof(T) == 4 ? 1 : NQ>(a, thr, counters, tiles, n_tiles, s);
    default: return launch<T, 128, 1>(a, thr, counters, tiles, n_tiles, s);
  }
}

}  // namespace

bool attn_q4_small_supported(int head_dim, long long pool_rows) {
  return head_dim <= 128 && head_dim % 32 == 0 && pool_rows < 0xFFFFFFFFll;
}

cudaError_t launch_attn_q4_small(const AttnArgs& a, const BucketTable& thr, int32_t* counters, const int2* tiles,
                                 int n_tiles, int rows, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (a.in_bf16)
    return rows == 8 ? launch_d<bf16, 1>(a, thr, counters, tiles, n_tiles, s)
                     : launch_d<bf16, 2>(a, thr, counters, tiles, n_tiles, s);
  return rows == 8 ? launch_d<float, 1>(a, thr, counters, tiles, n_tiles, s)
                   : launch_d<float, 2>(a, thr, counters, tiles, n_tiles, s);
}

}  // namespace hstu
