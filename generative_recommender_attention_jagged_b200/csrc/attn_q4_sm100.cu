// HSTU attention over the 4-bit paged cache on the tcgen05 tensor cores: many
// new rows a user (requests with their candidates, ranking, prompts in parts).
//
// The arithmetic of attn_sm100_single.cu (one 128-row query tile per CTA,
// S = Q K^T and O += P V in tensor memory, bias + SiLU in registers, exact time
// buckets) with keys and values in 4 bits:
//
//   s_ij = alpha ks_j (q_i . (c_j - kz_j)) + bias,   o_i = sum_j (SiLU(s_ij) vs_j) (c'_j - vz_j)
//
// The operands of both products are the integers code - zero, exact in bf16; the
// scale of a key is the factor of its column of S (where alpha stood), the scale
// of a value a factor of its column of P.
//
// With 128 rows against a key tile the step is bound by instruction issue and by the
// latencies of its chain (S, SiLU, P), not by the cache's bytes (16 KB a tile).  16 users
// of 2048 to 4096 keys with 512 candidates, 4 heads: 173 us with the plan and the epilogue,
// 300 TFLOP/s, 59% of the issue slots used (75% while a block is in its loop); 8 users of
// 6144 to 8192 keys with 128 rows: 70 us.
//
//   - eight elementwise warps (two 32-key chunks of each tile each) turn S(t) into P(t).
//     S is double-buffered in tensor memory, so the tensor core does O += P(t - 1) V(t - 1)
//     and S(t + 1) meanwhile.
//   - eight widening warps turn the codes of K(t + 2), V(t + 2) into the 128B-swizzled
//     bf16 tiles the tensor core reads.  Each thread copies its own 16 bytes of two K and
//     two V rows (cp.async) into places of its own two tiles ahead, so nothing is handed
//     over; four lanes a row (64 contiguous bytes).  A tile takes 2.2 us; with one set of
//     sixteen warps doing both in turn it took 2.9: every warp waits for the same barriers
//     at the same time.
//   - they also look the tiles' pages, scales and timestamps up, for two tiles at once (KeyInfo,
//     8 stages: page ids, scales and codes each two tiles ahead of the next); one more warp
//     builds the position window (2 stages), one issues the MMAs.
//
// Weights: in fp32, then as two bf16 terms, of which the second takes the other half of the
// score's columns in tensor memory, with a GEMM each.  What LayerNorm leaves of o is as noisy
// as the weights however many keys there are, and only means that differ from head to head
// hide it: with one head the error of y is 1.63e-3 so (its own rounding), 2.3e-3 with one
// term (up to 1.8 times its own rounding in calls of few rows) and 4.0e-3 with the packed
// bf16 arithmetic of attn_sm100_single.cu.  16 x 512 candidates take 173 us, 166 and 156; 8 x
// 128 rows 70, 68 and 65.  The position bias is in bf16 (as there), and where a row's 32 keys
// lie in more than one time bucket the time bias and the sum of the two are (one packed
// addition instead of a copy of the weights' code for each mode); in one bucket the time bias
// is added in fp32.
//
// Tiles of new tokens (bf16 rows) take the same path without widening.  A value
// row that is not finite is stored as zeros and its scale set to NaN: the mask is
// applied to the finished weight, so rows that may not see the key stay finite.
// A CTA looks at the page ids it uses and, for head 0, at the order of the timestamps (users without
// new rows, which have no CTA, are checked for their lengths only).  Every wait is bounded.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>

#include "attn_common.cuh"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr int kEwWarps = 8;               // 2 warpgroups: two 32-key chunks of every key tile each
constexpr int kWideWarps = 8;             // 16 key rows of every tile each
constexpr int kWideThreads = 32 * kWideWarps;
constexpr int kMmaWarp = kEwWarps + kWideWarps;  // MMA issuer, TMEM owner, Q
constexpr int kWinWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 2);
constexpr int kKeyStages = 8;
constexpr int kWinStages = 2;
constexpr int kTailTiles = 4;             // what a user's last tiles cost beyond the others, in tiles
constexpr uint32_t kTmemCols = 512;       // S0 [0,128) S1 [128,256) O [256,384)

// What the elementwise warps need of a tile's keys.
struct KeyInfo {
  long long ts[kTile];    // timestamps (the last one repeated past the tile's width)
  float ks[kTile];        // alpha / 2 times the scale of the key (new tokens: alpha / 2); 0 past the width
  float vs[kTile];        // scale of the value (new tokens: 1); 0 past the width
};
struct Window {
  uint4 win[kWinChunks][8];
};

struct __align__(1024) SmemQ4 {
  uint8_t q[kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
  uint4 codes[2][2][2][kWideThreads];  // [stage][K, V][row of the thread]: each thread's 16 bytes
  KeyInfo key[kKeyStages];
  Window win[kWinStages];
  long long thr[kMaxBuckets];
  float rab_ts_half[kMaxBuckets];
  uint4 oct[32];
  uint32_t win_rs[kWinLoads * 16];
  uint64_t bar_q;
  uint64_t bar_key_full[kKeyStages];   // widening warps
  uint64_t bar_key_empty[kKeyStages];  // elementwise warps
  uint64_t bar_win_full[kWinStages];   // the window warp (which has seen the tile's KeyInfo)
  uint64_t bar_win_empty[kWinStages];  // elementwise warps
  uint64_t bar_s_full[2];  // S buffer b written: the K stage that it read is free
  uint64_t bar_p_full[2];  // P in buffer b written (elementwise warps)
  uint64_t bar_k_full[2];  // widening warps
  uint64_t bar_v_full[2];
  uint64_t bar_v_empty[2]; // the A.V GEMM that read the stage completed
  uint64_t bar_o_full;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(SmemQ4) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ void cp16_ca(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 8 codes of a word -> 8 bf16 code - zero (zz = the bf16 pair 128 + zero)
__device__ __forceinline__ uint4 widen8(uint32_t w, uint32_t zz) {
  return make_uint4(sub_bf16x2((w & 0x000F000Fu) | 0x43004300u, zz),
                    sub_bf16x2(((w >> 4) & 0x000F000Fu) | 0x43004300u, zz),
                    sub_bf16x2(((w >> 8) & 0x000F000Fu) | 0x43004300u, zz),
                    sub_bf16x2(((w >> 12) & 0x000F000Fu) | 0x43004300u, zz));
}
// a bf16 pair as two fp32
__device__ __forceinline__ uint64_t widen_pair(uint32_t w) {
  return pk2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// whether a bf16 pair holds an infinity or NaN
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Columns at a time.  The size of the loops counts here: a CTA runs six of them at once, and
// with the weights' code repeated for every mode of the time bias (146 KB) the warps waited for
// instructions more than for anything else (4.3 of 12 stall cycles an issue); so the bias is
// added first, in bf16 like the position bias, and one copy of the rest serves all modes.
constexpr int kCols = 32;

__device__ __noinline__ int bucket_slow(const long long* thr, long long x) { return bucket_search(thr, x); }

// Adds the time bias of kCols columns (0.5 * rab_ts of their buckets, see BiasMode; the chunk's
// mode is kBiasConst, kBiasEdge or else one bucket a column) to their position bias pw[k] =
// columns 2 k, 2 k + 1; returns what is left to add to every column.
__device__ __forceinline__ float add_time_bias(int mode, uint32_t (&pw)[kCols / 2], Walk& w, const long long* ts,
                                               int left, float tsb_lo, const long long* thr, const float* rts,
                                               const uint4* oct) {
  if (mode == kBiasConst) return w.tsb;
  if (mode == kBiasEdge) {  // `left` columns are before the edge
    const uint32_t lo = pack_bf16x2(tsb_lo, tsb_lo), hi = pack_bf16x2(w.tsb, w.tsb), mix = pack_bf16x2(tsb_lo, w.tsb);
#pragma unroll
    for (int k = 0; k < kCols / 2; ++k)
      pw[k] = add_bf16x2(pw[k], left >= 2 * k + 2 ? lo : left <= 2 * k ? hi : mix);
    return 0.f;
  }
  int b = 0;
#pragma unroll
  for (int k = 0; k < kCols / 2; ++k) {
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long x = max(w.t_i + 1 - ts[2 * k + e], 1ll);  // later keys only in masked columns
      b = (x >> 32) == 0 ? bucket_oct(oct, (unsigned int)x) : bucket_slow(thr, x);
      v[e] = rts[b];
    }
    pw[k] = add_bf16x2(pw[k], pack_bf16x2(v[0], v[1]));
  }
  // the walk goes on from the last column
  w.b = b;
  w.tlim = w.t_i + 1 - thr[b];
  w.tsb = rts[b];
  return 0.f;
}

// kCols scores of one row -> weights times the values' scales, in two bf16 terms (pairs: the
// first over the biases in pw, the second in lo; a weight that is not finite is NaN).  ks, vs:
// the columns' factors (the same for every lane).
__device__ __forceinline__ void weights_of(const uint32_t (&sr)[kCols], uint32_t (&pw)[kCols / 2],
                                           uint32_t (&lo)[kCols / 2], float tsb, const float* ks, const float* vs) {
  const uint64_t tsb2 = pk2(tsb, tsb), minus_one2 = pk2(-1.f, -1.f);
  float4 ks4 = {}, vs4 = {};
#pragma unroll
  for (int c = 0; c < kCols; c += 2) {
    if (c % 4 == 0) {
      ks4 = *reinterpret_cast<const float4*>(ks + c);
      vs4 = *reinterpret_cast<const float4*>(vs + c);
    }
    const uint64_t f2 = c % 4 == 0 ? pk2(ks4.x, ks4.y) : pk2(ks4.z, ks4.w);
    const uint64_t v2 = c % 4 == 0 ? pk2(vs4.x, vs4.y) : pk2(vs4.z, vs4.w);
    const uint64_t bias2 = add_pair(tsb2, widen_pair(pw[c >> 1]));
    const uint64_t h = fma2(pk2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), f2, bias2);  // half the score
    float h0, h1, p0, p1;
    upk2(h, h0, h1);
    const uint64_t p = mul_pair(fma2(h, pk2(tanh_approx(h0), tanh_approx(h1)), h), v2);
    upk2(p, p0, p1);
    pw[c >> 1] = pack_bf16x2(p0, p1);
    upk2(fma2(widen_pair(pw[c >> 1]), minus_one2, p), p0, p1);
    lo[c >> 1] = pack_bf16x2(p0, p1);
  }
}

// The bounded wait (as mbar_wait: about 2 s, or until another warp gave up), out of line and
// with a hint to sleep up to 20 us a try: a waiting warp that polls takes issue slots from the
// working ones, and inlined at every wait the code came to 9 KB.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort, WsHeader* hdr, int where) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (abort != nullptr && *(volatile int*)abort) return false;
    if (global_timer_ns() - t0 > 2000000000ull) {
      if (abort != nullptr) *(volatile int*)abort = 1;
      report_error(hdr, kErrTimeout, where);
      return false;
    }
  }
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, int* abort, WsHeader* hdr, int where) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, hdr, where);
}
// One lane polls for a warp (32 lanes of 16 waiting warps polling keep the shared-memory pipe from
// the warps that work).  The vote hands its answer to the others; what the barrier published is
// seen by them through the warp barrier behind it.
__device__ __forceinline__ bool warp_agree(bool ok) {
  ok = __all_sync(~0u, ok);
  __syncwarp();
  return ok;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort, WsHeader* hdr, int where) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = lane_wait(bar, parity, abort, hdr, where);
  return warp_agree(ok);
}
// A warp arrives once, when all its lanes are there.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_q4_sm100_kernel(const AttnArgs a, const BucketTable tab, const int2* tiles,
                         const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ uint8_t smem_raw[];
  SmemQ4& sm = aligned_smem<SmemQ4>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.num_splits;
  const int head = (int)(blockIdx.x / a.num_splits) % a.H;
  const int qt = (int)(blockIdx.x / a.num_splits) / a.H;

  grid_dependency_wait();
  const int valid = a.hdr->pad[0];
  const int2 item = tiles[qt];
  const int user = item.x;
  if (valid != 1 || user < 0) return;  // a user's lengths do not hold, or no tile
  const TileGeom g = tile_geom(a, user, item.y);
  // The last tiles (recent keys: a bucket edge every few columns; masked and new ones) take two to
  // three times the others' time: they count for more when the keys are split.
  int tb, te;
  const int tail = g.n_tiles >= 4 * a.num_splits ? kTailTiles : 0;
  split_range(g.n_tiles + tail, split, a.num_splits, tb, te);
  tb = min(tb, g.n_tiles);
  te = min(te, g.n_tiles);
  const int cnt = max(0, te - tb);
  const int prmin = min(g.qs, g.h);
  const int32_t* table = a.page_table + (size_t)user * a.max_pages;
  // head 0 of the user's last tile (it sees every key but the candidates) checks the timestamps on the way
  const bool checks = head == 0 && (item.y + 1) * kTile >= g.n - g.L;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_q, 1);
    for (int s = 0; s < kKeyStages; ++s) {
      mbar_init(&sm.bar_key_full[s], kWideWarps);
      mbar_init(&sm.bar_key_empty[s], kEwWarps);
    }
    for (int s = 0; s < kWinStages; ++s) {
      mbar_init(&sm.bar_win_full[s], 1);
      mbar_init(&sm.bar_win_empty[s], kEwWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.bar_s_full[b], 1);
      mbar_init(&sm.bar_p_full[b], kEwWarps);
      mbar_init(&sm.bar_k_full[b], kWideWarps);
      mbar_init(&sm.bar_v_full[b], kWideWarps);
      mbar_init(&sm.bar_v_empty[b], 1);
    }
    mbar_init(&sm.bar_o_full, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  int* abort_flag = &sm.abort;
  const int row_base = a.q_offsets[user] - g.L;  // row of key position p is row_base + p (p >= L)

  if (warp == kWinWarp) {
    // ------------------------------------------------------------------ position window (see Meta in attn_common.cuh)
    const int n_rab = 2 * a.n_max - 1;
    float mwin[kWinLoads];
    auto load_win = [&](int t) {
      int k0, width;
      key_tile(g, tb + t, k0, width);
      const int g0 = prmin + 255 - k0 + a.n_max - 1;
#pragma unroll
      for (int k = 0; k < kWinLoads; ++k) {
        const int idx = g0 - (lane + 32 * k);
        mwin[k] = (idx >= 0 && idx < n_rab) ? 0.5f * __ldg(a.rab_pos + idx) : 0.f;
      }
    };
    if (cnt > 0) load_win(0);
    for (int t = 0; t < cnt; ++t) {
      const int s = t % kWinStages;
      if (t >= kWinStages && !warp_wait(&sm.bar_win_empty[s], ((t / kWinStages) & 1) ^ 1, abort_flag, a.hdr, 52)) break;
      Window& m = sm.win[s];
      __syncwarp();
      uint16_t* rs16 = reinterpret_cast<uint16_t*>(sm.win_rs);
#pragma unroll
      for (int k = 0; k < kWinLoads; ++k) rs16[lane + 32 * k] = __bfloat16_as_ushort(__float2bfloat16_rn(mwin[k]));
      __syncwarp();
      for (int x = lane; x < kWinChunks * 8; x += 32) {
        const int f = x >> 3, p = x & 7;
        const int wb = 4 * f + (p >> 1);
        const uint32_t sh = 16u * (p & 1);
        const uint32_t x0 = sm.win_rs[wb], x1 = sm.win_rs[wb + 1], x2 = sm.win_rs[wb + 2], x3 = sm.win_rs[wb + 3],
                       x4 = sm.win_rs[wb + 4];
        m.win[f][p] = make_uint4(__funnelshift_r(x0, x1, sh), __funnelshift_r(x1, x2, sh), __funnelshift_r(x2, x3, sh),
                                 __funnelshift_r(x3, x4, sh));
      }
      // whoever sees this barrier has seen the tile's KeyInfo too
      if (!warp_wait(&sm.bar_key_full[t % kKeyStages], (t / kKeyStages) & 1, abort_flag, a.hdr, 52)) break;
      warp_arrive(&sm.bar_win_full[s]);
      if (t + 1 < cnt) load_win(t + 1);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      mbar_arrive_expect_tx(&sm.bar_q, kTileBytes);
      tma_load_3d(sm.q, &tm_q, &sm.bar_q, 0, head, g.qrow0);
      tma_load_3d(sm.q + kHalfBytes, &tm_q, &sm.bar_q, 64, head, g.qrow0);
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(128, 128, 0, 1);
      auto issue_s = [&](int t) {
        const uint32_t q_base = smem_u32(sm.q), k_base = smem_u32(sm.k[t & 1]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
          mma_ss(tmem + (t & 1) * 128, sw128_desc(q_base + off, 16, 1024), sw128_desc(k_base + off, 16, 1024), idesc_qk,
                 kk > 0);
        }
        mma_commit(&sm.bar_s_full[t & 1]);
      };
      auto issue_pv = [&](int t) {
        const uint32_t v_base = smem_u32(sm.v[t & 1]);
#pragma unroll
        for (int term = 1; term >= 0; --term)  // the smaller terms first
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + 256, tmem + (t & 1) * 128 + (kk >> 1) * 32 + 16 * term + (kk & 1) * 8,
                   sw128_desc(v_base + kk * 2048, kHalfBytes, 1024), idesc_pv, (t > 0 || kk > 0 || term == 0));
        mma_commit(&sm.bar_v_empty[t & 1]);
      };
      // Q has landed before anything else uses it (and before the CTA may exit)
      bool ok = lane_wait(&sm.bar_q, 0, abort_flag, a.hdr, 53);
#pragma unroll 1
      for (int t = -2; ok && t < cnt; ++t) {
        if (t >= 0) {
          ok = lane_wait(&sm.bar_p_full[t & 1], (t >> 1) & 1, abort_flag, a.hdr, 55) &&
               lane_wait(&sm.bar_v_full[t & 1], (t >> 1) & 1, abort_flag, a.hdr, 55);
          if (!ok) break;
          tc_fence_after();
          issue_pv(t);
        }
        if (t + 2 < cnt) {  // into the buffer whose P the GEMM above has read
          ok = lane_wait(&sm.bar_k_full[t & 1], ((t + 2) >> 1) & 1, abort_flag, a.hdr, 54);
          if (!ok) break;
          tc_fence_after();
          issue_s(t + 2);
        }
      }
      mma_commit(&sm.bar_o_full);
      lane_wait(&sm.bar_o_full, 0, nullptr, a.hdr, 58);
      lane_wait(&sm.bar_q, 0, nullptr, a.hdr, 58);
    }
    __syncwarp();
  } else if (warp >= kEwWarps) {
    // ------------------------------------------------------------------ widening warps
    const uint8_t* kp = static_cast<const uint8_t*>(a.k_pool);
    const uint8_t* vp = static_cast<const uint8_t*>(a.v_pool);
    const int wt = threadIdx.x - 32 * kEwWarps;
    // rows wr and wr + 8 and a quarter (32 dimensions) of each: four lanes a row.  The 16-byte chunk of
    // dimensions 32 wq + 8 c sits at chunk (4 (wq & 1) + c) ^ (row & 7) of half wq >> 1; threads of the
    // second half take their words in the order c ^ 2, so that the eight lanes of a quarter-warp store to
    // eight different places
    const int wr = 16 * (warp - kEwWarps) + (lane >> 2), wq = lane & 3;
    const int flip = wq & 2;
    uint32_t place[4];  // of the four chunks of row wr in a tile (row wr + 8: 1024 bytes on)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      place[c] = (wq >> 1) * kHalfBytes + wr * 128 + (((4 * (wq & 1) + (c ^ flip)) ^ (wr & 7)) << 4);
    // The warp looks its 16 keys up itself, one a lane and two tiles at once (lanes 0 .. 15: the even
    // one): page id, then scales and time, then the codes, each two tiles ahead of the next.
    const int kc = 16 * (warp - kEwWarps) + (lane & 15), odd = lane >> 4;
    constexpr uint32_t kNoRow = ~0u;  // (a pool has fewer rows: attn_q4_small_supported)
    int pid = 0;
    uint32_t row = kNoRow, row_next = kNoRow;  // pool row of the lane's key
    long long ts = 0, ts_before = 0;
    uint32_t km = 0, vm = 0;
    uint32_t zz0 = 0, zz1 = 0;  // 128 + zero of key | value as bf16: of the tiles being widened and the next two
    bool sorted = true;
    auto in_range = [](long long x) { return x <= kTsLimit && x >= -kTsLimit; };
    auto load_page = [&](int t) {
      int k0, width;
      if (t + odd >= cnt) return;
      key_tile(g, tb + t + odd, k0, width);
      pid = k0 < g.L ? table[page_index(a, k0 + min(kc, width - 1))] : 0;
    };
    auto load_scales = [&](int t) {
      int k0, width;
      row_next = kNoRow;
      if (t + odd >= cnt) return;
      key_tile(g, tb + t + odd, k0, width);
      const int j = k0 + min(kc, width - 1);
      const bool in = pid >= 0 && pid < a.num_pages;
      if (!in) report_error(a.hdr, kErrPage, user);
      const uint32_t r = ((uint32_t)(in ? pid : 0) * a.H + head) * a.page_size +
                         (k0 < g.L ? j - page_index(a, j) * a.page_size : 0);
      km = a.k_scales[r];
      vm = a.v_scales[r];
      ts = a.ts[g.tso + j];
      if (checks) ts_before = j > 0 ? a.ts[g.tso + j - 1] : LLONG_MIN;
      if (in && k0 < g.L && kc < width) row_next = r;
    };
    // the KeyInfo of tiles t and t + 1
    auto announce = [&](int t) {
      int k0, width;
      row = row_next;
      const bool held = row != kNoRow;  // cached
      const int tl = t + odd;
      if (tl < cnt) {
        key_tile(g, tb + tl, k0, width);
        const bool fresh = k0 >= g.L && kc < width;  // a new token
        KeyInfo& key = sm.key[tl % kKeyStages];
        if (checks) sorted &= ts >= ts_before && in_range(ts);
        key.ts[kc] = ts;
        key.ks[kc] = held ? 0.5f * a.alpha * meta_scale(km) : fresh ? 0.5f * a.alpha : 0.f;
        key.vs[kc] = held ? meta_scale(vm) : fresh ? 1.f : 0.f;
      }
      zz1 = held ? pack_bf16x2(128.f + meta_zero(km), 128.f + meta_zero(vm)) : 0x43004300u;  // exact
      __syncwarp();
      if ((lane & 15) == 0 && tl < cnt) mbar_arrive(&sm.bar_key_full[tl % kKeyStages]);
    };
    // tile t's codes into this thread's own places
    auto copy_codes = [&](int t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t r = __shfl_sync(~0u, row, 16 * (t & 1) + (lane >> 2) + 8 * x);
        if (r != kNoRow) {
          cp16_ca(&sm.codes[t & 1][0][x][wt], kp + (size_t)r * 64 + 16 * wq);
          cp16_ca(&sm.codes[t & 1][1][x][wt], vp + (size_t)r * 64 + 16 * wq);
        }
      }
    };
    auto store_rows = [&](uint8_t* tile, int t, int which) {  // which: 0 K, 1 V
      int k0, width;
      key_tile(g, tb + t, k0, width);
      const uint32_t base = smem_u32(tile);
      if (k0 < g.L) {  // cached keys
        uint4 w[2];
        uint32_t zz[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          w[x] = sm.codes[t & 1][which][x][wt];
          const uint32_t z = __shfl_sync(~0u, zz0, 16 * (t & 1) + (lane >> 2) + 8 * x);
          zz[x] = __byte_perm(z, z, which ? 0x3232 : 0x1010);
          // (rows past the width: what an earlier tile left, finite numbers under scales of 0)
          if (flip) w[x] = make_uint4(w[x].z, w[x].w, w[x].x, w[x].y);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) sts_v4(base + place[c] + 1024 * x, widen8(ww[c], zz[x]));
        }
      } else {  // new tokens: bf16 rows as they are (zeros past the width)
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int r = wr + 8 * x;
          const bool on = r < width;
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(which ? a.v : a.k) +
                                                            (size_t)(row_base + k0 + (on ? r : 0)) * a.qkv_stride +
                                                            head * kHeadDim + 32 * wq);
          uint4 w[4];
          bool bad = false;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = on ? src[c ^ flip] : make_uint4(0, 0, 0, 0);
            bad |= not_finite(w[c].x) | not_finite(w[c].y) | not_finite(w[c].z) | not_finite(w[c].w);
          }
          if (which) {  // a value row that is not finite: zeros, and a weight of NaN for the rows that see it
            bad = __any_sync(0xFu << (lane & ~3), bad);
            if (bad && wq == 0) sm.key[t % kKeyStages].vs[r] = __uint_as_float(0x7FC00000u);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sts_v4(base + place[c] + 1024 * x, which && bad ? make_uint4(0, 0, 0, 0) : w[c]);
        }
      }
      fence_proxy_async_smem();
    };
    bool ok = true;
#pragma unroll 1
    for (int t = -6; ok && t < cnt; ++t) {
      const int b = t & 1;
      if (b == 0) zz0 = zz1;
      if (t >= 0) {
        cp_wait<1>();
        // K(t) over K(t - 2), which S(t - 2) has read; then V(t) over V(t - 2)
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
          if (t >= 2)
            ok = warp_wait(which ? &sm.bar_v_empty[b] : &sm.bar_s_full[b], ((t - 2) >> 1) & 1, abort_flag, a.hdr, 57);
          if (!ok) break;
          store_rows(which ? sm.v[b] : sm.k[b], t, which);
          warp_arrive(which ? &sm.bar_v_full[b] : &sm.bar_k_full[b]);
        }
        if (!ok) break;
      }
      if (t >= -2 && t + 2 < cnt) {
        if (b == 0) {  // tiles t + 2 and t + 3
          const int tl = t + 2 + odd;
          if ((lane & 15) == 0 && tl < cnt && tl >= kKeyStages)
            ok = lane_wait(&sm.bar_key_empty[tl % kKeyStages], ((tl / kKeyStages) & 1) ^ 1, abort_flag, a.hdr, 51);
          ok = warp_agree(ok);
          if (!ok) break;
          announce(t + 2);
        }
        copy_codes(t + 2);
      }
      if (t >= -2) cp_commit();
      if (b == 0) {
        if (t >= -4 && t + 4 < cnt) load_scales(t + 4);
        if (t + 6 < cnt) load_page(t + 6);
      }
    }
    if (checks && split == a.num_splits - 1 && warp == kEwWarps)  // the candidates, which are no tile's keys
      for (int j = g.h + lane; j < g.n; j += 32)
        sorted &= in_range(a.ts[g.tso + j]) && (j == 0 || a.ts[g.tso + j] >= a.ts[g.tso + j - 1]);
    if (!sorted) report_error(a.hdr, kErrUnsorted, user);
    cp_wait<0>();
  } else {
    // ------------------------------------------------------------------ elementwise warps
    for (int x = threadIdx.x; x < kMaxBuckets; x += 32 * kEwWarps) {
      sm.thr[x] = tab.thr[x];
      sm.rab_ts_half[x] = x < a.nb ? 0.5f * a.rab_ts[x] : 0.f;
    }
    if (threadIdx.x < 32)
      sm.oct[threadIdx.x] = make_uint4(tab.oct[threadIdx.x][0], tab.oct[threadIdx.x][1], tab.oct[threadIdx.x][2],
                                       tab.oct[threadIdx.x][3]);
    named_bar_sync(5, 32 * kEwWarps);
    const int grp = warp >> 2;                // warpgroup = 64-key half of every key tile
    const int r = threadIdx.x & (kTile - 1);  // query row of the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int i = min(g.qs + r, g.n - 1);
    const int jmax = i < g.h ? i : g.h - 1;
    const int pr = min(i, g.h);
    const int zb = prmin + 255 - pr;
    Walk w;
    w.t_i = a.ts[g.tso + i];
    w.b = 0;
    w.tlim = 0;
    w.tsb = 0.f;
    bool ok = true;
    for (int t = 0; t < cnt; ++t) {
      const int b = t & 1;
      int k0, width;
      key_tile(g, tb + t, k0, width);
      if (lane == 0) {
        ok = lane_wait(&sm.bar_win_full[t % kWinStages], (t / kWinStages) & 1, abort_flag, a.hdr, 56) &&
             lane_wait(&sm.bar_s_full[b], (t >> 1) & 1, abort_flag, a.hdr, 56);
        // a tile of new tokens: the NaN scales of its value rows are set
        if (k0 >= g.L) ok = ok && lane_wait(&sm.bar_v_full[b], (t >> 1) & 1, abort_flag, a.hdr, 56);
      }
      ok = warp_agree(ok);
      if (!ok) break;
      tc_fence_after();
      const KeyInfo& key = sm.key[t % kKeyStages];
      const Window& m = sm.win[t % kWinStages];
      const int climit = min(jmax - k0, width - 1);  // columns c <= climit are allowed
      const uint32_t s_tmem = tmem + lane_base + b * 128;
      if (t == 0) {
        w.b = bucket_of_dt(sm.thr, w.t_i - key.ts[min(64 * grp, width - 1)]);
        w.tlim = w.t_i + 1 - sm.thr[w.b];
        w.tsb = sm.rab_ts_half[w.b];
      }
#pragma unroll 1
      for (int col0 = 64 * grp; col0 < 64 * grp + 64; col0 += kCols) {
        uint32_t sr[kCols];
        tmem_ld32(s_tmem + col0, sr);
        int pos;
        float tsb_lo;
        const int mode = chunk_mode(w, key.ts, col0, climit, sm.thr, sm.rab_ts_half, pos, tsb_lo);
        const int z0 = zb + col0;
        const uint32_t winb = smem_u32(&m.win[z0 >> 3][z0 & 7]);
        uint32_t pw[kCols / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v4 = lds_v4(winb + k * 8 * 16);
          pw[4 * k] = v4.x;
          pw[4 * k + 1] = v4.y;
          pw[4 * k + 2] = v4.z;
          pw[4 * k + 3] = v4.w;
        }
        const float tsb = add_time_bias(mode, pw, w, key.ts + col0, pos - col0, tsb_lo, sm.thr, sm.rab_ts_half, sm.oct);
        tmem_wait_ld(sr);
        uint32_t lo[kCols / 2];
        weights_of(sr, pw, lo, tsb, key.ks + col0, key.vs + col0);
        if (!__all_sync(~0u, climit >= col0 + kCols - 1)) {
          // the mask comes last: a masked key's scales, and so its weight, may be NaN
#pragma unroll
          for (int k = 0; k < kCols / 2; ++k) {
            const int left = climit - col0 - 2 * k;  // columns allowed after the pair's first
            const uint32_t on = left >= 1 ? ~0u : left == 0 ? 0x0000FFFFu : 0u;
            pw[k] &= on;
            lo[k] &= on;
          }
        }
        // the chunk's P goes over its own (read) columns: the first terms, then the second
        tmem_st16(s_tmem + col0, pw);
        tmem_st16(s_tmem + col0 + 16, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&sm.bar_p_full[b]);
      if (lane == 0) {
        mbar_arrive(&sm.bar_key_empty[t % kKeyStages]);
        mbar_arrive(&sm.bar_win_empty[t % kWinStages]);
      }
    }
    // with no key tile nothing waited for Q, which the staging below is over
    ok = ok && warp_wait(cnt > 0 ? &sm.bar_o_full : &sm.bar_q, 0, abort_flag, a.hdr, 57);
    ok = ew_all(ok, grp);  // the warps left the loop by themselves
    tc_fence_after();
    if (ok) {
      // O out through shared memory in whole row segments (as attn_sm100_single.cu), 32 columns at a time
      const uint32_t stage = grp == 0 ? smem_u32(sm.q) : smem_u32(sm.k[0]);
      const int wrank = warp & 3;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int col0 = 64 * grp + 32 * x;
        const uint32_t slab = stage + x * (kTileBytes / 2);
        uint32_t orr[32];
        if (cnt > 0) {
          tmem_ld32(tmem + lane_base + 256 + col0, orr);
          tmem_wait_ld(orr);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          sts_v4(slab + r * 128 + ((c ^ (r & 7)) << 4),
                 make_uint4(orr[4 * c], orr[4 * c + 1], orr[4 * c + 2], orr[4 * c + 3]));
        named_bar_sync(1 + grp, kTile);
#pragma unroll 1
        for (int rr = 4 * wrank + (lane >> 3); rr < kTile; rr += 16) {
          const int c = lane & 7;
          if (rr < g.nq_rows) {
            const uint4 val = lds_v4(slab + rr * 128 + ((c ^ (rr & 7)) << 4));
            float* orow = a.o_ws + (((size_t)split * a.T_q + (g.qrow0 + rr)) * a.H + head) * kHeadDim;
            *reinterpret_cast<uint4*>(orow + col0 + 4 * c) = val;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_attn_q4_sm100(const AttnArgs& a, const BucketTable& thr, const int2* tiles, const CUtensorMap& tm_q,
                                 cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_q4_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  // a CTA per listed tile, head and split
  const long long ctas = ((long long)a.T_q / kTile + a.B) * a.H * a.num_splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_dependent(attn_q4_sm100_kernel, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, s, a, thr, tiles, tm_q);
}

}  // namespace hstu
