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
// With 128 rows against a key tile the step is bound by instruction issue (the
// SiLU and the widening of the codes) and by tanh, not by the cache's bytes
// (16 KB a tile), so nothing waits on anything for long and the widening is
// spread over the same 16 elementwise warps:
//
//   - each thread copies its own 16 bytes of a K and of a V row (cp.async) into
//     a place of its own in shared memory two tiles ahead and later widens them
//     into the 128B-swizzled tile the tensor core reads: no hand-over, no
//     producer of its own, four lanes a row (64 contiguous bytes).
//   - the order of one warp at key tile t: bias + SiLU of S(t) -> P(t); widen
//     K(t + 2) and V(t + 1); request the codes of K(t + 4), V(t + 3).  S is
//     double-buffered in tensor memory, so while the warps work on S(t) and widen,
//     the tensor core does O += P(t - 1) V(t - 1) and S(t + 1).
//   - one warp looks pages, scales and timestamps up for the tiles ahead (KeyInfo,
//     5 stages), one builds the position window (2 stages), one issues the MMAs.
//
// Tiles of new tokens (bf16 rows) take the same path without widening.  A value
// row that is not finite is stored as zeros and its scale set to NaN: the mask is
// applied to the finished weight, so rows that may not see the key stay finite.
// There is no plan launch: a CTA finds its (user, tile) by a scan of the offsets,
// looks at the page ids it uses and, for head 0, at the order of the timestamps.  Every wait is bounded.
#include <cuda_bf16.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr int kEwWarps = 16;              // 4 warpgroups: one 32-key chunk of every key tile each
constexpr int kEwThreads = 32 * kEwWarps;
constexpr int kMmaWarp = kEwWarps;        // MMA issuer, TMEM owner, Q
constexpr int kKeyWarp = kEwWarps + 1;
constexpr int kWinWarp = kEwWarps + 2;
constexpr int kThreads = 32 * (kEwWarps + 3);
constexpr int kKeyStages = 5;
constexpr int kWinStages = 2;
constexpr uint32_t kTmemCols = 512;       // S0 [0,128) S1 [128,256) O [256,384)

// What the key warp finds out about a tile's keys.
struct KeyInfo {
  long long ts[kTile];    // timestamps (the last one repeated past the tile's width)
  long long row[kTile];   // pool row (page, head, slot) of a cached key, or -1
  float ks[kTile];        // alpha / 2 times the scale of the key (new tokens: alpha / 2); 0 past the width
  uint32_t vs[kTile / 2]; // bf16 pairs: scale of the value (new tokens: 1); 0 past the width
  uint32_t zz[kTile];     // bf16 128 + zero of the key | of the value
};
struct Window {
  uint4 win[kWinChunks][8];
};

struct __align__(1024) SmemQ4 {
  uint8_t q[kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
  uint4 codes[2][2][kEwThreads];  // [stage][K, V]: each thread's 16 bytes
  KeyInfo key[kKeyStages];
  Window win[kWinStages];
  long long thr[kMaxBuckets];
  float rab_ts_half[kMaxBuckets];
  uint4 oct[32];
  uint32_t win_rs[kWinLoads * 16];
  uint64_t bar_q;
  uint64_t bar_key_full[kKeyStages];   // 32 lanes of the key warp
  uint64_t bar_key_empty[kKeyStages];  // 16 elementwise warps
  uint64_t bar_win_full[kWinStages];
  uint64_t bar_win_empty[kWinStages];
  uint64_t bar_s_full[2];  // S buffer b written
  uint64_t bar_p_full[2];  // P in buffer b written (512 threads)
  uint64_t bar_kv_full;    // 512 threads: phase 0 = K(0), K(1), V(0); phase t + 1 = K(t + 2), V(t + 1)
  uint64_t bar_pv;         // O += P(t) V(t) completed
  uint64_t bar_o_full;
  uint32_t tmem_base;
  int abort;
  int item_user, item_tile;
  int scan[20];
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
  return make_uint4(sub_bf16x2((w & 0x000F000Fu) | 0x43004300u, zz), sub_bf16x2(((w >> 4) & 0x000F000Fu) | 0x43004300u, zz),
                    sub_bf16x2(((w >> 8) & 0x000F000Fu) | 0x43004300u, zz),
                    sub_bf16x2(((w >> 12) & 0x000F000Fu) | 0x43004300u, zz));
}
// whether a bf16 pair holds an infinity or NaN
__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// The user and 128-row tile of the qt-th query tile of the batch (all threads;
// thread x sums the tiles of its share of users, the warps' sums meet in sm.scan).
__device__ __forceinline__ void find_item(const AttnArgs& a, SmemQ4& sm, int qt) {
  const int per = (a.B + kThreads - 1) / kThreads;
  const int lo = min(a.B, (int)threadIdx.x * per), hi = min(a.B, lo + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0;
  for (int u = lo; u < hi; ++u) mine += max(0, (int)(((long long)a.q_offsets[u + 1] - a.q_offsets[u] + kTile - 1) / kTile));
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.scan[warp] = incl;
  if (threadIdx.x == 0) sm.item_user = -1;
  __syncthreads();
  int before = incl - mine;
  for (int w = 0; w < warp; ++w) before += sm.scan[w];
  if (qt >= before && qt < before + mine) {
    int at = before;
    for (int u = lo; u < hi; ++u) {
      const int tiles = max(0, (int)(((long long)a.q_offsets[u + 1] - a.q_offsets[u] + kTile - 1) / kTile));
      if (qt < at + tiles) {
        sm.item_user = u;
        sm.item_tile = qt - at;
        break;
      }
      at += tiles;
    }
  }
  __syncthreads();
}

template <bool PRECISE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_q4_sm100_kernel(const AttnArgs a, const BucketTable tab, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ uint8_t smem_raw[];
  SmemQ4& sm = aligned_smem<SmemQ4>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.num_splits;
  const int head = (int)(blockIdx.x / a.num_splits) % a.H;
  const int qt = (int)(blockIdx.x / a.num_splits) / a.H;

  if (blockIdx.x == 0)  // users without a tile of their own are checked here
    for (int u = threadIdx.x; u < a.B; u += kThreads) {
      int n, tso, pages;
      if (!check_user(a, u, n, tso, pages)) report_error(a.hdr, kErrLength, u);
    }
  find_item(a, sm, qt);
  const int user = sm.item_user;
  if (user < 0) return;
  int n_all, tso, pages_all;
  if (!check_user(a, user, n_all, tso, pages_all)) {
    if (threadIdx.x == 0) report_error(a.hdr, kErrLength, user);
    return;
  }
  const TileGeom g = tile_geom(a, user, sm.item_tile);
  int tb, te;
  split_range(g.n_tiles, split, a.num_splits, tb, te);
  const int cnt = max(0, te - tb);
  const int prmin = min(g.qs, g.h);
  const int32_t* table = a.page_table + (size_t)user * a.max_pages;

  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_q, 1);
    for (int s = 0; s < kKeyStages; ++s) {
      mbar_init(&sm.bar_key_full[s], 32);
      mbar_init(&sm.bar_key_empty[s], kEwWarps);
    }
    for (int s = 0; s < kWinStages; ++s) {
      mbar_init(&sm.bar_win_full[s], 32);
      mbar_init(&sm.bar_win_empty[s], kEwWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.bar_s_full[b], 1);
      mbar_init(&sm.bar_p_full[b], kEwThreads);
    }
    mbar_init(&sm.bar_kv_full, kEwThreads);
    mbar_init(&sm.bar_pv, 1);
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
  volatile int* abort_flag = &sm.abort;
  const int row_base = a.q_offsets[user] - g.L;  // row of key position p is row_base + p (p >= L)

  if (warp == kKeyWarp) {
    // ------------------------------------------------------------------ key warp
    // lane l holds keys l, l + 32, ..: looked up one tile ahead of the free stage
    long long kts[4], krow[4];
    float kks[4];
    uint32_t kvs[4], kzz[4];
    // head 0 of the user's last tile (it sees every key but the candidates) checks the timestamps on the way
    const bool checks = head == 0 && (sm.item_tile + 1) * kTile >= g.n - g.L;
    bool sorted = true;
    auto in_range = [](long long x) { return x <= kTsLimit && x >= -kTsLimit; };
    long long last_ts = LLONG_MIN;  // timestamp of the key before the tile
    // page ids of a tile's keys, loaded a tile before the scales that they lead to; no branch
    // stands between the loads of the four keys, so that their latencies overlap
    int pid[4];
    auto load_pages = [&](int t) {
      int k0, width;
      key_tile(g, tb + t, k0, width);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        pid[k] = k0 < g.L ? table[page_index(a, k0 + min(lane + 32 * k, width - 1))] : 0;
    };
    auto look_up = [&](int t) {
      int k0, width;
      key_tile(g, tb + t, k0, width);
      const bool cached = k0 < g.L;
      uint32_t km[4], vm[4];
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k, j = k0 + min(c, width - 1), page = page_index(a, j);
        kts[k] = a.ts[g.tso + j];
        const bool in = pid[k] >= 0 && pid[k] < a.num_pages;
        bad |= !in;
        krow[k] = ((long long)(in ? pid[k] : 0) * a.H + head) * a.page_size + (cached ? j - page * a.page_size : 0);
        km[k] = a.k_scales[krow[k]];
        vm[k] = a.v_scales[krow[k]];
        if (!in || !cached || c >= width) krow[k] = -1;
      }
      if (bad) report_error(a.hdr, kErrPage, user);
      if (t + 1 < cnt) load_pages(t + 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool fresh = !cached && lane + 32 * k < width;  // a new token
        const bool held = krow[k] >= 0;
        kks[k] = held ? 0.5f * a.alpha * meta_scale(km[k]) : fresh ? 0.5f * a.alpha : 0.f;
        kvs[k] = held ? vm[k] & 0xFFFFu : fresh ? 0x3F80u : 0u;
        // 128 + zero in bf16, exact
        kzz[k] = held ? pack_bf16x2(128.f + meta_zero(km[k]), 128.f + meta_zero(vm[k])) : 0x43004300u;
        if (checks) {
          long long before = __shfl_up_sync(~0u, kts[k], 1);
          if (lane == 0) before = last_ts;
          last_ts = __shfl_sync(~0u, kts[k], 31);
          sorted &= kts[k] >= before && in_range(kts[k]);
        }
      }
    };
    if (checks && cnt > 0) {
      int k0, width;
      key_tile(g, tb, k0, width);
      if (k0 > 0) last_ts = a.ts[g.tso + k0 - 1];
    }
    if (cnt > 0) {
      load_pages(0);
      look_up(0);
    }
    for (int t = 0; t < cnt; ++t) {
      const int s = t % kKeyStages;
      bool ok = true;
      if (lane == 0 && t >= kKeyStages)
        ok = mbar_wait(&sm.bar_key_empty[s], ((t / kKeyStages) & 1) ^ 1, abort_flag, a.hdr, 51);
      ok = __shfl_sync(~0u, ok, 0);
      if (!ok) break;
      KeyInfo& key = sm.key[s];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k;
        key.ts[c] = kts[k];
        key.row[c] = krow[k];
        key.ks[c] = kks[k];
        reinterpret_cast<uint16_t*>(key.vs)[c] = (uint16_t)kvs[k];
        key.zz[c] = kzz[k];
      }
      mbar_arrive(&sm.bar_key_full[s]);
      if (t + 1 < cnt) look_up(t + 1);
    }
    if (checks && split == a.num_splits - 1)  // the candidates, which are no tile's keys
      for (int j = g.h + lane; j < g.n; j += 32)
        sorted &= in_range(a.ts[g.tso + j]) && (j == 0 || a.ts[g.tso + j] >= a.ts[g.tso + j - 1]);
    if (!sorted) report_error(a.hdr, kErrUnsorted, user);
  } else if (warp == kWinWarp) {
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
      bool ok = true;
      if (lane == 0 && t >= kWinStages)
        ok = mbar_wait(&sm.bar_win_empty[s], ((t / kWinStages) & 1) ^ 1, abort_flag, a.hdr, 52);
      ok = __shfl_sync(~0u, ok, 0);
      if (!ok) break;
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
      mbar_arrive(&sm.bar_win_full[s]);
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
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256, tmem + (t & 1) * 128 + (kk >> 1) * 32 + (kk & 1) * 8,
                 sw128_desc(v_base + kk * 2048, kHalfBytes, 1024), idesc_pv, (t > 0 || kk > 0));
      };
      // Q has landed before anything else uses it (and before the CTA may exit)
      bool ok = mbar_wait(&sm.bar_q, 0, abort_flag, a.hdr, 53);
      if (ok && cnt > 0) ok = mbar_wait(&sm.bar_kv_full, 0, abort_flag, a.hdr, 54);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < min(cnt, 2); ++t) issue_s(t);
      }
      for (int t = 0; ok && t < cnt; ++t) {
        ok = mbar_wait(&sm.bar_p_full[t & 1], (t >> 1) & 1, abort_flag, a.hdr, 55);
        if (!ok) break;
        tc_fence_after();
        issue_pv(t);  // V(t): phase t of kv_full, waited for below (t - 1) or above (0)
        if (t + 1 < cnt) {
          // the commit comes after this wait: with it the elementwise warps could be
          // through the next phase of kv_full before this thread looked at this one
          ok = mbar_wait(&sm.bar_kv_full, (t + 1) & 1, abort_flag, a.hdr, 54);
          if (!ok) break;
          mma_commit(&sm.bar_pv);
          tc_fence_after();
          if (t + 2 < cnt) issue_s(t + 2);
        }
      }
      mma_commit(&sm.bar_o_full);
      mbar_wait(&sm.bar_o_full, 0, nullptr, a.hdr, 58);
      mbar_wait(&sm.bar_q, 0, nullptr, a.hdr, 58);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ elementwise warps
    for (int x = threadIdx.x; x < kMaxBuckets; x += kEwThreads) {
      sm.thr[x] = tab.thr[x];
      sm.rab_ts_half[x] = x < a.nb ? 0.5f * a.rab_ts[x] : 0.f;
    }
    if (threadIdx.x < 32)
      sm.oct[threadIdx.x] = make_uint4(tab.oct[threadIdx.x][0], tab.oct[threadIdx.x][1], tab.oct[threadIdx.x][2],
                                       tab.oct[threadIdx.x][3]);
    named_bar_sync(5, kEwThreads);
    const int grp = warp >> 2;                // warpgroup = 32-key chunk of every key tile
    const int r = threadIdx.x & (kTile - 1);  // query row of the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int i = min(g.qs + r, g.n - 1);
    const int jmax = i < g.h ? i : g.h - 1;
    const int pr = min(i, g.h);
    const int zb = prmin + 255 - pr;
    const int col0 = 32 * grp;
    const uint8_t* kp = static_cast<const uint8_t*>(a.k_pool);
    const uint8_t* vp = static_cast<const uint8_t*>(a.v_pool);

    // ---- widening: this thread's key row and quarter (32 dimensions) of every tile
    const int wr = 8 * warp + (lane >> 2), wq = lane & 3;
    // the 16-byte chunk of dimensions 32 wq + 8 c sits at chunk (4 (wq & 1) + c) ^ (wr & 7) of half wq >> 1;
    // threads of the second half take their words in the order c ^ 2, so that the eight lanes of a
    // quarter-warp store to eight different places
    const int flip = wq & 2;
    const uint32_t wbase = (wq >> 1) * kHalfBytes + wr * 128;
    const int wchunk = 4 * (wq & 1);
    auto request = [&](int t, int which) {  // codes of K (0) or V (1) of tile t into this thread's place
      if (t >= cnt) return;
      const long long row = sm.key[t % kKeyStages].row[wr];
      if (row >= 0) cp16_ca(&sm.codes[t & 1][which][threadIdx.x], (which ? vp : kp) + row * 64 + 16 * wq);
    };
    auto store_row = [&](uint8_t* tile, int t, int which) {
      KeyInfo& key = sm.key[t % kKeyStages];
      const uint32_t base = smem_u32(tile) + wbase;
      int k0, width;
      key_tile(g, tb + t, k0, width);
      if (k0 < g.L) {  // cached keys: codes (zeros for rows past the width)
        uint4 w = make_uint4(0, 0, 0, 0);
        uint32_t zz = 0x43004300u;
        if (key.row[wr] >= 0) {
          w = sm.codes[t & 1][which][threadIdx.x];
          const uint32_t z = key.zz[wr];
          zz = __byte_perm(z, z, which ? 0x3232 : 0x1010);
        }
        if (flip) w = make_uint4(w.z, w.w, w.x, w.y);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) sts_v4(base + (((wchunk + (c ^ flip)) ^ (wr & 7)) << 4), widen8(ww[c], zz));
      } else {  // new tokens: bf16 rows as they are (zeros past the width)
        const bool on = wr < width;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(which ? a.v : a.k) +
                                                          (size_t)(row_base + k0 + (on ? wr : 0)) * a.qkv_stride +
                                                          head * kHeadDim + 32 * wq);
        uint4 w[4];
        bool bad = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          w[c] = on ? src[c] : make_uint4(0, 0, 0, 0);
          bad |= not_finite(w[c].x) | not_finite(w[c].y) | not_finite(w[c].z) | not_finite(w[c].w);
        }
        if (which) {  // a value row that is not finite: zeros, and a weight of NaN for the rows that see it
          bad = __any_sync(0xFu << (lane & ~3), bad);
          if (bad && wq == 0) reinterpret_cast<uint16_t*>(key.vs)[wr] = 0x7FC0u;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts_v4(base + (((wchunk + c) ^ (wr & 7)) << 4), which && bad ? make_uint4(0, 0, 0, 0) : w[c]);
      }
    };
    auto key_ready = [&](int t) -> bool {
      return t >= cnt || mbar_wait(&sm.bar_key_full[t % kKeyStages], (t / kKeyStages) & 1, abort_flag, a.hdr, 56);
    };

    bool ok = true;
    // first tiles: K(0), K(1), V(0) now; the codes of K(2), V(1) and K(3), V(2) on their way
    if (cnt > 0) {
      ok = key_ready(0) && key_ready(1) && key_ready(2) && key_ready(3);
      ok = ew_all(ok, grp);
      if (ok) {
        request(0, 0);
        request(1, 0);
        request(0, 1);
        cp_commit();
        cp_wait<0>();
        store_row(sm.k[0], 0, 0);
        if (cnt > 1) store_row(sm.k[1], 1, 0);
        store_row(sm.v[0], 0, 1);
        fence_proxy_async_smem();
        mbar_arrive(&sm.bar_kv_full);
        request(2, 0);
        request(1, 1);
        cp_commit();
        request(3, 0);
        request(2, 1);
        cp_commit();
      }
    }
    Walk w;
    w.t_i = a.ts[g.tso + i];
    w.b = 0;
    w.tlim = 0;
    w.tsb = 0.f;
    // (leaving the loop is agreed on by the warpgroup: ew_all)
    const int steps = ok ? cnt : 0;
    for (int t = 0; t < steps; ++t) {
      const int b = t & 1;
      int k0, width;
      key_tile(g, tb + t, k0, width);
      ok = ok && mbar_wait(&sm.bar_win_full[t % kWinStages], (t / kWinStages) & 1, abort_flag, a.hdr, 56);
      ok = ok && mbar_wait(&sm.bar_s_full[b], (t >> 1) & 1, abort_flag, a.hdr, 56);
      // a tile of new tokens: every thread has seen its value rows (the NaN scales)
      if (k0 >= g.L) ok = ok && mbar_wait(&sm.bar_kv_full, t & 1, abort_flag, a.hdr, 56);
      ok = ew_all(ok, grp);
      if (!ok) break;
      tc_fence_after();
      const KeyInfo& key = sm.key[t % kKeyStages];
      const Window& m = sm.win[t % kWinStages];
      const int climit = min(jmax - k0, width - 1);  // columns c <= climit are allowed
      const uint32_t s_tmem = tmem + lane_base + b * 128;
      uint32_t sr[32];
      tmem_ld32(s_tmem + col0, sr);
      if (t == 0) {
        w.b = bucket_of_dt(sm.thr, w.t_i - key.ts[min(col0, width - 1)]);
        w.tlim = w.t_i + 1 - sm.thr[w.b];
        w.tsb = sm.rab_ts_half[w.b];
      }
      const bool need_mask = !__all_sync(~0u, climit >= col0 + 31);
      int pos;
      float tsb_lo;
      const int mode = chunk_mode(w, key.ts, col0, climit, sm.thr, sm.rab_ts_half, pos, tsb_lo);
      const int z0 = zb + col0;
      const uint32_t winb = smem_u32(&m.win[z0 >> 3][z0 & 7]);
      uint32_t pw[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 v4 = lds_v4(winb + k * 8 * 16);
        pw[4 * k] = v4.x;
        pw[4 * k + 1] = v4.y;
        pw[4 * k + 2] = v4.z;
        pw[4 * k + 3] = v4.w;
      }
      tmem_wait_ld(sr);
      uint32_t pk[16];
      const float* ks = key.ks + col0;
      const uint32_t* vs = key.vs + col0 / 2;
      if (need_mask)
        silu_chunk_mode<true, PRECISE, true>(mode, sr, pw, pk, key.ts, col0, climit, pos, tsb_lo, 0.f, w, sm.thr,
                                             sm.rab_ts_half, sm.oct, ks, vs);
      else
        silu_chunk_mode<false, PRECISE, true>(mode, sr, pw, pk, key.ts, col0, climit, pos, tsb_lo, 0.f, w, sm.thr,
                                              sm.rab_ts_half, sm.oct, ks, vs);
      tmem_st16(s_tmem + col0, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.bar_p_full[b]);
      // ---- K(t + 2) over K(t) (S(t) has read it), V(t + 1) over V(t - 1)
      if (t + 1 < cnt) {
        cp_wait<1>();
        if (t + 2 < cnt) store_row(sm.k[b], t + 2, 0);
        if (t > 0) ok = mbar_wait(&sm.bar_pv, (t - 1) & 1, abort_flag, a.hdr, 57);
        ok = ew_all(ok, grp);
        if (!ok) break;
        store_row(sm.v[b ^ 1], t + 1, 1);
        fence_proxy_async_smem();
        mbar_arrive(&sm.bar_kv_full);
      }
      // the stages of tile t are free; the codes two tiles further are asked for
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.bar_key_empty[t % kKeyStages]);
        mbar_arrive(&sm.bar_win_empty[t % kWinStages]);
      }
      ok = key_ready(t + 4);
      ok = __all_sync(~0u, ok);
      if (ok) {
        request(t + 4, 0);
        request(t + 3, 1);
      }
      cp_commit();
    }
    cp_wait<0>();
    if (ok && cnt > 0) {
      ok = ew_all(mbar_wait(&sm.bar_o_full, 0, abort_flag, a.hdr, 57), grp);
      tc_fence_after();
    } else if (ok) {
      ok = ew_all(mbar_wait(&sm.bar_q, 0, abort_flag, a.hdr, 57), grp);  // the staging below is over Q
    }
    if (ok) {
      // O out through shared memory in whole row segments (as attn_sm100_single.cu)
      const uint32_t stage = (grp < 2 ? smem_u32(sm.q) : smem_u32(sm.k[0])) + (grp & 1) * (kTileBytes / 2);
      const int wrank = warp & 3;
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
        sts_v4(stage + r * 128 + ((c ^ (r & 7)) << 4),
               make_uint4(orr[4 * c], orr[4 * c + 1], orr[4 * c + 2], orr[4 * c + 3]));
      named_bar_sync(1 + grp, kTile);
#pragma unroll 1
      for (int rr = 4 * wrank + (lane >> 3); rr < kTile; rr += 16) {
        const int c = lane & 7;
        if (rr < g.nq_rows) {
          const uint4 val = lds_v4(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
          float* orow = a.o_ws + (((size_t)split * a.T_q + (g.qrow0 + rr)) * a.H + head) * kHeadDim;
          *reinterpret_cast<uint4*>(orow + col0 + 4 * c) = val;
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

cudaError_t launch_attn_q4_sm100(const AttnArgs& a, const BucketTable& thr, const CUtensorMap& tm_q, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(attn_q4_sm100_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attn_q4_sm100_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  // sum over users of ceil(rows / 128) <= T / 128 + B query tiles
  const long long tiles = (long long)a.T_q / kTile + a.B;
  const long long ctas = tiles * a.H * a.num_splits;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  if (a.precise_silu)
    attn_q4_sm100_kernel<true><<<(unsigned)ctas, kThreads, kSmemBytes, s>>>(a, thr, tm_q);
  else
    attn_q4_sm100_kernel<false><<<(unsigned)ctas, kThreads, kSmemBytes, s>>>(a, thr, tm_q);
  return cudaGetLastError();
}

}  // namespace hstu
