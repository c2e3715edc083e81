// Paged KV cache held in 4 bits: the write side (append) and the read-back.
//
// The pool has the paged layout of hstu_kv.cu with a row of d / 2 bytes for
// each token and head and one (scale, zero) word beside it; the row format is
// in quant_common.cuh.  Both kernels move each row once.  24576 tokens of 4 heads of
// 128 bf16 elements and their rows in the pool are 64 MB, 9.8 us at the copy's
// bandwidth.  The append takes 31 us: 21 instructions an element for the exact codes,
// the row's extremes and its format fill 60% of the issue slots, and a token's steps
// wait for one another.  The read-back takes 17 us: 56% of the issue slots, the rest
// mostly waits for the chain offsets - page table - row (34 warps an SM).
//
// A warp takes a token: G lanes hold a row (8 W elements each), so 32 / G heads
// go at once, K and V of two such groups of heads together (four independent
// 16-byte loads a lane).  In the append a warp's tokens are consecutive, so that
// user and page are looked up where they change (both kernels together 53.5 us,
// against 56.6 with a lookup for every token).
//
// Append is one launch for up to 256 users: every block works the allocation out
// for itself (one user a thread, one block-wide scan) from lengths, table and
// stack as they were, and copies its tokens; the block that was the last to read
// them (a counter) also writes the new table entries, lengths and stack height.
// Nothing is changed before every block has read it, and nothing at all if the
// batch does not fit.  More users take the plan launch of hstu_kv.cu first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.cuh"
#include "hstu.h"
#include "hstu_internal.h"
#include "kv_common.h"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kFusedUsers = kRowThreads;
constexpr int32_t kErrPool = -10;

struct Q4Pool {
  uint8_t* k;
  uint8_t* v;
  uint32_t* k_meta;
  uint32_t* v_meta;
};

// The users of a batch as a block of the one-launch append sees them.
struct FusedPlan {
  int32_t off[kFusedUsers + 1];  // rows of k_new
  int32_t old[kFusedUsers];      // cached tokens before
  int32_t app[kFusedUsers];      // appended tokens
  int32_t pre[kFusedUsers];      // pages taken by the users before
  int32_t part[kFusedUsers];     // the partly filled last page, where tokens go into it
  int32_t warp_sum[kRowWarps];
  int32_t err, total, fc, last;
};

// The allocation of kv_append_plan_kernel (same checks, same order of pages), in shared memory.
__device__ void plan_append(const KvArgs& a, FusedPlan& p) {
  const int u = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (u == 0) {
    p.err = 0;
    p.fc = *a.free_count;
  }
  if (u <= a.B) p.off[u] = a.new_offsets[u];
  if (u == 0 && a.B == kFusedUsers) p.off[a.B] = a.new_offsets[a.B];
  __syncthreads();
  int need = 0;
  if (u < a.B) {
    const int L = a.cached_lens[u], r0 = p.off[u], r1 = p.off[u + 1], n_new = r1 - r0;
    const int app = a.num_append ? a.num_append[u] : n_new;
    p.old[u] = L;
    p.app[u] = app;
    if (L < 0 || r0 < 0 || r1 > a.total_new || n_new < 0 || app < 0 || app > n_new) {
      atomicCAS(&p.err, 0, kErrLength);
    } else {
      const long long have = ((long long)L + a.P - 1) / a.P, want = ((long long)L + app + a.P - 1) / a.P;
      if (want > a.max_pages) {
        atomicCAS(&p.err, 0, kErrPool);
      } else {
        need = (int)(want - have);
        if (app > 0 && L % a.P != 0) {  // the partly filled last page receives tokens
          const int pid = a.page_table[(size_t)u * a.max_pages + L / a.P];
          if (pid < 0 || pid >= a.num_pages) atomicCAS(&p.err, 0, kErrPage);
          p.part[u] = pid;
        }
      }
    }
  }
  int incl = need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) p.warp_sum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    if (w < warp) before += p.warp_sum[w];
    total += p.warp_sum[w];
  }
  if (u < a.B) p.pre[u] = before + incl - need;
  if (u == 0) {
    p.total = total;
    if (p.err == 0 && (total > p.fc || p.fc > a.num_pages)) p.err = kErrPool;
  }
  __syncthreads();
  if (p.err == 0)  // the pages about to be taken must be pool pages
    for (int x = p.fc - total + u; x < p.fc; x += kRowThreads) {
      const int pid = a.free_pages[x];
      if (pid < 0 || pid >= a.num_pages) atomicCAS(&p.err, 0, kErrPage);
    }
  __syncthreads();
}

// largest u with off[u] <= row
__device__ __forceinline__ int user_of(const int32_t* off, int B, int row) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// This lane's elements of a token's rows: K, V of head h, K, V of the group of heads behind it.
template <typename T, int G, int W>
__device__ __forceinline__ void load_rows(const KvArgs& a, int row, int h, Elems8<T> (&x)[4][W]) {
  const int g = threadIdx.x % G, words = a.d / 8;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int hi = h + (i >> 1) * (32 / G), wi = g + G * w;
      if (hi < a.H && wi < words)
        x[i][w].load(reinterpret_cast<const T*>(i & 1 ? a.v_new : a.k_new) + (size_t)row * a.kv_stride +
                     (size_t)hi * a.d + 8 * wi);
      else
        x[i][w].zero();
    }
}

// Rows of one token (K and V, all heads; x: those of the first heads) into slot rows slot0 + h * P of the pool.
template <typename T, int G, int W>
__device__ __forceinline__ void quantise_token(const KvArgs& a, const Q4Pool& pool, int row, size_t page_row, int slot,
                                               Elems8<T> (&x)[4][W]) {
  const int lane = threadIdx.x & 31, g = lane % G;
  const int words = a.d / 8;
  constexpr int kHeads = 32 / G;
  for (int h0 = lane / G; h0 - lane / G < a.H; h0 += 2 * kHeads) {
    if (h0 >= 2 * kHeads) load_rows<T, G, W>(a, row, h0, x);
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      auto ex = x[i][0].extremes();
#pragma unroll
      for (int w = 1; w < W; ++w) ex = Elems8<T>::join(ex, x[i][w].extremes());
#pragma unroll
      for (int o = G / 2; o >= 1; o >>= 1) ex = Elems8<T>::join(ex, Elems8<T>::other(ex, o));
      if ((lane & 3) == i) {  // lane i of a group of four works row i's format out for all
        lo = Elems8<T>::lowest(ex);
        hi = Elems8<T>::highest(ex);
      }
    }
    bool clamp;
    const Quant4 f = quant4_of(lo, hi, clamp);
    const unsigned clamps = __ballot_sync(~0u, clamp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = (lane & ~3) + i;
      const float s = __shfl_sync(~0u, f.s, from), inv = __shfl_sync(~0u, f.inv, from), z = __shfl_sync(~0u, f.z, from);
      const uint32_t meta = __shfl_sync(~0u, f.meta, from);
      const bool cl = (clamps >> from) & 1;
      const int h = h0 + (i >> 1) * kHeads;
      if (h < a.H) {
        const size_t at = (page_row + h) * a.P + slot;
        uint32_t* dst = reinterpret_cast<uint32_t*>((i & 1 ? pool.v : pool.k) + at * (a.d / 2));
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (g + G * w < words) {
            float e[8];
            x[i][w].get(e);
            dst[g + G * w] = quant4_word<sizeof(T) == 2>(s, inv, z, cl, e);
          }
        if (g == 0) (i & 1 ? pool.v_meta : pool.k_meta)[at] = meta;
      }
    }
  }
}

template <typename T, int G, int W, bool FUSED>
__global__ void __launch_bounds__(kRowThreads) kv_append_q4_kernel(const KvArgs a, const Q4Pool pool) {
  __shared__ FusedPlan p;
  if constexpr (FUSED) {
    plan_append(a, p);
    if (p.err != 0) {  // the same in every block
      if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.hdr, p.err, 0);
      return;
    }
    // this block has read all that an append changes (the stack's entries stay as they are)
    if (threadIdx.x == 0) {
      __threadfence();
      p.last = atomicAdd(&a.hdr->blocks_done, 1) == (int)gridDim.x - 1;
      __threadfence();
    }
  } else {
    if (a.hdr->pad[0] != 1) return;
  }
  const int32_t* off = FUSED ? p.off : a.new_offsets;
  const int32_t* app = FUSED ? p.app : a.n_app;
  const int32_t* old = FUSED ? p.old : a.l_old;
  // a warp takes tokens in a row: user and page are looked up where they change
  const int first = off[0], total = off[a.B] - first, warps = gridDim.x * kRowWarps;
  const int per = (total + warps - 1) / warps;
  const int lo = min(total, (int)(blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * per), end = first + min(total, lo + per);
  int u = 0, next = first, left = 0, page = 0, slot = 0, pid = 0;  // next: first row of the next user
  for (int row = first + lo; row < end; ++row) {
    bool look = false;
    if (row >= next || row == first + lo) {
      u = user_of(off, a.B, row);
      next = off[u + 1];
      const int j = row - off[u], pos = old[u] + j;
      left = app[u] - j;  // tokens of the user still to append
      page = pos / a.P;
      slot = pos - page * a.P;
      look = true;
    }
    if (left-- <= 0) continue;
    Elems8<T> x[4][W];
    load_rows<T, G, W>(a, row, (threadIdx.x & 31) / G, x);  // on their way while the page is looked up
    if (slot == a.P) {
      ++page;
      slot = 0;
      look = true;
    }
    if (look) {
      if constexpr (FUSED) {
        const int have = (old[u] + a.P - 1) / a.P;
        pid = page < have ? p.part[u] : a.free_pages[p.fc - 1 - p.pre[u] - (page - have)];
      } else {
        pid = a.page_table[(size_t)u * a.max_pages + page];
      }
    }
    quantise_token<T, G, W>(a, pool, row, (size_t)pid * a.H, slot++, x);
  }
  if constexpr (FUSED) {
    // the block that was last to read the old state writes the new one
    __syncthreads();
    if (!p.last) return;
    const int u = threadIdx.x;
    if (u < a.B) {
      const int have = (p.old[u] + a.P - 1) / a.P;
      const int need = (int)(((long long)p.old[u] + p.app[u] + a.P - 1) / a.P) - have;
      int32_t* row = a.page_table + (size_t)u * a.max_pages + have;
      for (int j = 0; j < need; ++j) row[j] = a.free_pages[p.fc - 1 - p.pre[u] - j];
      a.cached_lens[u] = p.old[u] + p.app[u];
    }
    if (u == 0) *a.free_count = p.fc - p.total;
  }
}

// ---- read-back ------------------------------------------------------------------
struct ReadArgs {
  int32_t B, H, d, P, num_pages, max_pages, total;
  const int32_t* page_table;
  const int32_t* cached_lens;
  const int32_t* starts;
  const int32_t* offsets;
  void* k_out;
  void* v_out;
  WsHeader* hdr;
};

// Rows are independent: a user whose range or page is bad reports its error and
// its rows stay as they were.  The first block also looks at the offsets, since a
// user's rows past the output have no warp that would report them.
template <typename T, int G, int W>
__global__ void __launch_bounds__(kRowThreads) kv_read_q4_kernel(const ReadArgs a, const Q4Pool pool) {
  const int lane = threadIdx.x & 31, g = lane % G;
  const int words = a.d / 8;
  constexpr int kHeads = 32 / G;
  if (blockIdx.x == 0)
    for (int u = threadIdx.x; u < a.B; u += kRowThreads) {
      const int r0 = a.offsets[u], r1 = a.offsets[u + 1];
      if ((u == 0 && r0 != 0) || r1 < r0 || r1 > a.total) report_error(a.hdr, kErrLength, u);
    }
  for (int row = blockIdx.x * kRowWarps + (threadIdx.x >> 5); row < a.total; row += gridDim.x * kRowWarps) {
    const int u = user_of(a.offsets, a.B, row);
    const int r0 = a.offsets[u], r1 = a.offsets[u + 1];
    if (row < r0 || row >= r1) continue;  // before the first user, behind the last, or offsets that decrease
    const long long pos = (long long)a.starts[u] + (row - r0);
    const int page = (int)(pos / a.P);
    if (a.starts[u] < 0 || pos >= a.cached_lens[u] || page >= a.max_pages) {
      if (lane == 0) report_error(a.hdr, kErrLength, u);
      continue;
    }
    const int pid = a.page_table[(size_t)u * a.max_pages + page];
    if (pid < 0 || pid >= a.num_pages) {
      if (lane == 0) report_error(a.hdr, kErrPage, u);
      continue;
    }
    const int slot = (int)(pos - (long long)page * a.P);
    for (int h0 = lane / G; h0 < a.H; h0 += 2 * kHeads) {
      uint32_t meta[2][2], code[2][2][W];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int h = h0 + i * kHeads;
          const size_t at = ((size_t)pid * a.H + (h < a.H ? h : h0)) * a.P + slot;
          meta[i][v] = (v ? pool.v_meta : pool.k_meta)[at];
#pragma unroll
          for (int w = 0; w < W; ++w)
            code[i][v][w] = g + G * w < words
                                ? reinterpret_cast<const uint32_t*>((v ? pool.v : pool.k) + at * (a.d / 2))[g + G * w]
                                : 0u;
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int h = h0 + i * kHeads;
          const float s = meta_scale(meta[i][v]), z = meta_zero(meta[i][v]);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            if (h >= a.H || g + G * w >= words) continue;
            T* out = static_cast<T*>(v ? a.v_out : a.k_out) + ((size_t)row * a.H + h) * a.d + 8 * (g + G * w);
            const uint32_t c = code[i][v][w];
            if constexpr (sizeof(T) == 2) {
              // code - zero is exact in bf16 and the product is rounded once, two elements at a time
              const __nv_bfloat162 s2 = __float2bfloat162_rn(s), z2 = __float2bfloat162_rn(128.f + z);
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t q = ((c >> (4 * e)) & 0x000F000Fu) | 0x43004300u;
                const __nv_bfloat162 p = __hmul2(s2, __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q), z2));
                y[e] = *reinterpret_cast<const uint32_t*>(&p);
              }
              *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
            } else {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)  // 2^23 + code, exact
                y[e] = s * (__uint_as_float(((c >> nibble_shift(e)) & 15u) | 0x4B000000u) - (8388608.f + z));
              store8(out, y);
            }
          }
        }
    }
  }
}

// lanes of a row and words of a lane for a head size
template <template <int, int> class F, typename... Args>
cudaError_t by_head_dim(int d, Args&&... args) {
  if (d <= 32) return F<4, 1>::run(args...);
  if (d <= 64) return F<8, 1>::run(args...);
  if (d <= 128) return F<16, 1>::run(args...);
  return F<16, 2>::run(args...);
}

template <int G, int W>
struct Append {
  static cudaError_t run(const KvArgs& a, const Q4Pool& pool, bool bf16, bool fused, int blocks, cudaStream_t s) {
    if (fused) {
      if (bf16) kv_append_q4_kernel<__nv_bfloat16, G, W, true><<<blocks, kRowThreads, 0, s>>>(a, pool);
      else kv_append_q4_kernel<float, G, W, true><<<blocks, kRowThreads, 0, s>>>(a, pool);
    } else {
      if (bf16) kv_append_q4_kernel<__nv_bfloat16, G, W, false><<<blocks, kRowThreads, 0, s>>>(a, pool);
      else kv_append_q4_kernel<float, G, W, false><<<blocks, kRowThreads, 0, s>>>(a, pool);
    }
    return cudaGetLastError();
  }
};

template <int G, int W>
struct Read {
  static cudaError_t run(const ReadArgs& a, const Q4Pool& pool, bool bf16, int blocks, cudaStream_t s) {
    if (bf16) kv_read_q4_kernel<__nv_bfloat16, G, W><<<blocks, kRowThreads, 0, s>>>(a, pool);
    else kv_read_q4_kernel<float, G, W><<<blocks, kRowThreads, 0, s>>>(a, pool);
    return cudaGetLastError();
  }
};

// a warp a token, up to so many blocks of 8 warps an SM
int row_blocks(int rows, int per_sm) { return std::max(1, std::min((rows + kRowWarps - 1) / kRowWarps, 148 * per_sm)); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t ws_bytes_for(const hstu_kv_params* p) {
  return sizeof(WsHeader) + ((size_t)p->batch * 2 * sizeof(int32_t) + 255) / 256 * 256;
}

int check(const hstu_kv_params* p) {
  if (!p || p->batch <= 0 || p->num_heads <= 0 || p->head_dim <= 0 || p->page_size <= 0 || p->num_pages <= 0 ||
      p->max_pages_per_user <= 0 || p->kv_stride < 0 || p->total_new < 0)
    return HSTU_ERR_INVALID_ARG;
  if (p->dtype != HSTU_DT_BF16 && p->dtype != HSTU_DT_F32) return HSTU_ERR_INVALID_ARG;
  if (p->head_dim % 32 || p->head_dim > 256) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

size_t hstu_kv_q4_workspace_size(const hstu_kv_params* p) { return check(p) == HSTU_OK ? ws_bytes_for(p) : 0; }

int hstu_kv_append_q4(const hstu_kv_params* p, const void* k_new, const void* v_new, const int32_t* new_offsets,
                      const int32_t* num_append, void* k_pool, void* v_pool, void* k_scales, void* v_scales,
                      int32_t* page_table, int32_t* cached_lens, int32_t* free_pages, int32_t* free_count,
                      void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  if (int rc = check(p)) return rc;
  if ((p->total_new > 0 && (!k_new || !v_new)) || !new_offsets || !k_pool || !v_pool || !k_scales || !v_scales ||
      !page_table || !cached_lens || !free_pages || !free_count || !workspace)
    return HSTU_ERR_INVALID_ARG;
  const int esize = p->dtype == HSTU_DT_BF16 ? 2 : 4;
  const long long stride = p->kv_stride ? p->kv_stride : (long long)p->num_heads * p->head_dim;
  if (stride < (long long)p->num_heads * p->head_dim) return HSTU_ERR_INVALID_ARG;
  if ((stride * esize) % 16 || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
      !aligned16(k_scales) || !aligned16(v_scales) || !aligned16(workspace))
    return HSTU_ERR_ALIGNMENT;
  if (workspace_bytes < ws_bytes_for(p)) return HSTU_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  KvArgs a{};
  a.B = p->batch;
  a.H = p->num_heads;
  a.d = p->head_dim;
  a.P = p->page_size;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages_per_user;
  a.esize = esize;
  a.total_new = p->total_new;
  a.kv_stride = stride;
  a.k_new = static_cast<const uint8_t*>(k_new);
  a.v_new = static_cast<const uint8_t*>(v_new);
  a.new_offsets = new_offsets;
  a.num_append = num_append;
  a.page_table = page_table;
  a.cached_lens = cached_lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.hdr = static_cast<WsHeader*>(workspace);
  a.l_old = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + sizeof(WsHeader));
  a.n_app = a.l_old + p->batch;
  const Q4Pool pool{static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool), static_cast<uint32_t*>(k_scales),
                    static_cast<uint32_t*>(v_scales)};
  if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return HSTU_ERR_CUDA;
  const bool fused = p->batch <= kFusedUsers;
  if (!fused) {
    if (launch_kv_append_plan(a, s) != cudaSuccess) return HSTU_ERR_CUDA;
    if (p->total_new == 0) return HSTU_OK;
  }
  return by_head_dim<Append>(p->head_dim, a, pool, p->dtype == HSTU_DT_BF16, fused, row_blocks(p->total_new, 4), s) ==
                 cudaSuccess
             ? HSTU_OK
             : HSTU_ERR_CUDA;
}

int hstu_kv_read_q4(const hstu_kv_params* p, const void* k_pool, const void* v_pool, const void* k_scales,
                    const void* v_scales, const int32_t* page_table, const int32_t* cached_lens,
                    const int32_t* starts, const int32_t* offsets, void* k_out, void* v_out, void* workspace,
                    size_t workspace_bytes, hstu_stream_t stream) {
  if (int rc = check(p)) return rc;
  if ((p->total_new > 0 && (!k_out || !v_out)) || !k_pool || !v_pool || !k_scales || !v_scales || !page_table ||
      !cached_lens || !starts || !offsets || !workspace)
    return HSTU_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_scales) ||
      !aligned16(v_scales) || !aligned16(workspace))
    return HSTU_ERR_ALIGNMENT;
  if (workspace_bytes < sizeof(WsHeader)) return HSTU_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), s) != cudaSuccess) return HSTU_ERR_CUDA;
  ReadArgs a;
  a.B = p->batch;
  a.H = p->num_heads;
  a.d = p->head_dim;
  a.P = p->page_size;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages_per_user;
  a.total = p->total_new;
  a.page_table = page_table;
  a.cached_lens = cached_lens;
  a.starts = starts;
  a.offsets = offsets;
  a.k_out = k_out;
  a.v_out = v_out;
  a.hdr = static_cast<WsHeader*>(workspace);
  const Q4Pool pool{static_cast<uint8_t*>(const_cast<void*>(k_pool)), static_cast<uint8_t*>(const_cast<void*>(v_pool)),
                    static_cast<uint32_t*>(const_cast<void*>(k_scales)),
                    static_cast<uint32_t*>(const_cast<void*>(v_scales))};
  const cudaError_t e =
      by_head_dim<Read>(p->head_dim, a, pool, p->dtype == HSTU_DT_BF16, row_blocks(p->total_new, 8), s);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
