// Paged KV cache held in 4 bits: the write side (append) and the read-back.
//
// The pool has the paged layout of hstu_kv.cu with a row of d / 2 bytes for
// each token and head and one (scale, zero) word beside it; the row format is
// in quant_common.cuh.  Append = the plan of hstu_kv.cu (pages, new lengths)
// and a kernel that quantises every appended token's K and V rows into their
// slots; read = the same walk backwards, dense rows out.  Both move each row
// once and are bound by the bytes of k_new / v_new (or of the dense output).
//
// A group of G lanes owns a row (one token, one head, K or V): each lane holds
// W words of 8 elements, the extremes meet in log2(G) shuffles.
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

struct Q4Pool {
  uint8_t* k;
  uint8_t* v;
  uint32_t* k_meta;
  uint32_t* v_meta;
};

// Quantises the appended tokens of user blockIdx.x into the pool.
template <typename T, int G, int W>
__global__ void __launch_bounds__(kRowThreads) kv_append_q4_kernel(const KvArgs a, const Q4Pool pool) {
  if (a.hdr->pad[0] != 1) return;
  const int u = blockIdx.x;
  const int app = a.n_app[u];
  if (app <= 0) return;
  const int L = a.l_old[u];
  const int row0 = a.new_offsets[u];
  const int32_t* prow = a.page_table + (size_t)u * a.max_pages;
  const int words = a.d / 8;
  const int g = threadIdx.x % G;
  constexpr int kRows = kRowThreads / G;  // rows per block and step
  const long long items = 2ll * app * a.H;
  for (long long base = (long long)blockIdx.y * kRows; base < items; base += (long long)gridDim.y * kRows) {
    const long long it = base + threadIdx.x / G;
    const bool on = it < items;  // all lanes stay for the shuffles
    const int is_v = on && it >= (long long)app * a.H;
    const int y = on ? (int)(it - (is_v ? (long long)app * a.H : 0)) : 0;
    const int j = y / a.H, h = y - j * a.H;
    const T* src = reinterpret_cast<const T*>(is_v ? a.v_new : a.k_new) + (size_t)(row0 + j) * a.kv_stride +
                   (size_t)h * a.d;
    float x[W][8];
    float lo = 0.f, hi = 0.f;
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int wi = g + G * w;
      if (on && wi < words) {
        load8(src + 8 * wi, x[w]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo = fminf(lo, x[w][e]);
          hi = fmaxf(hi, x[w][e]);
          bits = max(bits, __float_as_uint(x[w][e]) & 0x7FFFFFFFu);
        }
      }
    }
#pragma unroll
    for (int o = G / 2; o >= 1; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
      bits = max(bits, __shfl_xor_sync(~0u, bits, o));
    }
    if (!on) continue;
    const Quant4 f = quant4_of(lo, hi, bits < 0x7F800000u);
    const int pos = L + j;
    const size_t slot = ((size_t)prow[pos / a.P] * a.H + h) * a.P + pos % a.P;
    uint32_t* dst = reinterpret_cast<uint32_t*>((is_v ? pool.v : pool.k) + slot * (a.d / 2));
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int wi = g + G * w;
      if (wi < words) {
        uint32_t word = 0;
        if (f.live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) word |= quant4_code(f, x[w][e]) << nibble_shift(e);
        }
        dst[wi] = word;
      }
    }
    if (g == 0) (is_v ? pool.v_meta : pool.k_meta)[slot] = f.meta;
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

// One step of a thread: 8 elements of one row.  Rows are independent: a user
// whose range or page is bad reports its error and its rows stay as they were.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) kv_read_q4_kernel(const ReadArgs a, const Q4Pool pool) {
  const int words = a.d / 8;
  const long long per_token = (long long)a.H * words;
  const long long items = (long long)a.total * per_token;
  for (long long x = blockIdx.x * (long long)kRowThreads + threadIdx.x; x < 2 * items;
       x += (long long)gridDim.x * kRowThreads) {
    const bool is_v = x >= items;
    const long long y = is_v ? x - items : x;
    const int row = (int)(y / per_token);
    const int rem = (int)(y - row * per_token);
    const int h = rem / words, w = rem - h * words;
    // user of the row: the last one whose rows start at or before it
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.offsets[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    const int r0 = a.offsets[lo], r1 = a.offsets[lo + 1];
    if (row < r0 || row >= r1) {
      // before the first user, behind the last, or offsets that decrease
      if (a.offsets[0] != 0 || r1 < r0) report_error(a.hdr, kErrLength, lo);
      continue;
    }
    const long long pos = (long long)a.starts[lo] + (row - r0);
    if (pos < 0 || a.starts[lo] < 0 || pos >= a.cached_lens[lo] || pos / a.P >= a.max_pages) {
      report_error(a.hdr, kErrLength, lo);
      continue;
    }
    const int pid = a.page_table[(size_t)lo * a.max_pages + pos / a.P];
    if (pid < 0 || pid >= a.num_pages) {
      report_error(a.hdr, kErrPage, lo);
      continue;
    }
    const size_t slot = ((size_t)pid * a.H + h) * a.P + (int)(pos % a.P);
    const uint32_t meta = (is_v ? pool.v_meta : pool.k_meta)[slot];
    const uint32_t code = reinterpret_cast<const uint32_t*>((is_v ? pool.v : pool.k) + slot * (a.d / 2))[w];
    const float s = meta_scale(meta), z = meta_zero(meta);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s * ((float)((code >> nibble_shift(e)) & 15u) - z);
    T* out = static_cast<T*>(is_v ? a.v_out : a.k_out) + ((size_t)row * a.H + h) * a.d + 8 * w;
    store8(out, v);
  }
}

template <typename T, int G, int W>
cudaError_t launch_append_q4(const KvArgs& a, const Q4Pool& pool, int parts, cudaStream_t s) {
  kv_append_q4_kernel<T, G, W><<<dim3(a.B, parts), kRowThreads, 0, s>>>(a, pool);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append_q4(const KvArgs& a, const Q4Pool& pool, int parts, cudaStream_t s) {
  if (a.d <= 32) return launch_append_q4<T, 4, 1>(a, pool, parts, s);
  if (a.d <= 64) return launch_append_q4<T, 8, 1>(a, pool, parts, s);
  if (a.d <= 128) return launch_append_q4<T, 16, 1>(a, pool, parts, s);
  return launch_append_q4<T, 16, 2>(a, pool, parts, s);
}

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
  if (launch_kv_append_plan(a, s) != cudaSuccess) return HSTU_ERR_CUDA;
  if (p->total_new == 0) return HSTU_OK;
  const int parts = 8;
  const cudaError_t e = p->dtype == HSTU_DT_BF16 ? launch_append_q4<__nv_bfloat16>(a, pool, parts, s)
                                                 : launch_append_q4<float>(a, pool, parts, s);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
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
  if (p->total_new == 0) return HSTU_OK;
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
  const long long steps = 2ll * p->total_new * p->num_heads * (p->head_dim / 8);
  const int blocks = (int)std::min<long long>((steps + kRowThreads - 1) / kRowThreads, 148 * 16);
  if (p->dtype == HSTU_DT_BF16)
    kv_read_q4_kernel<__nv_bfloat16><<<blocks, kRowThreads, 0, s>>>(a, pool);
  else
    kv_read_q4_kernel<float><<<blocks, kRowThreads, 0, s>>>(a, pool);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
