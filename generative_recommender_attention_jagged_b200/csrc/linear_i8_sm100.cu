// Linear layer in 8-bit integers: y = act(x W + bias) with x quantised token
// by token and W channel by channel (formats in quant_common.cuh), the integer
// products summed exactly in int32 on the tensor cores (tcgen05 kind::i8).
//
//   scale_x[t] = amax_t / 127,  code[t, k] = rint(x[t, k] / scale_x[t])
//   y[t, n] = act(scale_x[t] * scale_w[n] * sum_k code[t, k] wq[n, k] + bias[n])
//
// Two launches: the rows are quantised into the workspace (one warp a row, one
// read of x), then the GEMM runs on the codes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "device_common.cuh"
#include "hstu.h"
#include "hstu_internal.h"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr size_t kHeaderBytes = sizeof(WsHeader);

// ---- quantise rows ------------------------------------------------------------
constexpr int kRowRegs = 4;  // a warp keeps up to 4 x 256 elements of its row in registers

__device__ __forceinline__ uint32_t abs_bits_max(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// 8 codes as 8 bytes
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv) {
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = __float_as_uint(round_quotient(x[i], s, inv));
  const uint32_t a = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
  const uint32_t b = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
  return make_uint2(a, b);
}

template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, long long rows, int cols,
                                                         long long x_stride, int8_t* __restrict__ xq,
                                                         float* __restrict__ scale, WsHeader* hdr) {
  if (blockIdx.x == 0 && threadIdx.x < sizeof(WsHeader) / 4) reinterpret_cast<int32_t*>(hdr)[threadIdx.x] = 0;
  const int lane = threadIdx.x & 31;
  for (long long r = blockIdx.x * 8ll + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8ll) {
    const T* row = x + r * x_stride;
    float keep[kRowRegs][8];
    uint32_t amax_bits = 0;
#pragma unroll
    for (int j = 0; j < kRowRegs; ++j) {
      const int c = 256 * j + 8 * lane;
      if (c < cols) {
        load8(row + c, keep[j]);
        amax_bits = abs_bits_max(keep[j], amax_bits);
      }
    }
    for (int c = 256 * kRowRegs + 8 * lane; c < cols; c += 256) {
      float v[8];
      load8(row + c, v);
      amax_bits = abs_bits_max(v, amax_bits);
    }
    amax_bits = __reduce_max_sync(~0u, amax_bits);
    const bool finite = amax_bits < 0x7F800000u;
    float s = __fdiv_rn(__uint_as_float(amax_bits), 127.f);
    const bool live = finite && s >= FLT_MIN;
    const float inv = live ? 1.f / s : 0.f;
    if (lane == 0) scale[r] = live ? s : (finite ? 0.f : __uint_as_float(0x7FC00000u));
    int8_t* out = xq + r * cols;
#pragma unroll
    for (int j = 0; j < kRowRegs; ++j) {
      const int c = 256 * j + 8 * lane;
      if (c < cols) *reinterpret_cast<uint2*>(out + c) = live ? codes8(keep[j], s, inv) : make_uint2(0, 0);
    }
    for (int c = 256 * kRowRegs + 8 * lane; c < cols; c += 256) {
      float v[8];
      load8(row + c, v);
      *reinterpret_cast<uint2*>(out + c) = live ? codes8(v, s, inv) : make_uint2(0, 0);
    }
  }
}

// ---- quantise a weight: w [K, N] -> wq [N, K], one scale a channel -------------
// A block owns 32 channels: amax down the rows (lane = channel, coalesced), then
// 32 x 32 tiles of codes turned through shared memory so that wq is written in rows.
template <typename T>
__global__ void __launch_bounds__(256) quant_weight_kernel(const T* __restrict__ w, int K, int N,
                                                           int8_t* __restrict__ wq, float* __restrict__ scale) {
  __shared__ uint32_t part[8][32];
  __shared__ int8_t tile[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + lane;
  uint32_t m = 0;
  if (n < N)
    for (int k = warp; k < K; k += 8) m = max(m, __float_as_uint((float)w[(size_t)k * N + n]) & 0x7FFFFFFFu);
  part[warp][lane] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = max(m, part[i][lane]);
  const bool finite = m < 0x7F800000u;
  const float s = __fdiv_rn(__uint_as_float(m), 127.f);
  const bool live = finite && s >= FLT_MIN;
  const float inv = live ? 1.f / s : 0.f;
  if (warp == 0 && n < N) scale[n] = live ? s : (finite ? 0.f : __uint_as_float(0x7FC00000u));
  for (int k0 = 0; k0 < K; k0 += 32) {
    __syncthreads();
    for (int i = warp; i < 32; i += 8) {
      const int k = k0 + i;
      int8_t q = 0;
      if (n < N && k < K && live)
        q = (int8_t)(__float_as_uint(round_quotient((float)w[(size_t)k * N + n], s, inv)) & 0xFFu);
      tile[i][lane] = q;
    }
    __syncthreads();
    for (int i = warp; i < 32; i += 8) {
      const int nn = blockIdx.x * 32 + i, k = k0 + lane;
      if (nn < N && k < K) wq[(size_t)nn * K + k] = tile[lane][i];
    }
  }
}

// ---- GEMM ---------------------------------------------------------------------
constexpr int kBM = 128;   // rows per CTA
constexpr int kBK = 128;   // codes per K block: one 128-byte swizzled row
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps);

template <int BN>
struct __align__(1024) SmemI8 {
  static constexpr int kStages = 4;
  uint8_t x[kStages][kBM * kBK];
  uint8_t w[kStages][BN * kBK];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};

struct GemmI8Args {
  long long T;
  int K, N;
  long long out_stride;  // elements
  int silu;
  const float* x_scale;
  const float* w_scale;
  const float* bias;
  void* out;
  WsHeader* hdr;
};

// Instruction descriptor of kind::i8: signed 8-bit operands, both K-major, int32 sums.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4)                    // D format: s32
         | (1u << 7)                  // A format: signed
         | (1u << 10)                 // B format: signed
         | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// SiLU for a bf16 result: h + h tanh h with h = x / 2 (error of tanh.approx
// 2^-11, below the rounding to bf16); for an fp32 result x / (1 + exp(-x)).
template <typename TOut>
__device__ __forceinline__ float act_i8(float x, int silu) {
  if (!silu) return x;
  if constexpr (sizeof(TOut) == 2) {
    const float h = 0.5f * x;
    return fmaf(h, tanh_approx(h), h);
  } else {
    return x / (1.f + expf(-x));
  }
}

// One CTA per 128 x BN output tile.  Warp 0: TMA producer; warp 1: MMA issuer
// and owner of tensor memory; warps 2-5: epilogue (thread = output row).
template <int BN, typename TOut>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_i8_kernel(const GemmI8Args a, const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ CUtensorMap tm_w) {
  using Smem = SmemI8<BN>;
  constexpr int kStages = Smem::kStages;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = aligned_smem<Smem>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = (a.N + BN - 1) / BN;
  const int m0 = (int)(blockIdx.x / tiles_n) * kBM, n0 = (int)(blockIdx.x % tiles_n) * BN;
  const int nk = (a.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = 0; kb < nk; ++kb) {
        const int s = kb % kStages;
        if (!mbar_wait(&sm.empty[s], ((kb / kStages) & 1) ^ 1, abort_flag, a.hdr, 41)) break;
        mbar_arrive_expect_tx(&sm.full[s], kBM * kBK + BN * kBK);
        tma_load_2d(sm.x[s], &tm_x, &sm.full[s], kb * kBK, m0);
        tma_load_2d(sm.w[s], &tm_w, &sm.full[s], kb * kBK, n0);
        issued = kb + 1;
      }
      // no copy may still be landing when the CTA exits
      for (int t = max(0, issued - kStages); t < issued; ++t)
        mbar_wait(&sm.full[t % kStages], (t / kStages) & 1, nullptr, a.hdr, 49);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8(kBM, BN);
      for (int kb = 0; kb < nk; ++kb) {
        const int s = kb % kStages;
        if (!mbar_wait(&sm.full[s], (kb / kStages) & 1, abort_flag, a.hdr, 42)) break;
        tc_fence_after();
        const uint32_t xb = smem_u32(sm.x[s]), wb = smem_u32(sm.w[s]);
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)
          mma_i8_ss(tmem, sw128_desc(xb + kk * 32, 16, 1024), sw128_desc(wb + kk * 32, 16, 1024), idesc,
                    (kb | kk) != 0);
        mma_commit(&sm.empty[s]);
      }
      mma_commit(&sm.done);
      mbar_wait(&sm.done, 0, nullptr, a.hdr, 48);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    const long long row = m0 + quarter * 32 + lane;
    const bool ok = mbar_wait(&sm.done, 0, abort_flag, a.hdr, 43) && !*abort_flag;
    if (__all_sync(~0u, ok)) {
      tc_fence_after();
      const float xs = row < a.T ? a.x_scale[row] : 0.f;
      TOut* out = static_cast<TOut*>(a.out) + row * a.out_stride;
#pragma unroll 1
      for (int c0 = 0; c0 < BN && n0 + c0 < a.N; c0 += 32) {
        uint32_t acc[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + c0, acc);
        tmem_wait_ld(acc);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          const int n = n0 + c0 + e;
          if (n >= a.N) break;  // N is a multiple of 8
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float b = a.bias ? __ldg(a.bias + n + i) : 0.f;
            y[i] = act_i8<TOut>(fmaf(__int2float_rn((int)acc[e + i]), xs * __ldg(a.w_scale + n + i), b), a.silu);
          }
          if (row < a.T) store8(out + n, y);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, BN);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// [rows, K] codes, packed rows: box = box_rows x 128 codes, 128B swizzle, zeros outside
bool encode_codes(CUtensorMap* m, const void* base, long long rows, int K, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename TOut>
cudaError_t launch_single(const GemmI8Args& a, const void* xq, const void* wq, int dev, cudaStream_t s) {
  constexpr size_t smem = sizeof(SmemI8<BN>) + 1024;
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(gemm_i8_kernel<BN, TOut>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  CUtensorMap tx, tw;
  if (!encode_codes(&tx, xq, a.T, a.K, kBM) || !encode_codes(&tw, wq, a.N, a.K, BN)) return cudaErrorInvalidValue;
  const long long tiles = ((a.T + kBM - 1) / kBM) * ((a.N + BN - 1) / BN);
  gemm_i8_kernel<BN, TOut><<<(unsigned)tiles, kThreads, smem, s>>>(a, tx, tw);
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// status header, the rows' codes, the rows' scales
size_t ws_bytes_for(const hstu_linear_i8_params* p) {
  return kHeaderBytes + round256((size_t)p->rows * p->d_in) + round256((size_t)p->rows * sizeof(float));
}

int check(const hstu_linear_i8_params* p) {
  if (!p || p->rows < 0 || p->d_in <= 0 || p->d_out <= 0 || p->x_stride < 0 || p->out_stride < 0)
    return HSTU_ERR_INVALID_ARG;
  if ((p->dtype != HSTU_DT_BF16 && p->dtype != HSTU_DT_F32) ||
      (p->out_dtype != HSTU_DT_BF16 && p->out_dtype != HSTU_DT_F32) || (p->flags & ~HSTU_LIN_SILU))
    return HSTU_ERR_INVALID_ARG;
  if (p->rows > 0x7FFFFF00ll || p->d_in > HSTU_I8_MAX_D_IN) return HSTU_ERR_UNSUPPORTED;
  const long long xs = p->x_stride ? p->x_stride : p->d_in, os = p->out_stride ? p->out_stride : p->d_out;
  if (xs < p->d_in || os < p->d_out) return HSTU_ERR_INVALID_ARG;
  if (p->d_in % 16 || p->d_out % 8 || xs % (p->dtype == HSTU_DT_BF16 ? 8 : 4) ||
      os % (p->out_dtype == HSTU_DT_BF16 ? 8 : 4))
    return HSTU_ERR_ALIGNMENT;
  return HSTU_OK;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

size_t hstu_linear_i8_workspace_size(const hstu_linear_i8_params* p) { return check(p) == HSTU_OK ? ws_bytes_for(p) : 0; }

int hstu_quant_i8_weight(const void* w, int32_t d_in, int32_t d_out, hstu_dtype dtype, int8_t* w_q, float* w_scale,
                         hstu_stream_t stream) {
  if (d_in <= 0 || d_out <= 0 || (dtype != HSTU_DT_BF16 && dtype != HSTU_DT_F32) || !w || !w_q || !w_scale)
    return HSTU_ERR_INVALID_ARG;
  if (d_in > HSTU_I8_MAX_D_IN) return HSTU_ERR_UNSUPPORTED;
  if (d_in % 16 || d_out % 8 || !aligned16(w) || !aligned16(w_q) || !aligned16(w_scale)) return HSTU_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = (d_out + 31) / 32;
  if (dtype == HSTU_DT_BF16)
    quant_weight_kernel<<<blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), d_in, d_out, w_q, w_scale);
  else
    quant_weight_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(w), d_in, d_out, w_q, w_scale);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

int hstu_linear_i8(const hstu_linear_i8_params* p, const void* x, const int8_t* w_q, const float* w_scale,
                   const float* bias, void* out, void* workspace, size_t workspace_bytes, hstu_stream_t stream) {
  if (int rc = check(p)) return rc;
  if (p->rows == 0) return HSTU_OK;
  if (!x || !w_q || !w_scale || !out || !workspace) return HSTU_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_q) || !aligned16(w_scale) || !aligned16(bias) || !aligned16(out) ||
      !aligned16(workspace))
    return HSTU_ERR_ALIGNMENT;
  if (workspace_bytes < ws_bytes_for(p)) return HSTU_ERR_WORKSPACE;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return HSTU_ERR_CUDA;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(ws + kHeaderBytes);
  float* xscale = reinterpret_cast<float*>(ws + kHeaderBytes + round256((size_t)p->rows * p->d_in));
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  const long long xs = p->x_stride ? p->x_stride : p->d_in;
  const int blocks = (int)std::min<long long>((p->rows + 7) / 8, (long long)sms * 8);
  if (p->dtype == HSTU_DT_BF16)
    quant_rows_kernel<<<blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), p->rows, p->d_in, xs, xq, xscale, hdr);
  else
    quant_rows_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(x), p->rows, p->d_in, xs, xq, xscale, hdr);
  if (cudaGetLastError() != cudaSuccess) return HSTU_ERR_CUDA;
  GemmI8Args a;
  a.T = p->rows;
  a.K = p->d_in;
  a.N = p->d_out;
  a.out_stride = p->out_stride ? p->out_stride : p->d_out;
  a.silu = (p->flags & HSTU_LIN_SILU) ? 1 : 0;
  a.x_scale = xscale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.hdr = hdr;
  const cudaError_t e = p->out_dtype == HSTU_DT_BF16 ? launch_single<128, __nv_bfloat16>(a, xq, w_q, dev, s)
                                                     : launch_single<128, float>(a, xq, w_q, dev, s);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
