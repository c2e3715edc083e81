// Linear layer in 8-bit integers: y = act(x W + bias) with x quantised token
// by token and W channel by channel (formats in quant_common.cuh), the integer
// products summed exactly in int32 on the tensor cores (tcgen05 kind::i8).
//
//   scale_x[t] = amax_t / 127,  code[t, k] = rint(x[t, k] / scale_x[t])
//   y[t, n] = act(scale_x[t] * scale_w[n] * sum_k code[t, k] wq[n, k] + bias[n])
//
// Two launches: the rows are quantised into the workspace (one warp a row, one
// read of x), then the GEMM runs on the codes.  53,095 x 512 -> 2048 with bias and
// SiLU, bf16: 20 + 80 us (without SiLU 20 + 59); 8 rows of it 9 us, 1024 x 512 -> 512
// 12 us, both two launches' latencies.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "device_common.cuh"
#include "pair_common.cuh"
#include "hstu.h"
#include "hstu_internal.h"
#include "quant_common.cuh"

namespace hstu {
namespace {

constexpr size_t kHeaderBytes = sizeof(WsHeader);

// ---- quantise rows ------------------------------------------------------------
// A warp a row (two rows of up to 512 elements at once, so that one row's loads
// cover the other's reduction); rows of up to 1024 elements stay in registers, longer
// ones are read twice (the second time from L1 or L2).
constexpr int kRowRegs = 4;  // 4 x 256 elements

// the largest absolute value's bits (a NaN or infinity is above every finite one)
__device__ __forceinline__ uint32_t abs_bits_max(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// 8 codes as 8 bytes
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv) {
  float m[8];
  round_quotients8(x, s, inv, m);
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(m[i]);
  const uint32_t a = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  const uint32_t b = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
  return make_uint2(a, b);
}

// 8 elements as they lie
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax(uint32_t m) const {
    const uint32_t abs = 0x7FFF7FFFu;
    const uint32_t p = __vmaxu2(__vmaxu2(v.x & abs, v.y & abs), __vmaxu2(v.z & abs, v.w & abs));
    return max(m, max(p & 0xFFFF0000u, p << 16));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float x_[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, x_); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x_[i] = 0.f;
  }
  __device__ __forceinline__ uint32_t amax(uint32_t m) const { return abs_bits_max(x_, m); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x_[i];
  }
};

struct RowScale {
  float s, inv;
  bool live;
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits, float* out) {
  RowScale f;
  const bool finite = amax_bits < 0x7F800000u;
  f.s = __fdiv_rn(__uint_as_float(amax_bits), 127.f);
  f.live = finite && f.s >= FLT_MIN;
  f.inv = f.live ? 1.f / f.s : 0.f;
  if (out) *out = f.live ? f.s : (finite ? 0.f : __uint_as_float(0x7FC00000u));
  return f;
}

// R rows of a warp at once, up to 256 REGS elements of each in registers (LONG: the rest is read again)
template <typename T, int R, int REGS, bool LONG>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, long long rows, int cols,
                                                         long long x_stride, int8_t* __restrict__ xq,
                                                         float* __restrict__ scale, WsHeader* hdr) {
  if (blockIdx.x == 0 && threadIdx.x < sizeof(WsHeader) / 4) reinterpret_cast<int32_t*>(hdr)[threadIdx.x] = 0;
  const int lane = threadIdx.x & 31;
  const long long step = gridDim.x * 8ll * R;
  for (long long r0 = (blockIdx.x * 8ll + (threadIdx.x >> 5)) * R; r0 < rows; r0 += step) {
    Raw8<T> keep[R][REGS];
    uint32_t amax[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* row = x + min(r0 + i, rows - 1) * x_stride;
#pragma unroll
      for (int j = 0; j < REGS; ++j) {
        const int c = 256 * j + 8 * lane;
        if (c < cols) keep[i][j].load(row + c);
        else keep[i][j].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      amax[i] = 0;
#pragma unroll
      for (int j = 0; j < REGS; ++j) amax[i] = keep[i][j].amax(amax[i]);
      if constexpr (LONG) {
        const T* row = x + min(r0 + i, rows - 1) * x_stride;
#pragma unroll 4
        for (int c = 256 * REGS + 8 * lane; c < cols; c += 256) {
          Raw8<T> v;
          v.load(row + c);
          amax[i] = v.amax(amax[i]);
        }
      }
      amax[i] = __reduce_max_sync(~0u, amax[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r0 + i >= rows) break;
      const RowScale f = row_scale(amax[i], lane == 0 ? scale + r0 + i : nullptr);
      int8_t* out = xq + (r0 + i) * cols;
#pragma unroll
      for (int j = 0; j < REGS; ++j) {
        const int c = 256 * j + 8 * lane;
        if (c < cols) {
          float v[8];
          keep[i][j].get(v);
          *reinterpret_cast<uint2*>(out + c) = f.live ? codes8(v, f.s, f.inv) : make_uint2(0, 0);
        }
      }
      if constexpr (LONG) {
        const T* row = x + (r0 + i) * x_stride;
#pragma unroll 4
        for (int c = 256 * REGS + 8 * lane; c < cols; c += 256) {
          float v[8];
          load8(row + c, v);
          *reinterpret_cast<uint2*>(out + c) = f.live ? codes8(v, f.s, f.inv) : make_uint2(0, 0);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_quant_rows(const void* x, long long rows, int cols, long long stride, int8_t* xq, float* scale,
                              WsHeader* hdr, int sms, cudaStream_t s) {
  const T* p = static_cast<const T*>(x);
  if (cols <= 512) {
    const unsigned blocks = (unsigned)std::min<long long>((rows + 15) / 16, (long long)sms * 16);
    quant_rows_kernel<T, 2, 2, false><<<blocks, 256, 0, s>>>(p, rows, cols, stride, xq, scale, hdr);
  } else {
    const unsigned blocks = (unsigned)std::min<long long>((rows + 7) / 8, (long long)sms * 16);
    if (cols <= 256 * kRowRegs)
      quant_rows_kernel<T, 1, kRowRegs, false><<<blocks, 256, 0, s>>>(p, rows, cols, stride, xq, scale, hdr);
    else
      quant_rows_kernel<T, 1, kRowRegs, true><<<blocks, 256, 0, s>>>(p, rows, cols, stride, xq, scale, hdr);
  }
  return cudaGetLastError();
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

// SiLU for a bf16 result: x / (1 + exp(-x)) with the hardware's exponential and reciprocal,
// relative error below 2^-21 + 2^-23 |x| (0 for x < -87), far below the rounding to bf16.
// (h + h tanh h with h = x / 2 takes one such operation instead of two, but cancels for
// negative x: 2^-11 of |h| is three quarters of SiLU(-8).)  For an fp32 result the exact forms.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kMinusLog2e = -1.4426950408889634f;

template <typename TOut>
__device__ __forceinline__ float silu_i8(float x) {
  if constexpr (sizeof(TOut) == 2) return x * rcp_approx(1.f + ex2_approx(kMinusLog2e * x));
  else return x / (1.f + expf(-x));
}

// One CTA per 128 x BN output tile.  Warp 0: TMA producer; warp 1: MMA issuer
// and owner of tensor memory; warps 2-5: epilogue (thread = output row).
template <int BN, typename TOut, bool SILU>
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
            const float v = fmaf(__int2float_rn((int)acc[e + i]), xs * __ldg(a.w_scale + n + i), b);
            y[i] = SILU ? silu_i8<TOut>(v) : v;
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

// ---- GEMM on SM pairs -----------------------------------------------------------
// Large calls: the structure of gemm_sm100.cu (a cluster of two CTAs shares a
// 256 x 256 output tile, M = 256 MMAs issued by the even CTA, persistent over the
// tiles, two accumulators so that a tile's epilogue overlaps the next one's MMAs)
// with 8-bit operands, both K-major: a 128-code row is one 128-byte swizzled line,
// so a stage of 128 codes has the bytes of one of 64 bf16 and the MMAs take the
// same time for twice the K.
//
// At K = 512 the epilogue has as much to do as the tensor core: 128 x 256 sums per
// CTA and 2048 cycles of MMAs leave 8 cycles a warp row of 32, the time of one
// operation of the special-function unit.  SiLU takes two (exponential and reciprocal),
// so the int-to-float conversion, a third, is done on the other pipes: the halves of the
// int32 go into the mantissa of 2^23 (exact), 65536 hi + lo is one rounded FMA, and the
// multiplications are packed in pairs.  53,095 x 512 -> 2048 with both launches takes
// 100 us; one reciprocal for two outputs (1 / d0 = d1 / (d0 d1)) 103, -log2(e) folded
// into the scales 102, and SiLU by one tanh, which does not hold its precision below 0, 91.
// Sixteen epilogue warps (four to a scheduler, to cover their latencies) work in four
// groups of 64 columns, each with a staging box and barriers of its own.
constexpr int kPairStages = 4;
constexpr int kPairStage = kBM * kBK;   // 16 KB: this CTA's 128 rows of x, or 128 channels of w
constexpr int kPairEpiWarps = 16;      // four groups of 64 columns, a warp per 32 rows
constexpr int kPairThreads = 32 * (2 + kPairEpiWarps);
constexpr int kPairBN = 256;
constexpr int kBox = kBM * 128;         // 128 rows x 128 bytes of output

struct __align__(1024) SmemPair {
  uint8_t x[kPairStages][kPairStage];
  uint8_t w[kPairStages][kPairStage];
  uint8_t out[4][kBox];                 // a staging box for each group of 64 columns
  float wscale[4][64], bias[4][64];
  uint64_t full[kPairStages];           // even CTA: both CTAs' bytes of the stage landed
  uint64_t empty[kPairStages];          // both CTAs: the MMAs that read the stage completed
  uint64_t acc_full[2];
  uint64_t acc_empty[2];                // even CTA: both CTAs' epilogues read accumulator b
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  int issued;
};
constexpr size_t kSmemPair = sizeof(SmemPair) + 1024;
static_assert(kSmemPair <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// the 128 threads of an epilogue group agree on a flag
__device__ __forceinline__ bool group_all(bool ok, int group) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(5 + group)
      : "memory");
  return r != 0;
}

// two int32 as fp32, each rounded once: the signed upper and unsigned lower 16 bits sit
// exactly in the mantissa of 2^23
__device__ __forceinline__ uint64_t ints_to_float2(uint32_t a, uint32_t b) {
  const uint64_t hi = pack_pair(__uint_as_float(__byte_perm(a ^ 0x80000000u, 0x4B000000u, 0x7632)),
                            __uint_as_float(__byte_perm(b ^ 0x80000000u, 0x4B000000u, 0x7632)));
  const uint64_t lo = pack_pair(__uint_as_float((a & 0xFFFFu) | 0x4B000000u),
                                __uint_as_float((b & 0xFFFFu) | 0x4B000000u));
  const uint64_t h = add_pair(hi, pack_pair(-8421376.f, -8421376.f));  // 2^23 + 2^15
  return fma_pair(h, pack_pair(65536.f, 65536.f), add_pair(lo, pack_pair(-8388608.f, -8388608.f)));
}

template <typename TOut, bool SILU>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_i8_pair_kernel(const GemmI8Args a, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_out) {
  extern __shared__ uint8_t smem_raw[];
  SmemPair& sm = aligned_smem<SmemPair>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int tiles_n = (a.N + kPairBN - 1) / kPairBN;
  const int n_units = (int)((a.T + 2 * kBM - 1) / (2 * kBM)) * tiles_n;
  const int nk = (a.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * kPairEpiWarps);
    }
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    sm.issued = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem_base, 2 * kPairBN);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_out);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = pair; ok && u < n_units; u += n_pairs) {
        const int m0 = (u / tiles_n) * 2 * kBM + rank * kBM;
        const int n0 = (u % tiles_n) * kPairBN + rank * (kPairBN / 2);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % kPairStages;
          ok = mbar_wait(&sm.empty[s], ((it / kPairStages) & 1) ^ 1, abort_flag, a.hdr, 31);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(&sm.full[s], 4 * kPairStage);
          tma_load_2d_pair(sm.x[s], &tm_x, &sm.full[s], kb * kBK, m0);
          tma_load_2d_pair(sm.w[s], &tm_w, &sm.full[s], kb * kBK, n0);
          sm.issued = it + 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_i8(2 * kBM, kPairBN);
      int it = 0, tc = 0;
      bool ok = true;
      for (int u = pair; ok && u < n_units; u += n_pairs, ++tc) {
        const int b = tc & 1;
        ok = mbar_wait(&sm.acc_empty[b], ((tc >> 1) & 1) ^ 1, abort_flag, a.hdr, 32);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % kPairStages;
          ok = mbar_wait(&sm.full[s], (it / kPairStages) & 1, abort_flag, a.hdr, 33);
          if (!ok) break;
          tc_fence_after();
          const uint32_t xb = smem_u32(sm.x[s]), wb = smem_u32(sm.w[s]);
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            mma_i8_pair(tmem + b * kPairBN, sw128_desc(xb + kk * 32, 16, 1024), sw128_desc(wb + kk * 32, 16, 1024),
                        idesc, (kb | kk) != 0);
          mma_commit_pair(&sm.empty[s]);
        }
        if (ok) mma_commit_pair(&sm.acc_full[b]);
      }
      mma_commit_pair(&sm.done);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    constexpr bool kBf16 = sizeof(TOut) == 2;        // a box (128 bytes a row) holds 64 bf16 or 32 fp32 columns
    const int quarter = warp & 3, grp = (warp - 2) >> 2;
    const int te = threadIdx.x - 64 - 128 * grp;     // thread of the group
    const bool issuer = te == 0;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t empty_addr0 = map_shared(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t empty_addr1 = map_shared(smem_u32(&sm.acc_empty[1]), 0);
    float(&ws)[64] = sm.wscale[grp];
    float(&bs)[64] = sm.bias[grp];
    uint8_t* box = sm.out[grp];
    const uint32_t dst = smem_u32(box) + r * 128;
    int tc = 0;
    for (int u = pair; u < n_units; u += n_pairs, ++tc) {
      const int b = tc & 1;
      const int row0 = (u / tiles_n) * 2 * kBM + rank * kBM;
      const int n0 = (u % tiles_n) * kPairBN + 64 * grp;
      const float xs = row0 + r < a.T ? a.x_scale[row0 + r] : 0.f;
      const uint64_t xs2 = pack_pair(xs, xs);
      // the scales and biases of the group's columns (the barrier of the last tile's box is behind its reads)
      if (te < 64) {
        const int n = n0 + te;
        ws[te] = n < a.N ? __ldg(a.w_scale + n) : 0.f;
        bs[te] = n < a.N && a.bias ? __ldg(a.bias + n) : 0.f;
      }
      const bool ok = group_all(mbar_wait(&sm.acc_full[b], (tc >> 1) & 1, abort_flag, a.hdr, 34), grp);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc_tmem = tmem + lane_base + b * kPairBN + 64 * grp;
      uint32_t acc[2][32];
      tmem_ld32(acc_tmem, acc[0]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // chunks of 32 columns
        if (x == 0 || !kBf16) {
          // the last store from the box has read it
          if (issuer) bulk_wait_read();
          named_bar_sync(1 + grp, 128);
        }
        tmem_wait_ld(acc[x]);
        if (x == 0) {
          tmem_ld32(acc_tmem + 32, acc[1]);
        } else {
          // this warp's part of accumulator b is read: tell the even CTA's issuer
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(b ? empty_addr1 : empty_addr0);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const float4 wv = *reinterpret_cast<const float4*>(&ws[32 * x + e + k]);
            const float4 bv = *reinterpret_cast<const float4*>(&bs[32 * x + e + k]);
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              const uint32_t i0 = acc[x][e + k + q], i1 = acc[x][e + k + q + 1];
              // without SiLU the special-function unit is free for the conversion
              const uint64_t f2 =
                  SILU ? ints_to_float2(i0, i1) : pack_pair(__int2float_rn((int)i0), __int2float_rn((int)i1));
              const uint64_t v2 = fma_pair(f2, mul_pair(xs2, q ? pack_pair(wv.z, wv.w) : pack_pair(wv.x, wv.y)),
                                       q ? pack_pair(bv.z, bv.w) : pack_pair(bv.x, bv.y));
              float v0, v1;
              unpack_pair(v2, v0, v1);
              if constexpr (SILU && kBf16) {
                float n0, n1, d0, d1;
                unpack_pair(mul_pair(v2, pack_pair(kMinusLog2e, kMinusLog2e)), n0, n1);
                unpack_pair(add_pair(pack_pair(ex2_approx(n0), ex2_approx(n1)), pack_pair(1.f, 1.f)), d0, d1);
                unpack_pair(mul_pair(v2, pack_pair(rcp_approx(d0), rcp_approx(d1))), y[k + q], y[k + q + 1]);
              } else {
                y[k + q] = SILU ? silu_i8<TOut>(v0) : v0;
                y[k + q + 1] = SILU ? silu_i8<TOut>(v1) : v1;
              }
            }
          }
          // 16-byte chunk j of the box row at j ^ (r & 7) (the store's 128-byte swizzle)
          const int j0 = (kBf16 ? 32 * x : 0) + e;
          if constexpr (kBf16) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (((j0 / 8) ^ (r & 7)) << 4)),
                         "r"(pack_bf16x2(y[0], y[1])), "r"(pack_bf16x2(y[2], y[3])), "r"(pack_bf16x2(y[4], y[5])),
                         "r"(pack_bf16x2(y[6], y[7]))
                         : "memory");
          } else {
#pragma unroll
            for (int k = 0; k < 8; k += 4)
              asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(dst + ((((j0 + k) / 4) ^ (r & 7)) << 4)),
                           "f"(y[k]), "f"(y[k + 1]), "f"(y[k + 2]), "f"(y[k + 3])
                           : "memory");
          }
        }
        if (x == 1 || !kBf16) {
          fence_proxy_async_smem();
          named_bar_sync(1 + grp, 128);
          if (issuer) {
            const int c = n0 + (kBf16 ? 0 : 32 * x);
            if (c < a.N && row0 < a.T) tma_store_2d(&tm_out, box, c, row0);  // rows and columns outside are dropped
            bulk_commit();
          }
        }
      }
    }
    if (issuer) bulk_wait_all();
  }

  // as in gemm_sm100.cu: every MMA completed and every copy into either CTA is
  // accounted for before tensor memory is freed and either CTA exits
  if (warp == 1 && lane == 0) mbar_wait(&sm.done, 0, nullptr, a.hdr, 38);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (leader && warp == 0 && lane == 0) {
    const int mine = sm.issued;
    const int peer = (int)ld_shared_cluster_u32(map_shared(smem_u32(&sm.issued), 1));
    const int last = max(mine, peer);
    for (int t = max(0, last - kPairStages); t < last; ++t) {
      uint64_t* bar = &sm.full[t % kPairStages];
      if (t < mine && t >= peer) mbar_complete_tx(bar, 2 * kPairStage);
      if (t >= mine && t < peer) mbar_arrive_expect_tx(bar, 2 * kPairStage);
      mbar_wait(bar, (t / kPairStages) & 1, nullptr, a.hdr, 39);
    }
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * kPairBN);
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

long long pair_units(long long T, int N) { return ((T + 2 * kBM - 1) / (2 * kBM)) * ((N + kPairBN - 1) / kPairBN); }

template <int BN, typename TOut, bool SILU>
cudaError_t launch_single(const GemmI8Args& a, const void* xq, const void* wq, int dev, cudaStream_t s) {
  constexpr size_t smem = sizeof(SmemI8<BN>) + 1024;
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(gemm_i8_kernel<BN, TOut, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  CUtensorMap tx, tw;
  if (!encode_codes(&tx, xq, a.T, a.K, kBM) || !encode_codes(&tw, wq, a.N, a.K, BN)) return cudaErrorInvalidValue;
  const long long tiles = ((a.T + kBM - 1) / kBM) * ((a.N + BN - 1) / BN);
  gemm_i8_kernel<BN, TOut, SILU><<<(unsigned)tiles, kThreads, smem, s>>>(a, tx, tw);
  return cudaGetLastError();
}

// out [rows, N] with a row stride: box = 128 rows x 128 bytes, 128B swizzle
bool encode_out(CUtensorMap* m, void* base, long long rows, int N, long long stride, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int es = bf16 ? 2 : 4;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(stride * es)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)kBM};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TOut, bool SILU>
cudaError_t launch_pair(const GemmI8Args& a, const void* xq, const void* wq, int dev, int sms, cudaStream_t s) {
  static unsigned long long attr_set = 0;  // one bit per device
  if (!(attr_set & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(gemm_i8_pair_kernel<TOut, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemPair);
    if (e != cudaSuccess) return e;
    attr_set |= 1ull << dev;
  }
  CUtensorMap tx, tw, to;
  if (!encode_codes(&tx, xq, a.T, a.K, kBM) || !encode_codes(&tw, wq, a.N, a.K, kBM) ||
      !encode_out(&to, a.out, a.T, a.N, a.out_stride, sizeof(TOut) == 2))
    return cudaErrorInvalidValue;
  const long long units = pair_units(a.T, a.N);
  const int pairs = (int)std::max<long long>(1, std::min<long long>(units, sms / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kSmemPair;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_i8_pair_kernel<TOut, SILU>, a, tx, tw, to);
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

size_t hstu_linear_i8_workspace_size(const hstu_linear_i8_params* p) {
  return check(p) == HSTU_OK ? ws_bytes_for(p) : 0;
}

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
  if ((p->dtype == HSTU_DT_BF16 ? launch_quant_rows<__nv_bfloat16>(x, p->rows, p->d_in, xs, xq, xscale, hdr, sms, s)
                                : launch_quant_rows<float>(x, p->rows, p->d_in, xs, xq, xscale, hdr, sms, s)) !=
      cudaSuccess)
    return HSTU_ERR_CUDA;
  GemmI8Args a;
  a.T = p->rows;
  a.K = p->d_in;
  a.N = p->d_out;
  a.out_stride = p->out_stride ? p->out_stride : p->d_out;
  const bool silu = (p->flags & HSTU_LIN_SILU) != 0;
  a.x_scale = xscale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.hdr = hdr;
  // 128 x 128 tiles on single SMs while one wave of them does; 256 x 256 tiles on SM
  // pairs, persistent, above.  Single against pairs in us (with the quantisation of x; bf16,
  // with SiLU): rows x d_in x d_out 700 x 208 x 40 7.7 / 10.7, 8 x 512 x 2048 10.8 / 11.3,
  // 1024 x 512 x 2048 (128 tiles) 13.8 / 13.3, 2048 x 512 x 2048 (256) 23.2 / 13.8,
  // 16384 x 512 x 512 (512) 44 / 21.
  const long long single_tiles = ((p->rows + kBM - 1) / kBM) * ((p->d_out + 127) / 128);
  const bool bf16 = p->out_dtype == HSTU_DT_BF16;
  cudaError_t e;
  if (single_tiles > sms)
    e = bf16 ? (silu ? launch_pair<__nv_bfloat16, true>(a, xq, w_q, dev, sms, s)
                     : launch_pair<__nv_bfloat16, false>(a, xq, w_q, dev, sms, s))
             : (silu ? launch_pair<float, true>(a, xq, w_q, dev, sms, s)
                     : launch_pair<float, false>(a, xq, w_q, dev, sms, s));
  else
    e = bf16 ? (silu ? launch_single<128, __nv_bfloat16, true>(a, xq, w_q, dev, s)
                     : launch_single<128, __nv_bfloat16, false>(a, xq, w_q, dev, s))
             : (silu ? launch_single<128, float, true>(a, xq, w_q, dev, s)
                     : launch_single<128, float, false>(a, xq, w_q, dev, s));
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
