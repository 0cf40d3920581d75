// norm_quant.cu -- RMS norm with the residual's addition, written as the int8
// codes, scales and group sums that the quantized products read.
//
// Per row m, with n = K elements:
//     h     = bf16(x + residual)               (x itself without a residual)
//     u_k   = fl32(h_k w_k)                    (h_k without a weight)
//     U     = max_k |u_k|
//     code  = rne(fl32(u_k fl32(127 fl32(1 / U)))), clamped to [-127, 127]
//     sx    = fl32(fl32(U / 127) rstd),  rstd = 1 / sqrt(sum_k h_k^2 / n + eps)
//     xsum  = sums of 64 codes                 (when asked for)
// A NaN among the u_k makes U, and so sx, NaN (and the codes 0), as in act_quant.cuh.
// The row's 1 / rms multiplies every element alike, so it cancels in the codes
// (|u| / U has no rms in it) and goes into the scale: one pass over the row
// decides every code from u, as act_quant.cuh does from x (with the multiplier from
// the reciprocal: below), and no rounding of the sum of squares can move a code.  code sx
// is the quantized h rstd w.
//
// Bound: HBM.  2 (x) + 2 (residual) + 2 (h) + 1 (codes) bytes per element, each
// touched once: u stays in fp32 registers between the maximum and the codes.
// 16384 rows of 4096: 75.2 us, 96 % of the copy rate; 1111 rows of 5120: 9.9 us (61 %: a row
// to a block and five blocks to an SM, 740 of the 1111 at once, each a load, a reduction and a
// store long, and a sixth of the threads' places for chunks empty); one row 2.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act_quant.cuh"
#include "qk_internal.h"
#include "sm100.cuh"

namespace qk {
namespace {

constexpr int kWarps = 8;  // per block

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// bf16(a + b) of two packed pairs.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __floats2bfloat162_rn(bf_lo(a) + bf_lo(b), bf_hi(a) + bf_hi(b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The largest magnitude, NaN where one is: a row's NaN has to reach its scale.
__device__ __forceinline__ float max_nan(float a, float b, float c = 0.0f) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint4 add_chunk(uint4 a, uint4 b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                    add_bf16x2(a.w, b.w));
}

// u = h w of one chunk (8 elements); adds the squares of h and takes the maximum of |u|.
__device__ __forceinline__ void weigh(uint4 h, const float* __restrict__ weight, int c, float (&u)[8],
                                      float* ssq, float* top) {
  const uint32_t p[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[2 * i] = bf_lo(p[i]);
    u[2 * i + 1] = bf_hi(p[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) *ssq = fmaf(u[i], u[i], *ssq);
  if (weight != nullptr) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + 2 * c);
    const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + 2 * c + 1);
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __fmul_rn(u[i], w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) *top = max_nan(*top, u[i], u[i + 1]);
}

__device__ __forceinline__ uint2 code_chunk(const float (&u)[8], float r, int* sum) {
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int q = quant1(u[i], r);
    *sum += q;
    out[i >> 2] |= (uint32_t)(q & 0xFF) << (8 * (i & 3));
  }
  return make_uint2(out[0], out[1]);
}

// Two roundings (the header's rule), where act_multiplier has one.  Either is within 2^-23 of
// 127 / U, and a code within 1/2 + 2^-15 of u 127 / U: the two rules' codes differ, by one, only
// for values that close to halfway between two codes.
__device__ __forceinline__ float norm_multiplier(float top) {
  return top == 0.0f ? 0.0f : __fmul_rn(127.0f, __fdiv_rn(1.0f, top));
}

__device__ __forceinline__ float norm_scale(float top, float ssq, int K, float eps) {
  if (top == 0.0f) return 1.0f;
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ssq, (float)K) + eps));
  return __fmul_rn(act_scale(top), rstd);
}

// WPR warps share a row (kWarps / WPR rows per block); a thread holds CPT chunks
// of 8 elements.  CPT == 0: rows longer than 8 * 256 * 8 elements, read twice
// (the second time h, from where this thread wrote it, or x).
//
// Blocks per SM: what the registers of the chunks allow.  (A row of three chunks and eight warps
// would take 50, four blocks: 1111 rows of 5120, in L2, 8.8 us; in 48, five blocks and a spilled
// pointer, 8.7, and 8.5 by a maximum that drops NaN.)
constexpr int resident(int cpt) { return cpt == 8 ? 2 : cpt == 6 ? 3 : cpt == 4 ? 4 : cpt == 3 ? 5 : 6; }

template <int WPR, int CPT>
__global__ void __launch_bounds__(32 * kWarps, resident(CPT))
    norm_quant_kernel(const uint16_t* x, const uint16_t* residual, int M, int K,
                      const float* __restrict__ weight, float eps, uint16_t* h, int8_t* xq,
                      float* sx, int32_t* xsum) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int T = 32 * WPR;
  __shared__ float red_top[kWarps], red_ssq[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kWarps / WPR) + warp / WPR;
  const int t = (warp % WPR) * 32 + lane;
  const bool live = row < M;
  const int nch = live ? K >> 3 : 0;
  const size_t at = (size_t)(live ? row : 0) * (size_t)K;
  const uint4* px = reinterpret_cast<const uint4*>(x + at);
  const uint4* pr = reinterpret_cast<const uint4*>(residual + at);
  uint4* ph = reinterpret_cast<uint4*>(h + at);
  uint2* pq = reinterpret_cast<uint2*>(xq + at);
  const bool add = residual != nullptr;
  float ssq = 0.0f, top = 0.0f;
  constexpr int N = CPT > 0 ? CPT : 1;
  float u[N][8];
  if constexpr (CPT > 0) {
    uint4 v[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * T + t;
      if (c < nch) {
        v[i] = __ldcs(px + c);
        if (add) r[i] = __ldcs(pr + c);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * T + t;
      if (c < nch) {
        if (add) {
          v[i] = add_chunk(v[i], r[i]);
          ph[c] = v[i];
        }
        weigh(v[i], weight, c, u[i], &ssq, &top);
      }
    }
  } else {
    for (int c = t; c < nch; c += T) {
      uint4 v = px[c];
      if (add) {
        v = add_chunk(v, pr[c]);
        ph[c] = v;
      }
      weigh(v, weight, c, u[0], &ssq, &top);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ssq += __shfl_xor_sync(0xFFFFFFFFu, ssq, o);
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      red_top[warp] = top;
      red_ssq[warp] = ssq;
    }
    __syncthreads();
    ssq = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      ssq += red_ssq[(warp / WPR) * WPR + w];
      top = max_nan(top, red_top[(warp / WPR) * WPR + w]);
    }
  }
  if (!live) return;
  const float r = norm_multiplier(top);
  if (t == 0) sx[row] = norm_scale(top, ssq, K, eps);
  const int G = K >> 6;
  auto put = [&](int c, const float (&w)[8]) {
    int s = 0;
    if (c < nch) pq[c] = code_chunk(w, r, &s);
    if (xsum != nullptr) {
      s = group8_sum(s);
      if ((lane & 7) == 0 && c < nch) xsum[(size_t)row * G + (c >> 3)] = s;
    }
  };
  if constexpr (CPT > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * T + (t & ~31) < nch) put(i * T + t, u[i]);  // warp-uniform
  } else {
    float a = 0.0f, b = 0.0f;
    for (int c0 = t & ~31; c0 < nch; c0 += T) {
      const int c = c0 + lane;
      if (c < nch) weigh(add ? ph[c] : px[c], weight, c, u[0], &a, &b);
      put(c, u[0]);
    }
  }
}

}  // namespace

cudaError_t launch_norm_quant(const uint16_t* x, const uint16_t* residual, int64_t M, int64_t K,
                              const float* weight, float eps, uint16_t* h, int8_t* xq, float* sx,
                              int32_t* xsum, cudaStream_t s) {
  using Kern = void (*)(const uint16_t*, const uint16_t*, int, int, const float*, float, uint16_t*,
                        int8_t*, float*, int32_t*);
  const int nch = (int)(K / 8);
  // Few rows (at most one block per SM): a whole block per row.  Otherwise the
  // fewest warps per row that leave at most four chunks to a thread.
  int wpr = 8;
  if (M > num_sms())
    while (wpr > 1 && nch <= 32 * (wpr / 2) * 4) wpr >>= 1;
  const int cpt = (nch + 32 * wpr - 1) / (32 * wpr);
  Kern kernel;
  switch (wpr) {
    case 1: kernel = cpt <= 1 ? norm_quant_kernel<1, 1> : cpt <= 2 ? norm_quant_kernel<1, 2> : cpt <= 3 ? norm_quant_kernel<1, 3> : norm_quant_kernel<1, 4>; break;
    case 2: kernel = cpt <= 3 ? norm_quant_kernel<2, 3> : norm_quant_kernel<2, 4>; break;
    case 4: kernel = cpt <= 3 ? norm_quant_kernel<4, 3> : norm_quant_kernel<4, 4>; break;
    default:
      kernel = cpt <= 1   ? norm_quant_kernel<8, 1>
               : cpt <= 2 ? norm_quant_kernel<8, 2>
               : cpt <= 3 ? norm_quant_kernel<8, 3>
               : cpt <= 4 ? norm_quant_kernel<8, 4>
               : cpt <= 6 ? norm_quant_kernel<8, 6>
               : cpt <= 8 ? norm_quant_kernel<8, 8>
                          : norm_quant_kernel<8, 0>;
  }
  cudaLaunchConfig_t cfg = {};
  const int rows = kWarps / wpr;
  cfg.gridDim = dim3((unsigned)((M + rows - 1) / rows));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, x, residual, (int)M, (int)K, weight, eps, h, xq, sx, xsum);
}

}  // namespace qk
