// rope.cu -- rotary positions on the query and key heads of a projection's rows.
//
// Pair i of a head (i < rot / 2) is turned by the angle 2 pi frac(pos f_i), f_i in
// turns per position (fp64, made once by qk_rope_frequencies):
//     y_a = x_a c - x_b s,   y_b = x_b c + x_a s,   (c, s) = amplitude (cos, sin)
// a, b = i, i + rot / 2 (half layout) or 2 i, 2 i + 1 (interleaved); the rest of
// the head is copied.  pos f_i is taken in fp64 and only its fractional part goes
// on to fp32: at position 2^30 the angle is still good to 2^-22 turns, where a
// product in fp32 would keep none of its fraction.
//
// Bound: HBM, 2 bytes read and 2 written per element.  A block turns the heads
// of one or more tokens: it makes the tokens' rot / 2 angles once, in shared
// memory, and every head reads them there.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qk_internal.h"
#include "sm100.cuh"

namespace qk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 1024;  // angles a block keeps (tokens per block x rot / 2)

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

struct RopeArgs {
  const uint16_t* in[2];  // q, k
  uint16_t* out[2];
  long long in_stride[2], out_stride[2];  // elements between tokens
  int heads[2];
  int T, D, rot, tokens;  // tokens per block
  const int32_t* positions;
  const double* freq;
  float amplitude;
};

// kVec: 16-byte chunks (half layout: rot % 16 == 0, interleaved: rot % 8 == 0);
// otherwise one pair or one copied element per step.
template <bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  const int half = p.rot >> 1;
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half;
    const double turns = (double)__ldg(p.positions + t0 + tok) * __ldg(p.freq + f);
    const float frac = (float)(turns - rint(turns));  // [-1/2, 1/2]
    float s, c;
    sincospif(2.0f * frac, &s, &c);
    cs[i] = c * p.amplitude;
    sn[i] = s * p.amplitude;
  }
  __syncthreads();
  const int rotated = kVec ? (kHalf ? p.rot >> 4 : p.rot >> 3) : half;
  const int copied = kVec ? (p.D - p.rot) >> 3 : p.D - p.rot;
  const int per_head = rotated + copied;
  const int heads = p.heads[0] + p.heads[1];
  const int per_token = heads * per_head;
  for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
    const int tok = i / per_token, rest = i - tok * per_token;
    int hd = rest / per_head;
    const int e = rest - hd * per_head;
    const int which = hd >= p.heads[0];
    if (which) hd -= p.heads[0];
    const uint16_t* src = p.in[which] + (t0 + tok) * p.in_stride[which] + (long long)hd * p.D;
    uint16_t* dst = p.out[which] + (t0 + tok) * p.out_stride[which] + (long long)hd * p.D;
    const float* c = cs + tok * half;
    const float* s = sn + tok * half;
    if (e >= rotated) {  // behind the rotated part
      if (src == dst) continue;
      if constexpr (kVec)
        *reinterpret_cast<uint4*>(dst + p.rot + 8 * (e - rotated)) =
            *reinterpret_cast<const uint4*>(src + p.rot + 8 * (e - rotated));
      else
        dst[p.rot + e - rotated] = src[p.rot + e - rotated];
    } else if constexpr (kVec && kHalf) {
      const uint4 a4 = *reinterpret_cast<const uint4*>(src + 8 * e);
      const uint4 b4 = *reinterpret_cast<const uint4*>(src + half + 8 * e);
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
      uint32_t u[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c0 = c[8 * e + 2 * j], c1 = c[8 * e + 2 * j + 1];
        const float s0 = s[8 * e + 2 * j], s1 = s[8 * e + 2 * j + 1];
        u[j] = pack16(lo16(a[j]) * c0 - lo16(b[j]) * s0, hi16(a[j]) * c1 - hi16(b[j]) * s1);
        v[j] = pack16(lo16(b[j]) * c0 + lo16(a[j]) * s0, hi16(b[j]) * c1 + hi16(a[j]) * s1);
      }
      *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(dst + half + 8 * e) = make_uint4(v[0], v[1], v[2], v[3]);
    } else if constexpr (kVec) {
      const uint4 a4 = *reinterpret_cast<const uint4*>(src + 8 * e);
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w};
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c0 = c[4 * e + j], s0 = s[4 * e + j];
        u[j] = pack16(lo16(a[j]) * c0 - hi16(a[j]) * s0, hi16(a[j]) * c0 + lo16(a[j]) * s0);
      }
      *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      const int ia = kHalf ? e : 2 * e, ib = kHalf ? e + half : 2 * e + 1;
      const float a = lo16(src[ia]), b = lo16(src[ib]);
      const uint32_t r = pack16(a * c[e] - b * s[e], b * c[e] + a * s[e]);
      dst[ia] = (uint16_t)r;
      dst[ib] = (uint16_t)(r >> 16);
    }
  }
}

// Turns per position of every pair; see include/qk.h for the scalings.
__global__ void rope_freq_kernel(int rot, double base, int scaling, double factor, double trained,
                                 double slow, double fast, double* freq) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rot / 2) return;
  if (scaling == QK_ROPE_NTK && rot > 2)
    base *= pow(factor, (double)rot / (double)(rot - 2));
  const double turn = 6.283185307179586476925286766559;
  double f = pow(base, -2.0 * (double)i / (double)rot) / turn;
  if (scaling == QK_ROPE_LINEAR) f /= factor;
  if (scaling == QK_ROPE_BY_PARTS) {
    // turns over the trained length: many -> kept, few -> stretched by factor
    const double keep = fmin(1.0, fmax(0.0, (trained * f - slow) / (fast - slow)));
    f = f * keep + f / factor * (1.0 - keep);
  }
  freq[i] = f;
}

}  // namespace

cudaError_t launch_rope(const uint16_t* q, int64_t q_stride, uint16_t* q_out, int64_t q_out_stride,
                        int64_t H, const uint16_t* k, int64_t k_stride, uint16_t* k_out,
                        int64_t k_out_stride, int64_t Hkv, int64_t T, int64_t D, int64_t rot,
                        bool half, const int32_t* positions, const double* freq, float amplitude,
                        cudaStream_t s) {
  RopeArgs a = {};
  a.in[0] = q; a.in[1] = k;
  a.out[0] = q_out; a.out[1] = k_out;
  a.in_stride[0] = q_stride; a.in_stride[1] = k_stride;
  a.out_stride[0] = q_out_stride; a.out_stride[1] = k_out_stride;
  a.heads[0] = (int)H;
  a.heads[1] = k != nullptr ? (int)Hkv : 0;
  a.T = (int)T; a.D = (int)D; a.rot = (int)rot;
  a.positions = positions; a.freq = freq; a.amplitude = amplitude;
  // several tokens per block where one token's heads do not fill it, as long as
  // their angles fit and every SM keeps a block
  const int64_t steps = (H + a.heads[1]) * (D / 16);
  int64_t tokens = 1;
  while (tokens < 16 && tokens * steps < 2 * kThreads && 2 * tokens * (rot / 2) <= kMaxPairs &&
         T / (2 * tokens) >= num_sms())
    tokens *= 2;
  a.tokens = (int)tokens;
  const bool vec = half ? rot % 16 == 0 : rot % 8 == 0;
  void (*kernel)(RopeArgs) = half ? (vec ? rope_kernel<true, true> : rope_kernel<true, false>)
                                  : (vec ? rope_kernel<false, true> : rope_kernel<false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((T + tokens - 1) / tokens));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_rope_frequencies(int64_t rot, double base, int scaling, double factor,
                                    double trained, double slow, double fast, double* freq,
                                    cudaStream_t s) {
  const int n = (int)(rot / 2);
  rope_freq_kernel<<<(n + 127) / 128, 128, 0, s>>>((int)rot, base, scaling, factor, trained, slow,
                                                  fast, freq);
  return cudaGetLastError();
}

}  // namespace qk
