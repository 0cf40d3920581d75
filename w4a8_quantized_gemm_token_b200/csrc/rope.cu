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
// memory, and every head reads them there.  14040 tokens of 48 heads of 128, 32
// dims rotated in pairs: 61 us, 86 % of the copy rate (one chunk at a time 81 us; four or six
// blocks per SM instead of five 64 and 66); all 128 in halves 59 us, in pairs 62; 32 in halves
// 70 us (75 %: two steps are in flight there, and one that is copied loads one chunk).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fast_div.cuh"
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
  int T, D, rot, tokens;       // tokens per block
  FastDiv per_token, per_head;  // steps of a token; of a head
  FastDiv turned, copied;       // of a head: rotated steps; copied ones (kVec)
  const int32_t* positions;
  const double* freq;
  float amplitude;
};

// kVec: 16-byte chunks (half layout: rot % 16 == 0, interleaved: rot % 8 == 0), with
// kUnroll steps' loads of a thread in flight, the first ones before the angles are
// made; otherwise one pair or one copied element per step.
constexpr int unroll(bool half) { return half ? 2 : 4; }  // (a step of the half layout loads two chunks)

template <bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const RopeArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  const int half = p.rot >> 1;
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  auto angles = [&]() {
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
  };
  const int steps = nt * p.per_token.d;
  if constexpr (kVec) {
    // a token's steps: every head's rotated chunks, then every head's others, so that few
    // warps have both
    constexpr int U = unroll(kHalf);
    auto row = [&](auto* const (&base)[2], const long long (&stride)[2], int which, int tok) {
      return which ? base[1] + (t0 + tok) * stride[1] : base[0] + (t0 + tok) * stride[0];
    };
    const int nturned = p.turned.d * (p.heads[0] + p.heads[1]);
    for (int base = 0; base < steps; base += U * kThreads) {
      int where[U];  // element of the token's heads, the token << 26, in k << 30
      int angle[U];  // the chunk's first; -1: a copied chunk
      uint4 a4[U], b4[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int i = base + u * kThreads + threadIdx.x;
        if (i >= steps) continue;
        int tok = 0, hd, at;
        if (p.tokens > 1) {
          tok = quot(i, p.per_token);
          i -= tok * p.per_token.d;
        }
        if (i < nturned) {
          hd = quot(i, p.turned);
          const int e = i - hd * p.turned.d;
          at = 8 * e;
          angle[u] = tok * half + (kHalf ? 8 : 4) * e;
        } else {
          i -= nturned;
          hd = quot(i, p.copied);
          at = p.rot + 8 * (i - hd * p.copied.d);
          angle[u] = -1;
        }
        const int which = hd >= p.heads[0];
        if (which) hd -= p.heads[0];
        at += hd * p.D;
        where[u] = at | tok << 26 | which << 30;
        const uint16_t* src = row(p.in, p.in_stride, which, tok) + at;
        a4[u] = __ldcs(reinterpret_cast<const uint4*>(src));
        if (kHalf && angle[u] >= 0) b4[u] = __ldcs(reinterpret_cast<const uint4*>(src + half));
      }
      if (base == 0) angles();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (base + u * kThreads + threadIdx.x >= steps) continue;
        const int which = where[u] >> 30, tok = where[u] >> 26 & 15;
        uint16_t* dst = row(p.out, p.out_stride, which, tok) + (where[u] & ((1 << 26) - 1));
        if (angle[u] < 0) {
          if (p.in[which] != p.out[which]) *reinterpret_cast<uint4*>(dst) = a4[u];
          continue;
        }
        const uint32_t a[4] = {a4[u].x, a4[u].y, a4[u].z, a4[u].w};
        uint32_t x[4];
        if constexpr (kHalf) {
          const float4* c = reinterpret_cast<const float4*>(cs + angle[u]);
          const float4* s = reinterpret_cast<const float4*>(sn + angle[u]);
          const uint32_t b[4] = {b4[u].x, b4[u].y, b4[u].z, b4[u].w};
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 cc = c[j], ss = s[j];
            const uint32_t a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
            x[2 * j] = pack16(lo16(a0) * cc.x - lo16(b0) * ss.x, hi16(a0) * cc.y - hi16(b0) * ss.y);
            x[2 * j + 1] = pack16(lo16(a1) * cc.z - lo16(b1) * ss.z, hi16(a1) * cc.w - hi16(b1) * ss.w);
            y[2 * j] = pack16(lo16(b0) * cc.x + lo16(a0) * ss.x, hi16(b0) * cc.y + hi16(a0) * ss.y);
            y[2 * j + 1] = pack16(lo16(b1) * cc.z + lo16(a1) * ss.z, hi16(b1) * cc.w + hi16(a1) * ss.w);
          }
          *reinterpret_cast<uint4*>(dst + half) = make_uint4(y[0], y[1], y[2], y[3]);
        } else {
          const float4 cc = *reinterpret_cast<const float4*>(cs + angle[u]);
          const float4 ss = *reinterpret_cast<const float4*>(sn + angle[u]);
          const float c[4] = {cc.x, cc.y, cc.z, cc.w}, s[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = pack16(lo16(a[j]) * c[j] - hi16(a[j]) * s[j], hi16(a[j]) * c[j] + lo16(a[j]) * s[j]);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  } else {
    angles();
    for (int i = threadIdx.x; i < steps; i += kThreads) {
      const int tok = quot(i, p.per_token), rest = i - tok * p.per_token.d;
      int hd = quot(rest, p.per_head);
      const int e = rest - hd * p.per_head.d;
      const int which = hd >= p.heads[0];
      if (which) hd -= p.heads[0];
      const uint16_t* src = p.in[which] + (t0 + tok) * p.in_stride[which] + hd * p.D;
      uint16_t* dst = p.out[which] + (t0 + tok) * p.out_stride[which] + hd * p.D;
      if (e >= half) {
        const int at = p.rot + e - half;
        if (src != dst) dst[at] = src[at];
        continue;
      }
      const int ia = kHalf ? e : 2 * e, ib = kHalf ? e + half : 2 * e + 1;
      const float a = lo16(src[ia]), b = lo16(src[ib]);
      const float c = cs[tok * half + e], s = sn[tok * half + e];
      const uint32_t y = pack16(a * c - b * s, b * c + a * s);
      dst[ia] = (uint16_t)y;
      dst[ib] = (uint16_t)(y >> 16);
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
  const bool vec = half ? rot % 16 == 0 : rot % 8 == 0;
  const int turned = (int)(vec ? (half ? rot / 16 : rot / 8) : rot / 2);
  const int copied = (int)(vec ? (D - rot) / 8 : D - rot), per_head = turned + copied;
  a.turned = fast_div(turned);
  a.copied = fast_div(copied > 0 ? copied : 1);
  a.per_head = fast_div(per_head);
  a.per_token = fast_div(per_head * (a.heads[0] + a.heads[1]));
  // as many tokens per block as one pass of its threads holds, as long as their angles
  // fit and every SM keeps a block
  int64_t tokens = 1;
  while (tokens < 16 && 2 * tokens * a.per_token.d <= unroll(half) * kThreads &&
         2 * tokens * (rot / 2) <= kMaxPairs && T / (2 * tokens) >= num_sms())
    tokens *= 2;
  a.tokens = (int)tokens;
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
