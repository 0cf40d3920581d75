// kv4_cache.cu -- writing tokens into the 4-bit key/value cache, and reading them
// back as bf16.
//
// Per token, kv head and group of 64 dims, the affine rule of the W4 weights:
//     s = fp16((max - min) / 15), o = fp16(min),
//     code = rne(clamp((w - o) fl32(1 / s), 0, 15))   (0 where s = 0),
// fp32 arithmetic, one rounding per operation; the value is code s + o.
//
// Bound: HBM (4 D bytes of bf16 and 9 D / 8 of record per token and head).  Eight
// lanes hold a group (16 bytes each); the request of a row is found by a 32-way
// search over the row bounds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fast_div.cuh"
#include "kv4.cuh"
#include "sm100.cuh"

namespace qk {
namespace {

constexpr int kThreads = 128;

// The request that row belongs to, by the whole warp (B when it is behind the
// last one): the number of bounds cu[1 .. B] that are <= row, narrowed 32-fold a step.
__device__ __forceinline__ int find_request(const Kv4Req& r, int row) {
  if (r.cu == nullptr) return row / (r.T / r.B);
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = r.B;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + (lane + 1) * step;  // candidates lo + step, lo + 2 step, ...
    const bool below = i <= hi && __ldg(r.cu + i) <= row;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, below));
    lo += c * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Where a row of the call lives.
struct Place {
  long long at;  // byte offset of its record, for kv head 0
  int in;        // its token in the record; -1: nowhere (recorded); -2: nobody's row
};

// Of the warp's rows first .. first + n - 1 (n <= 32), lane r's: the rows of one
// request find it together, and every row's page is looked up at the same time.
__device__ __forceinline__ Place find_tokens(const Kv4Req& r, const Kv4Cache& c, const FastDiv& by_page,
                                             int first, int n, int rec, int* err) {
  const int lane = threadIdx.x & 31, row = first + lane;
  Place p = {0, -2};
  uint32_t todo = 0xFFFFFFFFu >> (32 - n);
  while (todo) {
    const int lead = first + __ffs(todo) - 1;
    const int b = find_request(r, lead);
    if (b >= r.B) break;  // behind the last request, and so are the rows that follow
    const Kv4Seq s = kv4_seq(r, b, err);
    // (row bounds that fall may leave the leading row outside of its request)
    const bool mine = (todo >> lane & 1u) && (row == lead || (row >= s.row0 && row < s.row0 + s.n));
    if (mine && row >= s.row0) {
      const int pos = s.len - s.n + (row - s.row0);
      p.in = -1;
      if (pos < 0 || row >= s.row0 + s.n) {  // no such token
        record_index(err);
      } else {
        const int pg = quot(pos, by_page);
        const int id = __ldg(r.page_table + (long long)b * r.max_pages + pg);
        if (id < 0 || id >= c.num_pages) {
          record_index(err);
        } else {
          const int off = pos - pg * c.page;
          p.at = ((long long)id * c.Hkv * (c.page >> 4) + (off >> 4)) * rec;
          p.in = off & 15;
        }
      }
    }
    todo &= ~__ballot_sync(0xFFFFFFFFu, mine);
  }
  return p;
}

// A warp takes a run of rows (as many as leave every SM its warps) and blockIdx.y
// picks kHeads steps of 32 / LANES heads: the rows' places are looked up together, a
// lane to a row, the loads of a row's steps are in flight at once and those of the next
// row while it is worked on, and what is computed per group (extremes, scale,
// reciprocal) is computed for the four steps together, a lane to a step.  10144 rows of 8
// heads of 128 dims: a row to a warp and head after head 21 us, four heads at once 17.5
// us, runs of 5 rows 16 us (read back: 22, 18, 15 us).
constexpr int kHeads = 4;

template <int D>
struct Lane {
  using L = Kv4<D>;
  static constexpr int LANES = D / 4;         // of one token and head: K row, then V row
  static constexpr int STEP = 32 / LANES;     // heads at a time
  int sub, d8, grp, w8;                       // head of the step; chunk of 8 dims, its group, place
  bool is_v;
  __device__ __forceinline__ Lane() {
    const int lane = threadIdx.x & 31, e = lane % LANES;
    sub = lane / LANES;
    is_v = e >= LANES / 2;
    d8 = e % (LANES / 2);
    grp = d8 >> 3;
    w8 = d8 & 7;
  }
  // byte offsets in a record, for the token at `place`
  __device__ __forceinline__ int code(int place) const {
    return is_v ? L::V_OFF + (((place >> 1) * 8 + w8) * L::NG + grp) * 8 + (place & 1) * 2
                : place * (D / 2) + (((w8 >> 1) * L::NG + grp) * 2 + (w8 & 1)) * 4;
  }
  __device__ __forceinline__ int scale(int place) const {
    return (is_v ? L::VS_OFF : L::KS_OFF) + (place * L::NG + grp) * 4;
  }
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const uint16_t* __restrict__ k, long long k_stride,
                      const uint16_t* __restrict__ v, long long v_stride, const Kv4Req req,
                      const Kv4Cache cache, const FastDiv by_page, int run, int* err) {
  pdl_launch_dependents();
  pdl_wait();
  using L = Kv4<D>;
  static_assert(kHeads == 4, "the exchange below");
  const Lane<D> me;
  const int first = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * run;
  const int n = min(run, req.T - first);
  if (n <= 0) return;
  const int groups = gridDim.y * kHeads * me.STEP;
  uint4 next[kHeads];
  // step q: row first + q % n, head group q / n
  auto load = [&](int r, int h0) {
    const long long row = first + r;
    const uint4* src = reinterpret_cast<const uint4*>((me.is_v ? v + row * v_stride : k + row * k_stride) +
                                                      (h0 + me.sub) * D) + me.d8;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      next[i] = make_uint4(0, 0, 0, 0);
      if (h0 + i * me.STEP + me.sub < cache.Hkv) next[i] = __ldg(src + i * me.STEP * (D / 8));
    }
  };
  int r = 0, h0 = blockIdx.y * kHeads * me.STEP;
  load(r, h0);  // (every row < T is there, whosever it is)
  const Place all = find_tokens(req, cache, by_page, first, n, L::REC, err);
  const int head_bytes = (cache.page >> 4) * L::REC, step_bytes = me.STEP * head_bytes;  // (< 2^19)
  // of the eight lanes of a group, two hold step `mine`'s extremes after the exchange
  const int lane = threadIdx.x & 31, mine = (lane & 1) * 2 + ((lane >> 1) & 1);
  for (;;) {
    const int row = r, head0 = h0;
    uint4 x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) x[i] = next[i];
    if (++r == n) {
      r = 0;
      h0 += groups;
    }
    const bool more = h0 < cache.Hkv;
    if (more) load(r, h0);
    const long long at = __shfl_sync(0xFFFFFFFFu, all.at, row);
    const int place = __shfl_sync(0xFFFFFFFFu, all.in, row);
    if (place < 0) {  // (the whole warp)
      if (!more) break;
      continue;
    }
    const int code = me.code(place), scale = me.scale(place);
    uint8_t* rec = cache.base + at + (long long)(head0 + me.sub) * head_bytes;
    uint32_t m[kHeads];  // (max, -min) of the step's group: over the lane, then over the group
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint32_t hi = max2(max2(x[i].x, x[i].y), max2(x[i].z, x[i].w));
      const uint32_t lo = min2(min2(x[i].x, x[i].y), min2(x[i].z, x[i].w)) ^ 0x80008000u;
      m[i] = max2(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
    }
    const bool odd = lane & 1, second = lane & 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m[i] = max2(odd ? m[i + 2] : m[i], __shfl_xor_sync(0xFFFFFFFFu, odd ? m[i] : m[i + 2], 1));
    uint32_t e = max2(second ? m[1] : m[0], __shfl_xor_sync(0xFFFFFFFFu, second ? m[0] : m[1], 2));
    e = max2(e, __shfl_xor_sync(0xFFFFFFFFu, e, 4));
    const float top = __uint_as_float(e << 16), low = -__uint_as_float(e & 0xFFFF0000u);
    const __half2 so = __halves2half2(__float2half_rn(__fdiv_rn(__fsub_rn(top, low), 15.0f)),
                                      __float2half_rn(low));
    // (a scale of 0 has only codes 0)
    const float inv = __low2float(so) != 0.0f ? 0.0625f * __frcp_rn(__low2float(so)) : 0.0f;
    if (!(lane & 4) && head0 + mine * me.STEP + me.sub < cache.Hkv)
      *reinterpret_cast<__half2*>(rec + mine * step_bytes + scale) = so;
    uint8_t* dst = rec + code;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, dst += step_bytes) {
      const int from_lane = (lane & 24) + (i >> 1) + (i & 1) * 2;  // step i's
      const float off = __half2float(__ushort_as_half(
          (unsigned short)__shfl_sync(0xFFFFFFFFu, (int)__half_as_ushort(__high2half(so)), from_lane)));
      const float r = __shfl_sync(0xFFFFFFFFu, inv, from_lane);
      const uint32_t p[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      // Everything by 1/16, so that the product's saturation is the clamp at 0.  1.5 2^19
      // added to a number below 1 rounds it to the nearest even 16th, in the low bits: eight
      // of them shifted and added leave the codes, and the constants' sum
      constexpr float kBias = 786432.0f;
      constexpr uint32_t kBits = 0x49400000u;
      uint32_t packed = 0;
#pragma unroll
      for (int j = 7; j >= 0; --j) {
        const float w = __uint_as_float((j & 1) ? p[j >> 1] & 0xFFFF0000u : p[j >> 1] << 16);
        const float y = fminf(__saturatef(__fmul_rn(__fsub_rn(w, off), r)), 0.9375f);
        packed = (packed << 4) + __float_as_uint(__fadd_rn(y, kBias));
      }
      packed -= kBits * 0x11111111u;
      if (head0 + i * me.STEP + me.sub >= cache.Hkv) continue;
      if (!me.is_v) {
        *reinterpret_cast<uint32_t*>(dst) = packed;
      } else {
        reinterpret_cast<uint16_t*>(dst)[0] = (uint16_t)packed;
        reinterpret_cast<uint16_t*>(dst)[2] = (uint16_t)(packed >> 16);
      }
    }
    if (!more) break;
  }
}

// A small whole number as fp32: in the low bits of 2^23, which is taken off again.
__device__ __forceinline__ float whole(uint32_t c) {
  return __uint_as_float(c | 0x4B000000u) - 8388608.0f;
}

// Rows whose token is nowhere (a length or page id out of bounds) come back as
// zeros; rows behind the last request are left as they were.
template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_gather_kernel(const Kv4Req req, const Kv4Cache cache, const FastDiv by_page, int run,
                      uint16_t* __restrict__ k, long long k_stride, uint16_t* __restrict__ v,
                      long long v_stride, int* err) {
  pdl_launch_dependents();
  pdl_wait();
  using L = Kv4<D>;
  const Lane<D> me;
  const int first = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * run;
  const int n = min(run, req.T - first);
  if (n <= 0) return;
  const int head_bytes = (cache.page >> 4) * L::REC, step_bytes = me.STEP * head_bytes;  // (< 2^19)
  const int groups = gridDim.y * kHeads * me.STEP;
  const Place all = find_tokens(req, cache, by_page, first, n, L::REC, err);
  uint2 codes[kHeads];
  uint32_t so[kHeads];
  int place = 0;
  auto load = [&](int r, int h0) {
    const long long at = __shfl_sync(0xFFFFFFFFu, all.at, r);
    place = __shfl_sync(0xFFFFFFFFu, all.in, r);
    const uint8_t* rec = cache.base + at + (long long)(h0 + me.sub) * head_bytes;
    const int code = me.code(place) & ~3, scale = me.scale(place);  // (a V word holds two tokens)
    const uint8_t* src = rec;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, src += step_bytes) {
      codes[i] = make_uint2(0, 0);
      so[i] = 0;
      if (place < 0 || h0 + i * me.STEP + me.sub >= cache.Hkv) continue;
      if (me.is_v)
        codes[i] = __ldg(reinterpret_cast<const uint2*>(src + code));
      else
        codes[i].x = __ldg(reinterpret_cast<const uint32_t*>(src + code));
      so[i] = __ldg(reinterpret_cast<const uint32_t*>(src + scale));
    }
  };
  int r = 0, h0 = blockIdx.y * kHeads * me.STEP;
  load(r, h0);
  for (;;) {
    const long long row = first + r;
    const int head0 = h0;
    const bool owned = place != -2;
    const uint32_t pick = !me.is_v ? 0x3210u : (place & 1) ? 0x7632u : 0x5410u;
    uint32_t packed[kHeads];
    float s[kHeads], o[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      packed[i] = __byte_perm(codes[i].x, codes[i].y, pick);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&so[i]));
      s[i] = f.x;
      o[i] = f.y;
    }
    if (++r == n) {
      r = 0;
      h0 += groups;
    }
    const bool more = h0 < cache.Hkv;
    if (more) load(r, h0);
    if (owned) {
      uint16_t* dst = (me.is_v ? v + row * v_stride : k + row * k_stride) + (head0 + me.sub) * D + 8 * me.d8;
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        if (head0 + i * me.STEP + me.sub >= cache.Hkv) continue;
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // code * scale is exact in fp32 (4 + 11 bits): one rounding of the sum, then bf16's
          const float a = fmaf(whole((packed[i] >> (8 * j)) & 15u), s[i], o[i]);
          const float b = fmaf(whole((packed[i] >> (8 * j + 4)) & 15u), s[i], o[i]);
          const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
          out[j] = *reinterpret_cast<const uint32_t*>(&y);
        }
        *reinterpret_cast<uint4*>(dst + i * me.STEP * D) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    if (!more) break;
  }
}

void grid_of(int64_t T, const Kv4Cache& c, int* run, cudaLaunchConfig_t* cfg,
             cudaLaunchAttribute* attr, cudaStream_t s) {
  const int heads = kHeads * (c.D == 64 ? 2 : 1);
  const int groups = std::min((c.Hkv + heads - 1) / heads, 64);
  const int64_t per_block = kThreads / 32, warps = (int64_t)num_sms() * 8 * per_block;
  *run = (int)std::min<int64_t>(32, (T * groups + warps - 1) / warps);
  const int64_t rows = *run * per_block;
  cfg->gridDim = dim3((unsigned)((T + rows - 1) / rows), (unsigned)groups);
  cfg->blockDim = dim3(kThreads);
  cfg->stream = s;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, const Kv4Req& req, const Kv4Cache& cache, int* err,
                              cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  int run;
  grid_of(req.T, cache, &run, &cfg, attr, s);
  auto kernel = cache.D == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>;
  return cudaLaunchKernelEx(&cfg, kernel, k, (long long)k_stride, v, (long long)v_stride, req,
                            cache, fast_div(cache.page), run, err);
}

cudaError_t launch_kv4_gather(const Kv4Req& req, const Kv4Cache& cache, uint16_t* k,
                              int64_t k_stride, uint16_t* v, int64_t v_stride, int* err,
                              cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  int run;
  grid_of(req.T, cache, &run, &cfg, attr, s);
  auto kernel = cache.D == 64 ? kv4_gather_kernel<64> : kv4_gather_kernel<128>;
  return cudaLaunchKernelEx(&cfg, kernel, req, cache, fast_div(cache.page), run, k, (long long)k_stride, v,
                            (long long)v_stride, err);
}

}  // namespace qk
