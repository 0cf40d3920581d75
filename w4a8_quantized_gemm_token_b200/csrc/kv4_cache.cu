// kv4_cache.cu -- writing tokens into the 4-bit key/value cache, and reading them
// back as bf16.
//
// Per token, kv head and group of 64 dims, the affine rule of the W4 weights:
//     s = fp16((max - min) / 15), o = fp16(min),
//     code = clamp(rne((w - o) fl32(1 / s)), 0, 15)   (0 where s = 0),
// fp32 arithmetic, one rounding per operation; the value is code s + o.
//
// Bound: HBM (4 D bytes of bf16 and 9 D / 8 of record per token and head).  Eight
// lanes hold a group (16 bytes each); the request of a row is found by a 32-way
// search over the row bounds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4.cuh"
#include "sm100.cuh"

namespace qk {
namespace {

constexpr int kThreads = 256;

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

// Where row `row` of the call lives: the byte offset of its record (for kv head 0)
// and its place in it; false (recorded, unless it is behind the last request) if nowhere.
__device__ __forceinline__ bool find_token(const Kv4Req& r, const Kv4Cache& c, int row, int rec,
                                           long long* at, int* place, int* err) {
  const int b = find_request(r, row);
  if (b >= r.B) return false;
  const Kv4Seq s = kv4_seq(r, b, err);
  const int pos = s.len - s.n + (row - s.row0);
  if (row < s.row0) return false;  // in front of the first request
  if (pos < 0 || row >= s.row0 + s.n) {  // no such token; or row bounds that fall
    record_index(err);
    return false;
  }
  const int pg = pos / c.page;
  const int id = __ldg(r.page_table + (long long)b * r.max_pages + pg);
  if (id < 0 || id >= c.num_pages) {
    record_index(err);
    return false;
  }
  const int in = pos - pg * c.page;
  const int tiles = c.page >> 4;
  *at = ((long long)id * c.Hkv * tiles + (in >> 4)) * rec;
  *place = in & 15;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const uint16_t* __restrict__ k, long long k_stride,
                      const uint16_t* __restrict__ v, long long v_stride, const Kv4Req req,
                      const Kv4Cache cache, int rows_per_block, int* err) {
  pdl_launch_dependents();
  pdl_wait();
  using L = Kv4<D>;
  constexpr int LANES = D / 4;           // of one token and head: K row, then V row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LANES, e = lane % LANES;  // D = 64: two heads at a time
  const bool is_v = e >= LANES / 2;
  const int d8 = e % (LANES / 2);        // chunk of 8 dims
  const int grp = d8 >> 3, w8 = d8 & 7;
  const int tiles = cache.page >> 4;
  for (int i = warp; i < rows_per_block; i += kThreads / 32) {
    const int row = blockIdx.x * rows_per_block + i;
    if (row >= req.T) break;
    long long at;
    int place;
    if (!find_token(req, cache, row, L::REC, &at, &place, err)) continue;  // warp-uniform
    const uint16_t* src = is_v ? v + row * v_stride : k + row * k_stride;
    for (int h0 = 0; h0 < cache.Hkv; h0 += 32 / LANES) {
      const int head = h0 + sub;
      const bool live = head < cache.Hkv;
      const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(src + (long long)head * D) + d8)
                           : make_uint4(0, 0, 0, 0);
      const uint32_t p[4] = {x.x, x.y, x.z, x.w};
      float w[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = __uint_as_float(p[j] << 16);
        w[2 * j + 1] = __uint_as_float(p[j] & 0xFFFF0000u);
      }
      float lo = w[0], hi = w[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        lo = fminf(lo, w[j]);
        hi = fmaxf(hi, w[j]);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
      }
      const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
      const __half oh = __float2half_rn(lo);
      const float s = __half2float(sh), off = __half2float(oh);
      uint32_t packed = 0;
      if (s != 0.0f) {
        const float r = __fdiv_rn(1.0f, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          int q = __float2int_rn(__fmul_rn(__fsub_rn(w[j], off), r));
          q = max(0, min(15, q));
          packed |= (uint32_t)q << (4 * j);
        }
      }
      if (!live) continue;
      uint8_t* rec = cache.base + at + (long long)head * tiles * L::REC;
      if (!is_v) {
        reinterpret_cast<uint32_t*>(rec + place * (D / 2))[((w8 >> 1) * L::NG + grp) * 2 + (w8 & 1)] =
            packed;
      } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(
            rec + L::V_OFF + (((place >> 1) * 8 + w8) * L::NG + grp) * 8 + (place & 1) * 2);
        dst[0] = (uint16_t)packed;
        dst[2] = (uint16_t)(packed >> 16);
      }
      if (w8 == 0) {
        __half2* sc = reinterpret_cast<__half2*>(rec + (is_v ? L::VS_OFF : L::KS_OFF));
        sc[place * L::NG + grp] = __halves2half2(sh, oh);
      }
    }
  }
}

// Rows whose token is nowhere (a length or page id out of bounds) come back as
// zeros; rows behind the last request are left as they were.
template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_gather_kernel(const Kv4Req req, const Kv4Cache cache, uint16_t* __restrict__ k,
                      long long k_stride, uint16_t* __restrict__ v, long long v_stride,
                      int rows_per_block, int* err) {
  pdl_launch_dependents();
  pdl_wait();
  using L = Kv4<D>;
  constexpr int LANES = D / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LANES, e = lane % LANES;
  const bool is_v = e >= LANES / 2;
  const int d8 = e % (LANES / 2);
  const int grp = d8 >> 3, w8 = d8 & 7;
  const int tiles = cache.page >> 4;
  for (int i = warp; i < rows_per_block; i += kThreads / 32) {
    const int row = blockIdx.x * rows_per_block + i;
    if (row >= req.T) break;
    long long at = 0;
    int place = 0;
    const bool found = find_token(req, cache, row, L::REC, &at, &place, err);
    if (!found) {
      const int b = find_request(req, row);
      if (b >= req.B || row < kv4_seq(req, b, err).row0) continue;
    }
    uint16_t* dst = is_v ? v + row * v_stride : k + row * k_stride;
    for (int head = sub; head < cache.Hkv; head += 32 / LANES) {
      uint32_t out[4] = {0, 0, 0, 0};
      if (found) {
        const uint8_t* rec = cache.base + at + (long long)head * tiles * L::REC;
        uint32_t packed;
        if (!is_v) {
          packed = reinterpret_cast<const uint32_t*>(
              rec + place * (D / 2))[((w8 >> 1) * L::NG + grp) * 2 + (w8 & 1)];
        } else {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(
              rec + L::V_OFF + (((place >> 1) * 8 + w8) * L::NG + grp) * 8 + (place & 1) * 2);
          packed = src[0] | (uint32_t)src[2] << 16;
        }
        const __half2 so = reinterpret_cast<const __half2*>(
            rec + (is_v ? L::VS_OFF : L::KS_OFF))[place * L::NG + grp];
        const float s = __low2float(so), o = __high2float(so);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // code * scale is exact in fp32 (4 + 11 bits): one rounding of the sum, then bf16's
          const float a = fmaf((float)((packed >> (8 * j)) & 15u), s, o);
          const float b = fmaf((float)((packed >> (8 * j + 4)) & 15u), s, o);
          const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
          out[j] = *reinterpret_cast<const uint32_t*>(&r);
        }
      }
      *(reinterpret_cast<uint4*>(dst + (long long)head * D) + d8) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

void grid_of(int64_t T, int* rows, cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr,
             cudaStream_t s) {
  // a warp per row; more rows per block once every SM has its share of blocks
  *rows = kThreads / 32;
  cfg->gridDim = dim3((unsigned)((T + *rows - 1) / *rows));
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
  int rows;
  grid_of(req.T, &rows, &cfg, attr, s);
  auto kernel = cache.D == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>;
  return cudaLaunchKernelEx(&cfg, kernel, k, (long long)k_stride, v, (long long)v_stride, req,
                            cache, rows, err);
}

cudaError_t launch_kv4_gather(const Kv4Req& req, const Kv4Cache& cache, uint16_t* k,
                              int64_t k_stride, uint16_t* v, int64_t v_stride, int* err,
                              cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  int rows;
  grid_of(req.T, &rows, &cfg, attr, s);
  auto kernel = cache.D == 64 ? kv4_gather_kernel<64> : kv4_gather_kernel<128>;
  return cudaLaunchKernelEx(&cfg, kernel, req, cache, k, (long long)k_stride, v,
                            (long long)v_stride, rows, err);
}

}  // namespace qk
