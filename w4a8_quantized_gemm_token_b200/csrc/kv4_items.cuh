// kv4_items.cuh -- how the attention's work over the 4-bit cache is laid out, for the
// kernels that read it (kv4_attn.cu, kv4_chunk.cu).  An item is (request, row tile, kv
// head): ROWS query rows, a row being a token and one of its G heads.  Its units are the
// blocks of 2^LOG keys that it sees.  All units of all items are laid end to end (kv
// heads innermost, then row tiles, then requests) and cut into equal spans.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fast_div.cuh"
#include "kv4.cuh"
#include "sm100.cuh"

namespace qk {

// The least product of a weight (1 for a row's largest) and a scale that a row's reference is
// set by.  Below fp16's least scale, 2^-24, only where the keys of large weight have scale 0;
// with 2^-64 the weights stay below 2^78, and their sums with offsets (2^16, 2^26 keys) below
// 2^120.
constexpr float kLightest = 0x1p-64f;

__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

constexpr float kLeast = -3.0e38f;  // the least maximum that is kept

// The reference that a row's largest score sets (top, in units of log2; heavy: the largest weight
// times scale if that score's weight is 1): added to the scores, it puts `heavy` into [2^5, 2^6).
// From |top| = 2^26 on one step of it in fp32 is 8 and more: it would not land there, the products
// could leave fp16, and fp32 scores hold no difference that a softmax could tell.  Such a row
// is NaN.
__device__ __forceinline__ float reference(float top, float heavy) {
  if (fabsf(top) >= 0x1p26f && top > -INFINITY) return __int_as_float(0x7FFFFFFF);
  return (float)(5 - exponent(fmaxf(heavy, kLightest))) - fmaxf(top, kLeast);
}

constexpr int kMaxBlocks = 160;  // a block per SM; the workspace holds this many

struct Kv4Args {
  const uint16_t* q;
  long long q_stride;
  int H, G;
  FastDiv by_g, by_page;  // rows per token; records per page
  Kv4Req req;
  Kv4Cache cache;
  float sc;  // scale log2 e
  int window, sinks;
  uint16_t* out;
  uint8_t* ws;
  int* err;
};

// ---- items

struct Item {
  int b, rt, kvh;
  int row0, n, len, nrt;
  int cnt, ns, first;  // units, how many of them are sinks' blocks, first block behind those
  int p0, p1;          // positions of the tile's first and last row
  int whole0, whole1;  // every row sees all keys of units [whole0, whole1)
};

template <int ROWS>
__device__ __forceinline__ void set_request(const Kv4Args& a, Item& it, const Kv4Seq& s) {
  it.row0 = s.row0;
  it.n = s.n;
  it.len = s.len;
  it.nrt = (s.n * a.G + ROWS - 1) / ROWS;
}

template <int ROWS>
__device__ __forceinline__ void load_request(const Kv4Args& a, Item& it) {
  set_request<ROWS>(a, it, kv4_seq(a.req, it.b, a.err));
}

// The blocks that row tile rt of the request sees; one empty unit where it sees none.
template <int ROWS, int LOG = 4>
__device__ __forceinline__ void load_tile(const Kv4Args& a, Item& it) {
  constexpr int KEYS = 1 << LOG;
  const int last = it.n * a.G - 1;
  it.p0 = it.len - it.n + quot(it.rt * ROWS, a.by_g);
  it.p1 = it.len - it.n + quot(min(it.rt * ROWS + ROWS - 1, last), a.by_g);
  it.ns = it.first = it.whole0 = it.whole1 = 0;
  it.cnt = 1;
  if (it.p1 < 0) return;
  const int end = (it.p1 >> LOG) + 1;
  if (a.window > 0) {
    it.first = max(it.p0 - a.window + 1, 0) >> LOG;
    it.ns = min((a.sinks + KEYS - 1) >> LOG, it.first);
    it.whole0 = it.ns + ((max(it.p1 - a.window + 1, 0) + KEYS - 1) >> LOG) - it.first;
  }
  it.cnt = it.ns + end - it.first;
  it.whole1 = max(it.ns + ((max(it.p0, -1) + 1) >> LOG) - it.first, it.whole0);
}

__device__ __forceinline__ int record_of(const Item& it, int k) {
  return k < it.ns ? k : it.first + k - it.ns;
}

// Steps to the next item (kv heads innermost, then row tiles, then requests).
template <int ROWS, int LOG = 4>
__device__ __forceinline__ void next_item(const Kv4Args& a, Item& it) {
  if (++it.kvh < a.cache.Hkv) return;
  it.kvh = 0;
  if (++it.rt >= it.nrt) {
    it.rt = 0;
#pragma unroll 1
    do {
      if (++it.b >= a.req.B) return;  // behind the last span
      load_request<ROWS>(a, it);
    } while (it.nrt == 0);
  }
  load_tile<ROWS, LOG>(a, it);
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Units of all row tiles of the request, for one kv head, by the whole warp.  PAD: units that
// an item counts for beside its own, where a new item costs as much as they do.
template <int ROWS, int LOG = 4, int PAD = 0>
__device__ __forceinline__ long long request_units(const Kv4Args& a, const Item& base) {
  long long sum = 0;
#pragma unroll 1
  for (int rt0 = 0; rt0 < base.nrt; rt0 += 32) {
    Item it = base;
    it.rt = rt0 + (threadIdx.x & 31);
    uint32_t c = 0;
    if (it.rt < it.nrt) {
      load_tile<ROWS, LOG>(a, it);
      c = (uint32_t)(it.cnt + PAD);  // (at most 2^26)
    }
    sum += warp_sum(c);
  }
  return sum;
}

// The units in front of each thread's stretch of requests (up to the number of threads),
// and every stretch's first request.
template <int NW>
struct Kv4Scan {
  long long pre[32 * NW + 1];
  Kv4Seq seqs[32 * NW];
  long long tot[NW];
};

// Fills s, by the whole block of NW warps: `per` requests per thread, then a scan over threads.
template <int ROWS, int LOG, int PAD = 0, int NW>
__device__ __forceinline__ void scan_units(const Kv4Args& a, Kv4Scan<NW>& s, int per, int warp) {
  const int lane = threadIdx.x & 31;
  long long mine = 0;
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    Item it;
    it.b = threadIdx.x * per + i;
    it.nrt = 0;
    int one = 0;
    if (it.b < a.req.B) {
      const Kv4Seq sq = kv4_seq(a.req, it.b, a.err);
      if (i == 0) s.seqs[threadIdx.x] = sq;  // the stretch's first request
      set_request<ROWS>(a, it, sq);
      if (it.nrt == 1) {
        it.rt = 0;
        load_tile<ROWS, LOG>(a, it);
        one = it.cnt + PAD;
      }
    }
    long long u = one;
    uint32_t many = __ballot_sync(0xFFFFFFFFu, it.nrt > 1);
#pragma unroll 1
    while (many) {  // requests of several row tiles: the warp counts them together
      const int src = __ffs(many) - 1;
      many &= many - 1;
      Item big;
      big.n = __shfl_sync(0xFFFFFFFFu, it.n, src);
      big.len = __shfl_sync(0xFFFFFFFFu, it.len, src);
      big.nrt = __shfl_sync(0xFFFFFFFFu, it.nrt, src);
      const long long all = request_units<ROWS, LOG, PAD>(a, big);
      if (lane == src) u = all;
    }
    mine += u * a.cache.Hkv;
  }
  // inclusive scan over the warp, then over the warps
  long long sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s.tot[warp] = sum;
  __syncthreads();
  long long before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) before += w < warp ? s.tot[w] : 0;
  s.pre[threadIdx.x + 1] = before + sum;
  if (threadIdx.x == 0) s.pre[0] = 0;
  __syncthreads();
}

// The item that unit u0 is in, and which of the item's units it is (the first one where u0 is
// of the PAD in front), by a whole warp.
template <int ROWS, int LOG, int PAD = 0, int NW>
__device__ __forceinline__ bool locate_unit(const Kv4Args& a, const Kv4Scan<NW>& s, int per, long long u0,
                                            Item& it, int& k) {
  const int lane = threadIdx.x & 31;
  // the last t with s.pre[t] <= u0 (it has units): among every NW-th, then among those
  // behind it
  int lo = (__popc(__ballot_sync(0xFFFFFFFFu, s.pre[lane * NW] <= u0)) - 1) * NW;
  lo += __popc(__ballot_sync(0xFFFFFFFFu, lane < NW && s.pre[lo + min(lane, NW - 1)] <= u0)) - 1;
  long long rest = u0 - s.pre[lo];
  it.b = lo * per;
  set_request<ROWS>(a, it, s.seqs[lo]);
  if (per > 1) {
#pragma unroll 1
    for (;;) {
      const long long u = request_units<ROWS, LOG, PAD>(a, it) * a.cache.Hkv;
      if (rest < u || it.b + 1 >= a.req.B) break;
      rest -= u;
      ++it.b;
      load_request<ROWS>(a, it);
    }
  }
  int at = 0;  // the row tile
#pragma unroll 1
  for (int rt0 = 0; it.nrt > 1; rt0 += 32) {
    Item one = it;
    one.rt = rt0 + lane;
    long long c = 0;
    if (one.rt < one.nrt) {
      load_tile<ROWS, LOG>(a, one);
      c = (long long)(one.cnt + PAD) * a.cache.Hkv;
    }
    long long sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    const uint32_t over = __ballot_sync(0xFFFFFFFFu, sum > rest);
    if (over != 0) {
      const int src = __ffs(over) - 1;
      rest -= __shfl_sync(0xFFFFFFFFu, sum - c, src);
      at = rt0 + src;
      break;
    }
    rest -= __shfl_sync(0xFFFFFFFFu, sum, 31);
    if (rt0 + 32 >= it.nrt) return false;  // not reached: the units add up
  }
  it.rt = at;
  load_tile<ROWS, LOG>(a, it);
  const int cost = it.cnt + PAD;
  it.kvh = rest >> 31 ? (int)(rest / cost) : (int)((uint32_t)rest / (uint32_t)cost);
  k = max((int)(rest - (long long)it.kvh * cost) - PAD, 0);
  return true;
}

}  // namespace qk
