// kv4_attn.cu -- attention of a few new tokens per request over the 4-bit paged
// key/value cache (kv4.cuh), causal, with an optional sliding window and first
// tokens that stay visible.
//
// For query row i at position p (the rows are the last tokens of their request),
// over the visible keys j <= p with j > p - window or j < sinks:
//     x_j = scale sum_groups [ sK_jg (q_g . cK_jg) + oK_jg sum(q_g) ]
//     P_j = 2^((x_j - max) log2 e),   l = sum_j P_j
//     out = 1/l sum_j P_j (sV_jg cV_j + oV_jg)
// The codes (0..15) are exact in bf16, so the tensor cores take them as they are:
// q . c is exact products summed in fp32, and no dequantized K or V exists
// anywhere.  P_j sV_jg is split into two bf16 (16 bits of significand) and both
// halves are multiplied; rounding it once to bf16 would cost more than the
// output's own rounding, since P sV c and P oV nearly cancel.
//
// Bound: HBM (9 D / 8 bytes per visible token and kv head).  What has to keep up
// with it is the integer and fp32 work per code: 11 instructions unpack a word of
// 8 codes into the four bf16 pairs of a fragment (three shifts, four and-or with
// the exponent of 128, four subtractions of 128).  mma.sync is used rather than
// tcgen05 because its operands are registers: a tcgen05 tile of 128 would have to
// write the unpacked codes to shared memory (4 bytes per code written and read,
// against half a byte loaded) to multiply them with the 1 to 16 rows there are.
//
// Layout of the work: an item is (request, row tile, kv head), its units are the
// 16-token records it sees.  All units of all items are laid end to end and cut
// into equal spans, one per consumer warp, from the lengths on the device: one
// long request and a ragged batch fill the GPU alike, and no length goes through
// the host.  A warp that holds a whole item writes the output; the pieces of an
// item that is cut are joined in the block (through shared memory), and, where
// the cut is between blocks, by kv4_join_kernel from the workspace, in the order
// of the units: no atomics, the same bits on every run.
//
// One producer warp per block runs every consumer's ring of bulk copies (lane c
// for consumer c): it walks the items, looks the pages up and keeps each ring full.
//
// A row tile is 16 rows (kWide) or 8: with 8 the tile's upper half of the
// 16-row fragments holds the low halves of P sV, so that both halves cost one mma.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4.cuh"
#include "sm100.cuh"

namespace qk {
namespace {

constexpr int kMaxBlocks = 160;  // a block per SM; the workspace holds this many

template <int D, bool kWide>
struct Cfg {
  static constexpr int ROWS = kWide ? 16 : 8;
  // 11 consumers and the producer: three warps to a quarter of the SM, 168
  // registers a thread (a thirteenth warp would leave 128)
  static constexpr int NW = 11;
  static constexpr int STAGES = kWide ? 5 : 6;         // records in a consumer's ring
  static constexpr int THREADS = 32 * (NW + 1);
  static constexpr int LD = D + 4;                     // floats per row of a piece in shared memory
  static constexpr int PIECE = (ROWS * LD + 2 * ROWS) * 4;  // O rows, then m, l
  static constexpr int RING = STAGES * Kv4<D>::REC;
  static constexpr int SM_RING = 0;
  static constexpr int SM_HEAD = SM_RING + NW * RING;  // piece of an item that began before the span
  static constexpr int SM_BAR = SM_HEAD + NW * PIECE;  // full, empty per stage and consumer
  static constexpr int SM_BAD = SM_BAR + NW * STAGES * 16;
  static constexpr int SM_SPAN = (SM_BAD + NW * STAGES * 4 + 15) / 16 * 16;
  static constexpr int SMEM = SM_SPAN + NW * 32 + 128;
  static_assert(PIECE <= RING, "a span's last piece is kept in its ring");
  static_assert(SM_HEAD % 16 == 0 && SM_BAR % 16 == 0 && SM_SPAN % 16 == 0, "alignment");
  static_assert(SMEM + 8 * (THREADS + 64) <= 232448, "with the static shared memory");
};

struct Args {
  const uint16_t* q;
  long long q_stride;
  int H, G;
  Kv4Req req;
  Kv4Cache cache;
  float sc;  // scale log2 e
  int window, sinks;
  uint16_t* out;
  uint8_t* ws;
  int* err;
};

// ---- workspace: header, a word per block, then two pieces per block (its first
// item's, where that began in an earlier block, and its last's)
struct Meta {
  int flags;  // 1: a first piece, 2: it ends its item, 4: a last piece (of item b, rt, kvh)
  int b, rt, kvh;
};
constexpr size_t kMetaOff = 256;
constexpr size_t kPieceOff = kMetaOff + kMaxBlocks * sizeof(Meta);
__host__ __device__ constexpr size_t piece_floats(int D) { return (size_t)16 * (D + 2); }

__device__ __forceinline__ float* piece_at(uint8_t* ws, int D, int block, int which) {
  return reinterpret_cast<float*>(ws + kPieceOff) + (size_t)(2 * block + which) * piece_floats(D);
}

// ---- items

struct Item {
  int b, rt, kvh;
  int row0, n, len, nrt;
  int cnt, ns, first;  // units, how many of them are sinks' records, first record behind those
  int p0, p1;          // positions of the tile's first and last row
};

template <int ROWS>
__device__ __forceinline__ void load_request(const Args& a, Item& it) {
  const Kv4Seq s = kv4_seq(a.req, it.b, a.err);
  it.row0 = s.row0;
  it.n = s.n;
  it.len = s.len;
  it.nrt = (int)(((long long)s.n * a.G + ROWS - 1) / ROWS);
}

// The records that row tile rt of the loaded request sees; one empty unit where it sees none.
template <int ROWS>
__device__ __forceinline__ void load_tile(const Args& a, Item& it) {
  const int last = it.n * a.G - 1;
  it.p0 = it.len - it.n + it.rt * ROWS / a.G;
  it.p1 = it.len - it.n + min(it.rt * ROWS + ROWS - 1, last) / a.G;
  it.ns = it.first = 0;
  it.cnt = 1;
  if (it.p1 < 0) return;
  const int end = (it.p1 >> 4) + 1;
  if (a.window > 0) {
    it.first = max(it.p0 - a.window + 1, 0) >> 4;
    it.ns = min((a.sinks + 15) >> 4, it.first);
  }
  it.cnt = it.ns + end - it.first;
}

// Steps to the next item (kv heads innermost, then row tiles, then requests).
template <int ROWS>
__device__ __forceinline__ void next_item(const Args& a, Item& it) {
  if (++it.kvh < a.cache.Hkv) return;
  it.kvh = 0;
  if (++it.rt >= it.nrt) {
    it.rt = 0;
    do {
      if (++it.b >= a.req.B) return;  // behind the last span
      load_request<ROWS>(a, it);
    } while (it.nrt == 0);
  }
  load_tile<ROWS>(a, it);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Units of all row tiles of the loaded request, for one kv head, by the whole warp.
template <int ROWS>
__device__ __forceinline__ long long request_units(const Args& a, const Item& base) {
  long long sum = 0;
  for (int rt0 = 0; rt0 < base.nrt; rt0 += 32) {
    Item it = base;
    it.rt = rt0 + (threadIdx.x & 31);
    int c = 0;
    if (it.rt < it.nrt) {
      load_tile<ROWS>(a, it);
      c = it.cnt;
    }
    sum += warp_sum(c);
  }
  return sum;
}

// What a consumer warp starts from, in shared memory for its producer lane.
struct Span {
  int b, rt, kvh, k;
  long long units;
  int pad[2];
};
static_assert(sizeof(Span) == 32, "span size");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// D += A B^T, 16 x 8 x 16, bf16 operands, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of w as a pair of bf16: 0x4300 | c is 128 + c, less 128.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  uint32_t r = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  const uint32_t base = 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&r),
                                   *reinterpret_cast<const __nv_bfloat162*>(&base));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// a, b as hi + lo, each a pair of bf16: hi truncates, lo rounds what is left.
__device__ __forceinline__ void split2(float a, float b, uint32_t* hi, uint32_t* lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  *hi = __byte_perm(ua, ub, 0x7632);
  *lo = pack16(a - __uint_as_float(ua & 0xFFFF0000u), b - __uint_as_float(ub & 0xFFFF0000u));
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], const uint8_t* p) {
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x; r[1] = v.y;
  }
}

constexpr float kNone = -1.0e30f;  // the reference maximum of a row that has seen nothing

template <int D, bool kWide>
__global__ void __launch_bounds__(Cfg<D, kWide>::THREADS, 1) kv4_attn_kernel(const Args a, int min_units) {
  using C = Cfg<D, kWide>;
  using L = Kv4<D>;
  constexpr int NG = L::NG, ROWS = C::ROWS, NW = C::NW, STAGES = C::STAGES;
  constexpr int RT = kWide ? 2 : 1;  // fragment row halves that hold rows of their own
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem<128>(smem_raw);
  __shared__ long long pre[C::THREADS + 1];
  __shared__ int seg_flags[NW];
  __shared__ int seg_item[NW][6];  // first piece's b, rt, kvh; last piece's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blockIdx.x;
  auto full = [&](int w, int s) { return smem_u32(smem + C::SM_BAR) + (uint32_t)(w * STAGES + s) * 16u; };
  auto empty = [&](int w, int s) { return full(w, s) + 8u; };
  int* bad = reinterpret_cast<int*>(smem + C::SM_BAD);
  Span* spans = reinterpret_cast<Span*>(smem + C::SM_SPAN);

  if (threadIdx.x < NW * STAGES) {
    mbar_init(full(0, threadIdx.x), 1);
    mbar_init(empty(0, threadIdx.x), 1);
  }
  fence_mbar_init();
  pdl_launch_dependents();
  pdl_wait();

  // ---- units in all: a stretch of requests per thread, then a scan over threads
  const int per = (a.req.B + C::THREADS - 1) / C::THREADS;
  {
    long long mine = 0;
    for (int i = 0; i < per; ++i) {
      Item it;
      it.b = threadIdx.x * per + i;
      it.nrt = 0;
      int one = 0;
      if (it.b < a.req.B) {
        load_request<ROWS>(a, it);
        if (it.nrt == 1) {
          it.rt = 0;
          load_tile<ROWS>(a, it);
          one = it.cnt;
        }
      }
      long long u = one;
      uint32_t many = __ballot_sync(0xFFFFFFFFu, it.nrt > 1);
      while (many) {  // requests of several row tiles: the warp counts them together
        const int src = __ffs(many) - 1;
        many &= many - 1;
        Item big;
        big.n = __shfl_sync(0xFFFFFFFFu, it.n, src);
        big.len = __shfl_sync(0xFFFFFFFFu, it.len, src);
        big.nrt = __shfl_sync(0xFFFFFFFFu, it.nrt, src);
        const long long s = request_units<ROWS>(a, big);
        if (lane == src) u = s;
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
    __shared__ long long tot[NW + 1];
    if (lane == 31) tot[warp] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += tot[w];
    pre[threadIdx.x + 1] = before + sum;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
  }
  const long long W = pre[C::THREADS];
  const long long want = (W + (long long)NW * min_units - 1) / ((long long)NW * min_units);
  const int blocks = (int)min((long long)gridDim.x, want);
  if (blk == 0 && threadIdx.x == 0) *reinterpret_cast<int*>(a.ws) = blocks;
  if (blk >= blocks) return;  // the whole block

  if (warp < NW) {
    // ---- this warp's span [u0, u1) and the item it starts in
    const long long slot = (long long)blk * NW + warp, slots = (long long)blocks * NW;
    const long long u0 = W * slot / slots, u1 = W * (slot + 1) / slots;
    Span sp = {};
    sp.units = u1 - u0;
    if (sp.units > 0) {
      int lo = 0, hi = C::THREADS - 1;  // the last t with pre[t] <= u0 and units behind it
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= u0) lo = mid; else hi = mid - 1;
      }
      long long rest = u0 - pre[lo];
      Item it;
      it.b = lo * per;
      for (;; ++it.b) {
        load_request<ROWS>(a, it);
        const long long u = request_units<ROWS>(a, it) * a.cache.Hkv;
        if (rest < u || it.b + 1 >= a.req.B) break;
        rest -= u;
      }
      for (int rt0 = 0;; rt0 += 32) {
        it.rt = rt0 + lane;
        long long c = 0;
        if (it.rt < it.nrt) {
          load_tile<ROWS>(a, it);
          c = (long long)it.cnt * a.cache.Hkv;
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
          const int cnt = __shfl_sync(0xFFFFFFFFu, it.cnt, src);
          sp.b = it.b;
          sp.rt = rt0 + src;
          sp.kvh = (int)(rest / cnt);
          sp.k = (int)(rest - (long long)sp.kvh * cnt);
          break;
        }
        rest -= __shfl_sync(0xFFFFFFFFu, sum, 31);
        if (rt0 + 32 >= it.nrt) {  // not reached: the units add up
          sp.units = 0;
          break;
        }
      }
    }
    if (lane == 0) {
      spans[warp] = sp;
      seg_flags[warp] = 0;
    }
  }
  __syncthreads();

  const int tiles_per_page = a.cache.page >> 4;
  if (warp == NW) {
    // ------------------------------------------------------------- producer
    long long left = 0, issued = 0;
    Item it = {};
    int k = 0;
    if (lane < NW) {
      const Span sp = spans[lane];
      left = sp.units;
      if (left > 0) {
        it.b = sp.b;
        it.rt = sp.rt;
        it.kvh = sp.kvh;
        k = sp.k;
        load_request<ROWS>(a, it);
        load_tile<ROWS>(a, it);
      }
    }
    auto lookup = [&]() -> int {  // the next unit's page
      if (left == 0 || it.p1 < 0) return -1;
      const int tile = k < it.ns ? k : it.first + k - it.ns;
      return __ldg(a.req.page_table + (long long)it.b * a.req.max_pages + tile / tiles_per_page);
    };
    int id = lookup();
    long long t0 = clock64();
    while (__any_sync(0xFFFFFFFFu, left > 0)) {
      bool moved = false;
      if (left > 0) {
        const int s = (int)(issued % STAGES);
        const uint32_t ph = (uint32_t)((issued / STAGES) & 1) ^ 1u;
        if (mbar_test(empty(lane, s), ph)) {
          moved = true;
          const int tile = k < it.ns ? k : it.first + k - it.ns;
          const bool seen = it.p1 >= 0;
          const bool ok = seen && id >= 0 && id < a.cache.num_pages;
          if (seen && !ok) record_index(a.err);
          bad[lane * STAGES + s] = ok ? 0 : 1;
          if (ok) {
            const long long rec = ((long long)id * a.cache.Hkv + it.kvh) * tiles_per_page + tile % tiles_per_page;
            mbar_arrive_expect_tx(full(lane, s), L::REC);
            bulk_load(smem_u32(smem + C::SM_RING + lane * C::RING + s * L::REC),
                      a.cache.base + rec * L::REC, L::REC, full(lane, s));
          } else {
            mbar_arrive(full(lane, s));
          }
          ++issued;
          --left;
          if (left > 0 && ++k == it.cnt) {
            k = 0;
            next_item<ROWS>(a, it);
          }
          id = lookup();
        }
      }
      if (__any_sync(0xFFFFFFFFu, moved)) {
        t0 = clock64();
      } else if (clock64() - t0 > QK_WAIT_LIMIT_CYCLES) {
        if (lane == 0) record_timeout(a.err);
        break;
      }
    }
    // every copy has landed before the block may end
    for (int j = 0; j < STAGES; ++j) {
      if (lane < NW && issued > j) {
        const long long u = issued - 1 - j;
        mbar_wait(full(lane, (int)(u % STAGES)), (uint32_t)((u / STAGES) & 1), a.err);
      }
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* ring = smem + C::SM_RING + warp * C::RING;
    const Span sp = spans[warp];
    Item it;
    it.b = sp.b;
    it.rt = sp.rt;
    it.kvh = sp.kvh;
    int k = sp.k;
    bool first_piece = sp.k > 0;
    int flags = 0;
    long long done = 0;
    bool ok = true;
    if (sp.units > 0) {
      load_request<ROWS>(a, it);
      load_tile<ROWS>(a, it);
    }
    while (done < sp.units && ok) {
      // ---- a segment: this span's units of one item
      uint32_t qa[RT][NG][2][4];  // per j: the pairs (i, i + 4) of dims 64 group + 16 t + 8 j
      float qsum[RT][NG];
      int pos[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = it.rt * ROWS + g + 8 * r;
        const int tok = row / a.G;
        const bool live = tok < it.n;
        pos[r] = live ? it.len - it.n + tok : -1;
        const uint16_t* src = a.q + (long long)(it.row0 + (live ? tok : 0)) * a.q_stride +
                              (long long)(it.kvh * a.G + row - tok * a.G) * D + 16 * t;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4*>(src + 64 * grp + 8 * j);
            qa[r][grp][j][0] = __byte_perm(x.x, x.z, 0x5410);
            qa[r][grp][j][1] = __byte_perm(x.x, x.z, 0x7632);
            qa[r][grp][j][2] = __byte_perm(x.y, x.w, 0x5410);
            qa[r][grp][j][3] = __byte_perm(x.y, x.w, 0x7632);
            const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sum += __uint_as_float(p[i] << 16) + __uint_as_float(p[i] & 0xFFFF0000u);
          }
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          qsum[r][grp] = sum;
        }
      }
      float m[RT], l[RT], off[RT][NG], o[NG][2][4][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        m[r] = kNone;
        l[r] = 0.0f;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) off[r][grp] = 0.0f;
      }
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[grp][h][i][c] = 0.0f;

      const long long room = sp.units - done;
      const int stop = (long long)(it.cnt - k) <= room ? it.cnt : k + (int)room;
      const bool ends = stop == it.cnt;
      for (; k < stop; ++k, ++done) {
        const int s = (int)(done % STAGES);
        if (!mbar_wait(full(warp, s), (uint32_t)((done / STAGES) & 1), a.err)) {
          ok = false;
          break;
        }
        if (bad[warp * STAGES + s]) {  // nothing to see, or no such page
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(warp, s));
          continue;
        }
        const uint8_t* rec = ring + s * L::REC;
        const int tile = k < it.ns ? k : it.first + k - it.ns;
        const int key0 = tile << 4;

        // ---- scores of 16 keys: x[half][row][column]
        float x[2][RT][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          uint32_t kw[2 * NG], ks[2 * NG];
          lds(kw, rec + ((8 * nt + g) * 4 + t) * 8 * NG);
          lds(ks, rec + L::KS_OFF + (8 * nt + 2 * t) * 4 * NG);
          float acc[NG][4];
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[grp][c] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 4; i += 2)
                mma(acc[grp], qa[0][grp][j][i], kWide ? qa[RT - 1][grp][j][i] : 0u,
                    qa[0][grp][j][i + 1], kWide ? qa[RT - 1][grp][j][i + 1] : 0u,
                    code_pair(kw[2 * grp + j], i), code_pair(kw[2 * grp + j], i + 1));
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) v[r] = 0.0f;
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) {
              const float2 so = __half22float2(*reinterpret_cast<const __half2*>(&ks[c * NG + grp]));
#pragma unroll
              for (int r = 0; r < RT; ++r)
                v[r] = fmaf(so.x, acc[grp][2 * r + c], fmaf(so.y, qsum[r][grp], v[r]));
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) x[nt][r][c] = v[r] * a.sc;
          }
        }
        // ---- masks: only records that some row does not see whole
        if (key0 + 15 > it.p0 ||
            (a.window > 0 && key0 <= it.p1 - a.window && key0 + 15 >= a.sinks)) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int key = key0 + 8 * nt + 2 * t + c;
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                bool see = key <= pos[r];
                if (a.window > 0) see = see && (key > pos[r] - a.window || key < a.sinks);
                if (!see) x[nt][r][c] = -INFINITY;
              }
            }
        }
        // ---- softmax: the reference maximum moves only by more than 2^8
        float alpha[RT];
        bool turn = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float top = fmaxf(fmaxf(x[0][r][0], x[0][r][1]), fmaxf(x[1][r][0], x[1][r][1]));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const float to = top > m[r] + 8.0f ? top : m[r];
          alpha[r] = ex2(m[r] - to);
          turn |= to != m[r];
          m[r] = to;
        }
        if (__any_sync(0xFFFFFFFFu, turn)) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            l[r] *= alpha[r];
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) off[r][grp] *= alpha[r];
          }
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[grp][h][i][c] *= alpha[kWide ? c >> 1 : 0];
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              x[nt][r][c] = ex2(x[nt][r][c] - m[r]);
              l[r] += x[nt][r][c];
            }
        // ---- values
        uint32_t vw[2][2 * NG], vs[2][2 * NG];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          lds(vw[nt], rec + L::V_OFF + ((4 * nt + t) * 8 + g) * 8 * NG);
          lds(vs[nt], rec + L::VS_OFF + (8 * nt + 2 * t) * 4 * NG);
        }
        __syncwarp();  // every lane has read the record
        if (lane == 0) mbar_arrive(empty(warp, s));
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          uint32_t hi[2][RT], lo[2][RT];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&vs[nt][grp]));
            const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&vs[nt][NG + grp]));
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              // a key that a row does not see has weight 0: its record may hold anything
              const float p0 = x[nt][r][0], p1 = x[nt][r][1];
              off[r][grp] += (p0 == 0.0f ? 0.0f : p0 * s0.y) + (p1 == 0.0f ? 0.0f : p1 * s1.y);
              split2(p0 == 0.0f ? 0.0f : p0 * s0.x, p1 == 0.0f ? 0.0f : p1 * s1.x, &hi[nt][r],
                     &lo[nt][r]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = code_pair(vw[0][2 * grp + h], i), b1 = code_pair(vw[1][2 * grp + h], i);
              if constexpr (kWide) {
                mma(o[grp][h][i], hi[0][0], hi[0][RT - 1], hi[1][0], hi[1][RT - 1], b0, b1);
                mma(o[grp][h][i], lo[0][0], lo[0][RT - 1], lo[1][0], lo[1][RT - 1], b0, b1);
              } else {
                mma(o[grp][h][i], hi[0][0], lo[0][0], hi[1][0], lo[1][0], b0, b1);
              }
            }
        }
      }
      if (!ok) break;

      // ---- the segment's sums: l, the offsets' part, and the low halves' rows
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          off[r][grp] += __shfl_xor_sync(0xFFFFFFFFu, off[r][grp], 1);
          off[r][grp] += __shfl_xor_sync(0xFFFFFFFFu, off[r][grp], 2);
        }
      }
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* v = o[grp][h][i];
            if constexpr (kWide) {
              v[0] += off[0][grp]; v[1] += off[0][grp];
              v[2] += off[RT - 1][grp]; v[3] += off[RT - 1][grp];
            } else {
              v[0] += v[2] + off[0][grp];
              v[1] += v[3] + off[0][grp];
            }
          }
      if (ends && !first_piece) {
        // the whole item: dims 64 group + 16 t + 8 c + 4 h + i of row g (+ 8)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int row = it.rt * ROWS + g + 8 * r;
          const int tok = row / a.G;
          if (tok >= it.n) continue;
          const float inv = l[r] > 0.0f ? 1.0f / l[r] : (l[r] == 0.0f ? 0.0f : l[r]);
          uint16_t* dst = a.out + ((long long)(it.row0 + tok) * a.H + it.kvh * a.G + row - tok * a.G) * D + 16 * t;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack16(o[grp][e >> 1][2 * (e & 1)][2 * r + c] * inv,
                              o[grp][e >> 1][2 * (e & 1) + 1][2 * r + c] * inv);
              *reinterpret_cast<uint4*>(dst + 64 * grp + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
      } else {
        // a piece: an item's end or middle goes to the head slot, its beginning to the ring
        // (whose copies have all been read: this is the span's last segment)
        float* piece = reinterpret_cast<float*>(first_piece ? smem + C::SM_HEAD + warp * C::PIECE
                                                            : smem + C::SM_RING + warp * C::RING);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float* dst = piece + (g + 8 * r) * C::LD + 16 * t;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float4*>(dst + 64 * grp + 8 * c + 4 * h) =
                    make_float4(o[grp][h][0][2 * r + c], o[grp][h][1][2 * r + c],
                                o[grp][h][2][2 * r + c], o[grp][h][3][2 * r + c]);
          if (t == 0) {
            piece[ROWS * C::LD + g + 8 * r] = m[r];
            piece[ROWS * C::LD + ROWS + g + 8 * r] = l[r];
          }
        }
        if (lane == 0) {
          int* id = seg_item[warp] + (first_piece ? 0 : 3);
          id[0] = it.b;
          id[1] = it.rt;
          id[2] = it.kvh;
        }
        flags |= first_piece ? (ends ? 3 : 1) : 4;
      }
      first_piece = false;
      if (ends && done < sp.units) {
        k = 0;
        next_item<ROWS>(a, it);
      }
    }
    if (lane == 0) seg_flags[warp] = flags;
  }
  __syncthreads();

  // ---- join the pieces that meet in this block
  Meta meta = {0, 0, 0, 0};
  int start = -1;       // warp whose last piece began the chain; -2: it began in an earlier block
  int from = 0;         // first head piece of the chain
  auto emit = [&](int last, bool ended) {
    // pieces: start's ring (where start >= 0), then the heads of warps from .. last
    const int* id = start >= 0 ? seg_item[start] + 3 : seg_item[from];
    const int b = id[0], rt = id[1], kvh = id[2];
    const bool whole = start >= 0 && ended;
    float* part = nullptr;
    if (!whole) {
      part = piece_at(a.ws, D, blk, start >= 0 ? 1 : 0);
      if (start >= 0) {
        meta.flags |= 4;
        meta.b = b;
        meta.rt = rt;
        meta.kvh = kvh;
      } else {
        meta.flags |= ended ? 3 : 1;
      }
    }
    Kv4Seq sq = {};
    if (whole) sq = kv4_seq(a.req, b, a.err);
    auto piece = [&](int w) {
      return reinterpret_cast<const float*>(w < from ? smem + C::SM_RING + start * C::RING
                                                     : smem + C::SM_HEAD + w * C::PIECE);
    };
    const int w0 = start >= 0 ? from - 1 : from;
    for (int e = threadIdx.x; e < ROWS * (D / 4); e += C::THREADS) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      float top = kNone;
      for (int w = w0; w <= last; ++w)
        if (w < from || (seg_flags[w] & 1)) top = fmaxf(top, piece(w)[ROWS * C::LD + r]);
      float sum = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
      for (int w = w0; w <= last; ++w) {
        if (w >= from && !(seg_flags[w] & 1)) continue;
        const float* p = piece(w);
        const float f = ex2(p[ROWS * C::LD + r] - top);
        sum = fmaf(f, p[ROWS * C::LD + ROWS + r], sum);
        const float4 x = *reinterpret_cast<const float4*>(p + r * C::LD + d);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (whole) {
        const int row = rt * ROWS + r, tok = row / a.G;
        if (tok < sq.n) {
          const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
          uint16_t* dst = a.out + ((long long)(sq.row0 + tok) * a.H + kvh * a.G + row - tok * a.G) * D + d;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack16(v.x * inv, v.y * inv), pack16(v.z * inv, v.w * inv));
        }
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = v;
        if (d == 0) {
          part[16 * D + r] = top;
          part[16 * D + 16 + r] = sum;
        }
      }
    }
  };
  for (int w = 0; w < NW; ++w) {
    const int f = seg_flags[w];
    if (f & 1) {
      if (start == -1) {
        start = -2;
        from = w;
      }
      if (f & 2) {
        emit(w, true);
        start = -1;
      }
    }
    if (f & 4) {
      start = w;
      from = w + 1;
    }
  }
  if (start != -1) emit(NW - 1, false);
  if (threadIdx.x == 0) reinterpret_cast<Meta*>(a.ws + kMetaOff)[blk] = meta;
}

// Joins the items that are cut between blocks: block (c, row) the one whose
// beginning is block c's last piece, with the first pieces of the blocks behind it.
template <int D, int ROWS>
__global__ void __launch_bounds__(D) kv4_join_kernel(const Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, r = blockIdx.y, d = threadIdx.x;
  const int blocks = *reinterpret_cast<const int*>(a.ws);
  if (c >= blocks) return;
  const Meta* meta = reinterpret_cast<const Meta*>(a.ws + kMetaOff);
  const Meta me = meta[c];
  if (!(me.flags & 4)) return;
  const Kv4Seq sq = kv4_seq(a.req, me.b, a.err);
  const int row = me.rt * ROWS + r, tok = row / a.G;
  if (tok >= sq.n) return;
  const float* p = piece_at(a.ws, D, c, 1);
  float top = p[16 * D + r], sum = p[16 * D + 16 + r], v = p[r * D + d];
  for (int e = c + 1; e < blocks; ++e) {
    const int f = meta[e].flags;
    if (!(f & 1)) continue;
    const float* x = piece_at(a.ws, D, e, 0);
    const float xm = x[16 * D + r];
    const float to = fmaxf(top, xm);
    const float fa = ex2(top - to), fb = ex2(xm - to);
    sum = fa * sum + fb * x[16 * D + 16 + r];
    v = fa * v + fb * x[r * D + d];
    top = to;
    if (f & 2) break;
  }
  const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
  const __nv_bfloat16 y = __float2bfloat16_rn(v * inv);
  a.out[((long long)(sq.row0 + tok) * a.H + me.kvh * a.G + row - tok * a.G) * D + d] =
      *reinterpret_cast<const uint16_t*>(&y);
}

template <int D, bool kWide>
cudaError_t launch(const Args& a, cudaStream_t s) {
  using C = Cfg<D, kWide>;
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !done[dev]) {
    e = cudaFuncSetAttribute(kv4_attn_kernel<D, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int blocks = num_sms() < kMaxBlocks ? num_sms() : kMaxBlocks;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_attn_kernel<D, kWide>, a, 2);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)blocks, C::ROWS);
  cfg.blockDim = dim3(D);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, C::ROWS>, a);
}

}  // namespace

size_t kv4_attention_workspace(int64_t D) {
  return kPieceOff + 2 * kMaxBlocks * piece_floats((int)D) * sizeof(float);
}

cudaError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t H, const Kv4Req& req,
                                 const Kv4Cache& cache, float scale, int64_t window, int64_t sinks,
                                 uint16_t* out, void* workspace, int* err, cudaStream_t s) {
  Args a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.H = (int)H;
  a.G = (int)(H / cache.Hkv);
  a.req = req;
  a.cache = cache;
  a.sc = scale * 1.4426950408889634f;
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.out = out;
  a.ws = static_cast<uint8_t*>(workspace);
  a.err = err;
  // rows of a request's tile: 8 where the batch's average request has no more
  const int64_t rows = a.G * ((req.T + req.B - 1) / req.B);
  const bool wide = rows > 8;
  if (cache.D == 64) return wide ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return wide ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace qk
