// kv4_attn.cu -- attention of a few new tokens per request over the 4-bit paged
// key/value cache (kv4.cuh), causal, with an optional sliding window and first
// tokens that stay visible.
//
// For query row i at position p (the rows are the last tokens of their request),
// over the visible keys j <= p with j > p - window or j < sinks:
//     x_j = scale sum_groups [ sK_jg (q_g . cK_jg) + oK_jg sum(q_g) ]
//     P_j = 2^((x_j - max) log2 e),   l = sum_j P_j
//     out = 1/l sum_j [ (P_j sV_jg) cV_j + P_j oV_jg ]
// No dequantized K or V exists anywhere.  A code 0..15 in bits 0-3 of an fp16 word
// of exponent 0 is the subnormal c 2^-24, in bits 4-7 it is 16 c 2^-24: one
// and-mask turns two nibbles of a word into an operand pair, and five instructions
// (a shift by 8 and four masks) a word of 8 codes into four.  The 16 goes into q
// (K) or into the end of the sums (V).  The other operands are fp16 too:
//  * q, times a power of two per row that puts its largest element into
//    [2^13, 2^14): exact, but for elements 2^-23 below the largest; sum(q_g) in three
//    pieces (33 bits), columns of one more product with the offsets;
//  * P sV: a row's reference is its maximum less what puts the largest P sV of the
//    record where it was set into [2^5, 2^6) (or the maximum's weight to 2^69, where
//    only values of scale 0 have much of it); a score 2^8 above that maximum sets it
//    anew, and so does a product of 2^15.  So P sV has 11 bits of significand down to
//    2^-19 of one that the row has met, and an error of 2^-30 of that one below.  P oV
//    and l stay in fp32.
// Sums are fp32 throughout.
//
// Bound: HBM (9 D / 8 bytes per visible token and kv head) and, about as much, the issue
// of instructions: 239 per record of 16 tokens (D = 128), 83 of them the unpacking.  64
// requests of 16384 tokens, 8 kv heads: 1.21 GB in 203 us (91 % of the copy rate) at 1965
// MHz; in a stream of seconds the power limit takes the clock to about 1650 MHz, and the
// kernel follows it (244 us).  Few records are bound by latency: 9.7 us for one
// request of 500 tokens, most of it the loads that depend on one another (lengths,
// page, record; metas, pieces).
// mma.sync is used rather than tcgen05 because its operands are registers: a
// tcgen05 tile of 128 would have to write the unpacked codes to shared memory (2
// bytes per code written and read, against half a byte loaded) to multiply them
// with the 1 to 16 rows there are.  The codes are the operand of 16 rows (keys for
// the scores, dims for the output) and the queries the one of 8 columns, so that
// eight rows of queries waste nothing.
//
// Layout of the work: an item is (request, row tile, kv head), its units are the
// 16-token records it sees.  All units of all items are laid end to end and cut
// into equal spans, one per warp, from the lengths on the device: one
// long request and a ragged batch fill the GPU alike, and no length goes through
// the host.  A warp that holds a whole item writes the output; the pieces of an
// item that is cut are joined in the block (through shared memory), and, where
// the cut is between blocks, by kv4_join_kernel from the workspace, in the order
// of the units: no atomics, the same bits on every run.
//
// A warp copies its records itself, four ahead, with 16-byte asynchronous copies of all
// its lanes, and numbers them itself, 32 units at a time and a lane to a unit (the walk
// over the items, the pages' ids).  It works in runs of records that are alike, so
// that a record's own work is in no loop with checks.  (A producer warp that issued
// bulk copies for the others, a lane after the other, took 109 cycles a record: 208 us
// at 64 x 16384 with no arithmetic at all.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kv4_chunk.h"
#include "kv4_items.cuh"
#include "sm100.cuh"

namespace qk {
namespace {

// NT tiles of 8 query rows per item.
template <int D, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  // Warps; the registers of the SM over four quarters.  (Times of each choice and its neighbours
  // as they were when it was made, not the present ones.)  D = 128: 12 of 168 registers (15 of
  // 128 spill a little: 236 us against 231 for 11 of 168, 64 x 16384), with two tiles 8 of
  // 255 (11 of 168 spill: 70 us against 62, 200 rows over 2500 tokens).  D = 64: 16
  // of 122 (12: 42.4 us against 40.5, 32 requests of 16384), with two tiles 8 of 207 (12
  // of 168: the same on long batches, 10.0 us against 8.9 on 4 requests of 500: what the
  // block leaves free of the SM lets the join's blocks start beside it).
  static constexpr int NW = D == 64 ? (NT == 1 ? 16 : 8) : (NT == 1 ? 12 : 8);
  static constexpr int WINDOW = 32;                    // units numbered at once
  static constexpr int STAGES = 4;                     // records in a warp's ring (six were no faster)
  static constexpr int THREADS = 32 * NW;
  static constexpr int LD = D + 4;                     // floats per row of a piece in shared memory
  static constexpr int PIECE = (ROWS * LD + 2 * ROWS) * 4;  // O rows, then every row's (m, l)
  static constexpr int RING = STAGES * Kv4<D>::REC;
  static constexpr int SM_RING = 0;
  static constexpr int SM_HEAD = SM_RING + NW * RING;  // piece of an item that began before the span
  static constexpr int SM_IDX = SM_HEAD + NW * PIECE;  // two windows of records' numbers
  static constexpr int SMEM = SM_IDX + NW * 2 * WINDOW * 4 + 128;
  static_assert(PIECE <= RING, "a span's last piece is kept in its ring");
  static_assert(SM_HEAD % 16 == 0 && SM_IDX % 16 == 0, "alignment");
  static_assert(SMEM + 24 * (THREADS + 64) <= 232448, "with the static shared memory");
};

// ---- workspace: the number of blocks with work, a Meta per block, then two pieces per block
// (of its first item, where that began in an earlier block, and of its last)
struct Meta {
  int flags;  // 1: a first piece, 2: it ends its item, 4: a last piece, of
  int rt, kvh, row0, n;  // this row tile and kv head of the request with these rows
  int pad[3];
};
static_assert(sizeof(Meta) == 32, "read as two 16-byte words");
constexpr size_t kMetaOff = 256;
constexpr size_t kPieceOff = kMetaOff + kMaxBlocks * sizeof(Meta);
__host__ __device__ constexpr size_t piece_floats(int D) { return (size_t)16 * (D + 2); }

__device__ __forceinline__ float* piece_at(uint8_t* ws, int D, int block, int which) {
  return reinterpret_cast<float*>(ws + kPieceOff) + (size_t)(2 * block + which) * piece_floats(D);
}

constexpr uint32_t kNoRecord = 0xFFFFFFFFu;

// Record number (over the whole cache) of unit k of an item, from the id of its page.
__device__ __forceinline__ int page_of(const Kv4Args& a, const Item& it, int k) {
  return quot(record_of(it, k), a.by_page);
}
__device__ __forceinline__ int page_id(const Kv4Args& a, const Item& it, int k) {
  if (it.p1 < 0) return 0;  // (an empty unit)
  return __ldg(a.req.page_table + (long long)it.b * a.req.max_pages + page_of(a, it, k));
}
__device__ __forceinline__ uint32_t record_number(const Kv4Args& a, const Item& it, int k, int id) {
  if (it.p1 < 0) return kNoRecord;
  if (id < 0 || id >= a.cache.num_pages) {
    record_index(a.err);
    return kNoRecord;
  }
  const int in = record_of(it, k) - page_of(a, it, k) * a.by_page.d;
  return ((uint32_t)id * (uint32_t)a.cache.Hkv + (uint32_t)it.kvh) * (uint32_t)a.by_page.d + (uint32_t)in;
}

// kBytes (16, or 8 or 4), kAt bytes behind both addresses.
template <int kBytes, int kAt>
__device__ __forceinline__ void copy(uint32_t dst, const uint8_t* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%2], 16;" ::"r"(dst), "l"(src), "n"(kAt) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0+%2], [%1+%2], %3;" ::"r"(dst), "l"(src), "n"(kAt), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, 16 x 8 x 16, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements, two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// 4 N bytes at a shared address; kOff: more bytes.
template <int kOff, int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], uint32_t at) {
  static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at), "n"(kOff));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2+%3];" : "=r"(r[0]), "=r"(r[1]) : "r"(at), "n"(kOff));
  else
    asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(r[0]) : "r"(at), "n"(kOff));
}

// The largest finite scale of a key's groups.
template <int N>
__device__ __forceinline__ float largest_scale(const uint32_t (&t)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float s = unpack_f16(t[i]).x;
    m = s < INFINITY ? fmaxf(m, s) : m;
  }
  return m;
}

// Over the lanes of equal lane % 4: over the keys, for a query row's column.
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

constexpr float kNone = -1.0e30f;   // the reference maximum of a row that has seen nothing

// Rows of P sV of 16 keys as fp16 (b0, b1 of the second product, one group).  With
// masks, a key that a row does not see has weight 0 whatever its record holds.
template <bool kMask>
__device__ __forceinline__ void weigh(const float (&p)[4], float s0, float s1, uint32_t (&w)[2]) {
  float v[4] = {p[0] * s0, p[1] * s0, p[2] * s1, p[3] * s1};
  if (kMask) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[i] == 0.0f ? 0.0f : v[i];
  }
  w[0] = pack_f16(v[0], v[1]);
  w[1] = pack_f16(v[2], v[3]);
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::THREADS, 1) kv4_attn_kernel(const Kv4Args a) {
  using C = Cfg<D, NT>;
  using L = Kv4<D>;
  constexpr int NG = L::NG, ROWS = C::ROWS, NW = C::NW, STAGES = C::STAGES, WINDOW = C::WINDOW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem<128>(smem_raw);
  __shared__ Kv4Scan<NW> scan;
  __shared__ int seg_flags[32];
  __shared__ __align__(16) int seg_item[NW][4];  // last piece's rt, kvh, row0, n
  __shared__ __align__(16) int ahead[NW][4];     // the next unit to be numbered: b, rt, kvh, unit of the item
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int blk = blockIdx.x;
  uint32_t* number = reinterpret_cast<uint32_t*>(smem + C::SM_IDX) + warp * 2 * WINDOW;

  pdl_launch_dependents();
  pdl_wait();

  // ---- units in all
  const int per = (a.req.B + C::THREADS - 1) / C::THREADS;
  scan_units<ROWS, 4>(a, scan, per, warp);
  const long long W = scan.pre[C::THREADS];
  // Where there are fewer units than warps, a unit to a warp; where there are less than
  // twice as many, two to a warp, and fewer blocks (257 units of 8 items: 8.9 us against 9.9
  // with two; 2056 units of 8: 11.2 us against 11.5 with one and some warps with two).
  const long long warps = (long long)gridDim.x * NW;
  const int least = W <= warps ? 1 : 2;
  const int blocks = W >= warps * least ? (int)gridDim.x : ((int)W + NW * least - 1) / (NW * least);
  if (blk == 0 && threadIdx.x == 0) *reinterpret_cast<int*>(a.ws) = blocks;
  if (blk >= blocks) return;  // the whole block

  Item it = {};
  int units = 0, k = 0;  // of this warp's span; the unit of the item that it begins with
  uint4 raw[NT][NG][2];  // this lane's query elements of a segment: row g, dims 16 t ..
  auto load_queries = [&]() {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = it.rt * ROWS + 8 * n + g;
      const int tok = quot(row, a.by_g);
      const bool live = tok < it.n;
      const uint16_t* src = a.q + (long long)(it.row0 + (live ? tok : 0)) * a.q_stride +
                            (long long)(it.kvh * a.G + row - tok * a.G) * D + 16 * t;
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          raw[n][grp][j] = make_uint4(0, 0, 0, 0);
          if (live) raw[n][grp][j] = *reinterpret_cast<const uint4*>(src + 64 * grp + 8 * j);
        }
    }
  };
  {
    // ---- this warp's span of W / slots units (one more for the first W % slots), and
    // the item it starts in
    const int slot = blk * NW + warp, slots = blocks * NW;
    const long long each = W >> 31 ? W / slots : (long long)((uint32_t)W / (uint32_t)slots);
    const int more = (int)(W - each * slots);
    const long long u0 = each * slot + min(slot, more);
    const long long all = each + (slot < more ? 1 : 0);
    const bool hours = all > 0x7FFFFF00ll;  // of work for one warp
    if (hours) record_timeout(a.err);
    units = hours ? 0 : (int)all;
    if (units > 0) {
      if (!locate_unit<ROWS, 4>(a, scan, per, u0, it, k)) units = 0;
      // (the ids of the first pages are on their way while the queries' addresses are made)
      if (it.p1 >= 0 && k + lane < it.cnt)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.req.page_table + (long long)it.b * a.req.max_pages +
                                                     page_of(a, it, k + lane)));
      load_queries();
    }
  }

  {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* ring = smem + C::SM_RING + warp * C::RING;
    // this lane's places in a record: codes of tokens g, g + 8; of pairs t, t + 4
    const uint32_t ring_k = smem_u32(ring) + (g * 4 + t) * 8 * NG;
    const uint32_t ring_v = smem_u32(ring) + L::V_OFF + (t * 8 + g) * 8 * NG;
    const uint32_t ring_s = smem_u32(ring) + L::KS_OFF + g * 4 * NG;
    bool first_piece = k > 0;
    int flags = 0;
    int done = 0;   // units worked on
    int asked = 0;  // units whose copies are issued, or passed over
    int known = 0;  // units that are numbered
    const uint32_t ring_dst = smem_u32(ring) + 16 * lane;
    uint32_t missing = 0, missing_next = 0;  // units of `done`'s window, and of the next, with no record
    // Numbers the next window of units, from unit u of an item on, a lane each; the units
    // of one item look their pages up together.
    auto number_from = [&](Item at, int u) {
      int have = 0;
      const int want = min(WINDOW, units - known);
      uint32_t mine = kNoRecord;
      while (have < want) {
        const int n = min(want - have, at.cnt - u), e = u + lane - have;
        if (lane >= have && lane < have + n) mine = record_number(a, at, e, page_id(a, at, e));
        have += n;
        u += n;
        if (u == at.cnt && known + have < units) {
          u = 0;
          next_item<ROWS>(a, at);
        }
      }
      const uint32_t none = __ballot_sync(0xFFFFFFFFu, mine == kNoRecord);
      (known == 0 ? missing : missing_next) = none;
      // (a record that is not there: the first one is copied in its place, and masked)
      number[(known + lane) % (2 * WINDOW)] = mine == kNoRecord ? 0u : mine;
      known += want;
      __syncwarp();
      if (lane == 0) *reinterpret_cast<int4*>(ahead[warp]) = make_int4(at.b, at.rt, at.kvh, u);
      __syncwarp();
    };
    auto number_more = [&]() {
      const int4 from = *reinterpret_cast<const int4*>(ahead[warp]);
      Item at;
      at.b = from.x;
      at.rt = from.y;
      at.kvh = from.z;
      if (per == 1)
        set_request<ROWS>(a, at, scan.seqs[at.b]);
      else
        load_request<ROWS>(a, at);
      load_tile<ROWS>(a, at);
      number_from(at, from.w);
    };
    // A unit's copies into its place in the ring.
    auto fetch = [&](int unit, uint32_t place) {
      uint32_t rec[1];
      lds<0>(rec, smem_u32(number) + unit % (2 * WINDOW) * 4);
      const uint8_t* src = a.cache.base + (unsigned long long)rec[0] * L::REC + 16 * lane;
      const uint32_t dst = ring_dst + place;
      copy<16, 0>(dst, src);
      copy<16, 512>(dst, src);
      if constexpr (NG == 2) {
        copy<16, 1024>(dst, src);
        copy<16, 1536>(dst, src);
      }
      static_assert(L::KS_OFF == 1024 * NG && L::REC - L::KS_OFF == 32 * 4 * NG, "the copies");
      copy<4 * NG, L::KS_OFF>(dst - (16 - 4 * NG) * lane, src - (16 - 4 * NG) * lane);
    };
    if (units > 0) number_from(it, k);
#pragma unroll 1
    for (; asked < STAGES; ++asked) {
      if (asked < units) fetch(asked, asked * L::REC);
      copies_commit();
    }
    uint32_t place = 0;  // of unit `done` in the ring, and then of unit `asked`
    while (done < units) {
      // ---- a segment: this span's units of one item
      // queries: fragments of row g (per j and half of a word's nibbles, the second
      // of a pair a 16th); sums and factors of rows 2 t, 2 t + 1, the columns of the scores
      uint32_t qb[NT][NG][2][4];
      uint32_t qo[NT];  // sum(q) per group in three fp16 pieces, a lane of the row to a piece
      float R[NT][2];
      int pos[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top = 0.0f, sum[NG];
#pragma unroll
        for (int grp = 0; grp < NG; ++grp)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {raw[n][grp][j].x, raw[n][grp][j].y, raw[n][grp][j].z, raw[n][grp][j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf_lo(w[i])), fabsf(bf_hi(w[i]))));
          }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // times 2^-e, the largest element comes into [2^13, 2^14)
        const int e = min(max(top == 0.0f ? 0 : exponent(top) - 13, -113), 113);
        const float f = pow2(-e);
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          sum[grp] = 0.0f;  // in the queries' unit: of rows near the largest bf16 it may leave fp32's range
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = raw[n][grp][j];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[grp] += fmaf(bf_lo(w[i]), f, bf_hi(w[i]) * f);
            qb[n][grp][j][0] = pack_f16(bf_lo(v.x) * f, bf_lo(v.z) * f);
            qb[n][grp][j][1] = pack_f16(bf_hi(v.x) * f * 0.0625f, bf_hi(v.z) * f * 0.0625f);
            qb[n][grp][j][2] = pack_f16(bf_lo(v.y) * f, bf_lo(v.w) * f);
            qb[n][grp][j][3] = pack_f16(bf_hi(v.y) * f * 0.0625f, bf_hi(v.w) * f * 0.0625f);
          }
          sum[grp] += __shfl_xor_sync(0xFFFFFFFFu, sum[grp], 1);
          sum[grp] += __shfl_xor_sync(0xFFFFFFFFu, sum[grp], 2);
        }
        // (up to 2^20 in the queries' unit: 2^-7 brings it into fp16's range)
        float piece[2] = {0.0f, 0.0f};
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          float rest = sum[grp] * 0x1p-7f;
          const float first = __half2float(__float2half_rn(rest));
          rest = t == 0 ? first : rest - first;
          const float second = __half2float(__float2half_rn(rest));
          rest = t <= 1 ? second : rest - second;
          piece[grp] = t == 3 ? 0.0f : rest;
        }
        qo[n] = pack_f16(piece[0], piece[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int from = 4 * (2 * t + c);  // a lane of row 2 t + c
          const int ec = __shfl_sync(0xFFFFFFFFu, e, from);
          // the scores' unit: x = 2^(24 + e) times what the codes' product gives
          // (neither 0 nor infinite: a masked score is -inf, one of 0 stays 0)
          R[n][c] = fminf(fmaxf(a.sc * pow2(ec) * 0x1p24f, 1.0e-35f), 3.0e38f);
          const int rc = it.rt * ROWS + 8 * n + 2 * t + c;
          const int tc = quot(rc, a.by_g);
          pos[n][c] = tc < it.n ? it.len - it.n + tc : -1;
        }
      }
      // nm: minus the reference, in units of log2; lim: the score that moves it (the
      // maximum and 2^8); o: rows g (even dims) and g + 8 (odd dims, 16-fold)
      float nm[NT][2], lim[NT][2], l[NT][2], off[NT][2][NG], o[NT][NG][2][2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          nm[n][c] = -fmaxf(kNone * R[n][c], kLeast);
          lim[n][c] = kNone;
          l[n][c] = 0.0f;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) off[n][c][grp] = 0.0f;
        }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int grp = 0; grp < NG; ++grp)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[n][grp][i >> 3][(i >> 2) & 1][i & 3] = 0.0f;
      auto rescale = [&](int n, const float (&alpha)[2]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[n][c] *= alpha[c];
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) off[n][c][grp] *= alpha[c];
        }
#pragma unroll
        for (int grp = 0; grp < NG; ++grp)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[n][grp][i >> 3][(i >> 2) & 1][i & 3] *= alpha[i & 1];
      };

      const int room = units - done;
      const int stop = it.cnt - k <= room ? it.cnt : k + room;
      const bool ends = stop == it.cnt;
      // A record: kMask where a row may not see all of its keys, dead where it is not there.
      bool fresh = true;  // nothing is summed yet
      auto step = [&](auto masks, int record, bool dead, bool more) {
        constexpr bool kMask = decltype(masks)::value;
        copies_wait<STAGES - 1>();
        __syncwarp();
        const uint32_t at_k = ring_k + place, at_v = ring_v + place, at_s = ring_s + place;
        // ---- scores: x[n][i], i = 0, 1 key g and rows 2 t, 2 t + 1; i = 2, 3 key g + 8
        float x[NT][4];
        {
          uint32_t k0[2 * NG], k1[2 * NG], s0[NG], s1[NG];
          lds<0>(k0, at_k);
          lds<8 * 4 * 8 * NG>(k1, at_k);
          lds<0>(s0, at_s);
          lds<8 * 4 * NG>(s1, at_s);
          // the offsets' part, 2^17-fold: keys by groups, times groups by rows, a pair of
          // columns to each piece of the sums
          const uint32_t o0 = NG == 2 ? __byte_perm(s0[0], s0[NG - 1], 0x7632) : s0[0] >> 16;
          const uint32_t o1 = NG == 2 ? __byte_perm(s1[0], s1[NG - 1], 0x7632) : s1[0] >> 16;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t c = k0[2 * grp + j], d = k1[2 * grp + j];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma(acc[n], c & 0x000F000Fu, d & 0x000F000Fu, c & 0x00F000F0u, d & 0x00F000F0u,
                      qb[n][grp][j][2 * h], qb[n][grp][j][2 * h + 1]);
                c >>= 8;
                d >>= 8;
              }
            }
            const float a0 = unpack_f16(s0[grp]).x, a1 = unpack_f16(s1[grp]).x;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                x[n][c] = grp == 0 ? a0 * acc[n][c] : fmaf(a0, acc[n][c], x[n][c]);
                x[n][2 + c] = grp == 0 ? a1 * acc[n][2 + c] : fmaf(a1, acc[n][2 + c], x[n][2 + c]);
              }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma(acc, o0, o1, 0u, 0u, qo[n], 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = fmaf(acc[i], 0x1p-17f, x[n][i]);
          }
        }
        if constexpr (kMask) {
          const int key0 = (record << 4) + g;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + 4 * (i & 2), p = pos[n][i & 1];
              bool see = key <= p && !dead;
              if (a.window > 0) see = see && (key > p - a.window || key < a.sinks);
              if (!see) x[n][i] = -INFINITY;
            }
        }
        // ---- values and their scales; the record's place is free then
        uint32_t v0[2 * NG], v1[2 * NG], t0[NG], t1[NG];
        lds<0>(v0, at_v);
        lds<4 * 8 * 8 * NG>(v1, at_v);
        lds<16 * 4 * NG>(t0, at_s);
        lds<24 * 4 * NG>(t1, at_s);
        __syncwarp();  // every lane has read the record
        if (more) fetch(asked, place);
        copies_commit();
        ++asked;
        place = place == (STAGES - 1) * L::REC ? 0 : place + L::REC;
        // ---- weights, and times scales, as the second product's operand.  A row's reference
        // moves where a score passes the last maximum by 2^8, or a product comes to 2^15 (the
        // half then carries into its sign bit)
        uint32_t w[NT][NG][2];
        float y[NT][4];
        auto weights = [&]() {
          uint32_t big = 0;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp) {
            const float s0 = unpack_f16(t0[grp]).x, s1 = unpack_f16(t1[grp]).x;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              weigh<kMask>(y[n], s0, s1, w[n][grp]);
              big = __vmaxu2(big, __vmaxu2(w[n][grp][0], w[n][grp][1]));
            }
          }
          return ((big + 0x08000800u) & 0x80008000u) != 0;
        };
        auto exponentials = [&]() {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[n][i] = ex2(fmaf(x[n][i], R[n][i & 1], nm[n][i & 1]));
        };
        exponentials();
        bool move = weights();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) move |= fmaxf(x[n][c], x[n][2 + c]) > lim[n][c];
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, move), 0)) {
          const float m0 = largest_scale(t0), m1 = largest_scale(t1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float alpha[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float top = column_max(fmaxf(x[n][c], x[n][2 + c]));
              const float heavy = column_max(fmaxf(ex2((x[n][c] - top) * R[n][c]) * m0,
                                                   ex2((x[n][2 + c] - top) * R[n][c]) * m1));
              const float was = nm[n][c];
              const float set = reference(top * R[n][c], heavy);
              if (top > lim[n][c]) {
                nm[n][c] = set;
                lim[n][c] = top + 8.0f / R[n][c];
              } else if (top > -INFINITY && set < nm[n][c] - 8.0f) {
                nm[n][c] = set;  // products of 2^13 and more
              }
              alpha[c] = ex2(nm[n][c] - was);
            }
            if (!fresh) rescale(n, alpha);
          }
          exponentials();
          weights();
        }
        fresh = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          l[n][0] += y[n][0] + y[n][2];
          l[n][1] += y[n][1] + y[n][3];
        }
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          const float o0 = unpack_f16(t0[grp]).y, o1 = unpack_f16(t1[grp]).y;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float y0 = y[n][c], y1 = y[n][2 + c];
              if (kMask)
                off[n][c][grp] += (y0 == 0.0f ? 0.0f : y0 * o0) + (y1 == 0.0f ? 0.0f : y1 * o1);
              else
                off[n][c][grp] = fmaf(y0, o0, fmaf(y1, o1, off[n][c][grp]));
            }
        }
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            w[n][grp][0] = transpose8(w[n][grp][0]);
            w[n][grp][1] = transpose8(w[n][grp][1]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t c = v0[2 * grp + h], d = v1[2 * grp + h];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma(o[n][grp][h][i], c & 0x000F000Fu, c & 0x00F000F0u, d & 0x000F000Fu,
                    d & 0x00F000F0u, w[n][grp][0], w[n][grp][1]);
              c >>= 8;
              d >>= 8;
            }
          }
        }
      };
      while (k < stop) {
        // a run of records alike: in one window of numbers, with the numbers of the
        // units asked for known, and all masked or none
        const bool more = asked < units;
        if (more && asked == known) number_more();
        int n = min(stop - k, WINDOW - done % WINDOW);
        if (more) n = min(n, known - asked);
        const bool whole = k >= it.whole0 && k < it.whole1;
        if (whole) n = min(n, it.whole1 - k);
        if (k < it.whole0) n = min(n, it.whole0 - k);
        const uint32_t none = missing >> (done % WINDOW);
        const bool dead = none & 1u;
        if (none != 0) n = dead ? 1 : min(n, __ffs(none) - 1);
        const int end = k + n;
        if (whole && !dead) {
#pragma unroll 1
          for (; k < end; ++k) step(std::false_type{}, 0, false, more);
        } else {
#pragma unroll 1
          for (; k < end; ++k) step(std::true_type{}, record_of(it, k), dead, more);
        }
        done += n;
        if (done % WINDOW == 0) missing = missing_next;
      }
      // ---- the segment's sums: l and the offsets' part over the lanes of a row; then
      // z = O of row 2 t + c, dims 64 group + 8 g + 4 h + 2 i + (0, 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], d);
#pragma unroll
            for (int grp = 0; grp < NG; ++grp)
              off[n][c][grp] += __shfl_xor_sync(0xFFFFFFFFu, off[n][c][grp], d);
          }
        }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int grp = 0; grp < NG; ++grp)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float& z = o[n][grp][i >> 3][(i >> 2) & 1][i & 3];
            z = fmaf(z, (i & 2) ? 0x1p20f : 0x1p24f, off[n][i & 1][grp]);
          }
      if (ends && !first_piece) {
        // the whole item
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = it.rt * ROWS + 8 * n + 2 * t + c;
            const int tok = quot(row, a.by_g);
            if (tok >= it.n) continue;
            const float inv = l[n][c] > 0.0f ? 1.0f / l[n][c] : l[n][c];  // (0, or NaN)
            uint16_t* dst = a.out + ((long long)(it.row0 + tok) * a.H + it.kvh * a.G + row - tok * a.G) * D + 8 * g;
#pragma unroll
            for (int grp = 0; grp < NG; ++grp) {
              uint32_t y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[i] = pack_bf16(o[n][grp][i >> 1][i & 1][c] * inv, o[n][grp][i >> 1][i & 1][2 + c] * inv);
              *reinterpret_cast<uint4*>(dst + 64 * grp) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
      } else {
        // a piece: an item's end or middle goes to the head slot, its beginning to the ring
        // (this is the span's last segment: nothing is in flight or unread)
        float* piece = reinterpret_cast<float*>(first_piece ? smem + C::SM_HEAD + warp * C::PIECE
                                                            : smem + C::SM_RING + warp * C::RING);
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = 8 * n + 2 * t + c;
            float* dst = piece + row * C::LD + 8 * g;
#pragma unroll
            for (int grp = 0; grp < NG; ++grp)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float4*>(dst + 64 * grp + 4 * h) =
                    make_float4(o[n][grp][h][0][c], o[n][grp][h][0][2 + c], o[n][grp][h][1][c],
                                o[n][grp][h][1][2 + c]);
            if (g == 0) {
              *reinterpret_cast<float2*>(piece + ROWS * C::LD + 2 * row) = make_float2(-nm[n][c], l[n][c]);
            }
          }
        if (lane == 0 && !first_piece) {
          *reinterpret_cast<int4*>(seg_item[warp]) = make_int4(it.rt, it.kvh, it.row0, it.n);
        }
        flags |= first_piece ? (ends ? 3 : 1) : 4;
      }
      first_piece = false;
      if (ends && done < units) {
        k = 0;
        next_item<ROWS>(a, it);
        load_queries();
      }
    }
    if (lane == 0) seg_flags[warp] = flags;
    if (warp == 0 && lane >= NW) seg_flags[lane] = 0;
  }
  __syncthreads();

  // ---- join the pieces that meet in this block: a chain is a last piece (in its
  // warp's ring), if it began here, and the first pieces of the warps behind it
  // (A chain is found by its bits, and a warp takes whole rows of it: what one warp does
  // alone here costs four cycles an instruction at least.)
  const int my_flags = seg_flags[lane];
  const uint32_t heads = __ballot_sync(0xFFFFFFFFu, my_flags & 1);
  const uint32_t ends = __ballot_sync(0xFFFFFFFFu, my_flags & 2);
  const uint32_t tails = __ballot_sync(0xFFFFFFFFu, my_flags & 4);
  const float* rest = reinterpret_cast<const float*>(smem + C::SM_HEAD);
  constexpr int LPR = D / 4, RPW = 32 / LPR, TURNS = ROWS / RPW;  // lanes per row, rows per warp
  Meta meta = {};
  int first_warp = 0;  // of the chain's first rows
  // the chain's last piece, -1 where it began in an earlier block; the warps behind it
  int start = -1;
  uint32_t behind = 0xFFFFFFFFu;
  if (heads == 0 || (tails & ((heads & (0u - heads)) - 1u)) != 0) {
    start = tails != 0 ? __ffs(tails) - 1 : 32;
    behind = tails != 0 ? 0xFFFFFFFEu << start : 0u;
  }
#pragma unroll 1
  while (start < 32) {
    const uint32_t end = ends & behind & (0u - (ends & behind));  // the warp that ends it, or none
    const uint32_t parts = heads & behind & (end != 0 ? 2u * end - 1u : 0xFFFFFFFFu);
    const bool whole = start >= 0 && end != 0;
    // (the warps of a chain are next to each other)
    const int pieces = __popc(parts) + (start >= 0), from = start >= 0 ? start : __ffs(parts) - 1;
    int4 item = make_int4(0, 0, 0, 0);
    if (start >= 0) {
      item = *reinterpret_cast<const int4*>(seg_item[start]);
      if (!whole) {
        meta.flags |= 4;
        meta.rt = item.x;
        meta.kvh = item.y;
        meta.row0 = item.z;
        meta.n = item.w;
      }
    } else {
      meta.flags |= end != 0 ? 3 : 1;
    }
    const float* first = reinterpret_cast<const float*>(smem + C::SM_RING + max(start, 0) * C::RING);
    int turn = warp - first_warp;
    if (turn < 0) turn += NW;
#pragma unroll 1
    for (; turn < TURNS; turn += NW) {
      const int r = turn * RPW + lane / LPR, d = 4 * (lane % LPR);
      float top = kLeast, sum = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 1
      for (int q0 = 0; q0 < pieces; q0 += 4) {
        float4 x[4];
        float2 ml[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = min(q0 + j, pieces - 1);  // (behind the last one: it again, with weight 0)
          const float* p = start >= 0 && q == 0 ? first : rest + (from + q) * (C::PIECE / 4);
          ml[j] = *reinterpret_cast<const float2*>(p + ROWS * C::LD + 2 * r);
          x[j] = *reinterpret_cast<const float4*>(p + r * C::LD + d);
          if (q0 + j >= pieces) ml[j] = make_float2(-INFINITY, 0.0f);
        }
        const float most = fmaxf(fmaxf(top, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
        const float keep = ex2(top - most);
        top = most;
        sum *= keep;
        v = make_float4(v.x * keep, v.y * keep, v.z * keep, v.w * keep);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float f = ex2(ml[j].x - top);
          sum = fmaf(f, ml[j].y, sum);
          v.x = fmaf(f, x[j].x, v.x);
          v.y = fmaf(f, x[j].y, v.y);
          v.z = fmaf(f, x[j].z, v.z);
          v.w = fmaf(f, x[j].w, v.w);
        }
      }
      if (whole) {
        const int row = item.x * ROWS + r, tok = quot(row, a.by_g);
        if (tok < item.w) {
          const float inv = sum > 0.0f ? __frcp_rn(sum) : sum;
          uint16_t* dst = a.out + ((long long)(item.z + tok) * a.H + item.y * a.G + row - tok * a.G) * D + d;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        }
      } else {
        float* part = piece_at(a.ws, D, blk, start >= 0 ? 1 : 0);
        *reinterpret_cast<float4*>(part + r * D + d) = v;
        if (d == 0) *reinterpret_cast<float2*>(part + 16 * D + 2 * r) = make_float2(top, sum);
      }
    }
    first_warp = (first_warp + TURNS) % NW;
    const uint32_t left = end != 0 ? tails & behind & ~(end - 1u) : 0u;
    start = left != 0 ? __ffs(left) - 1 : 32;
    behind = 0xFFFFFFFEu << (start & 31);
  }
  if (threadIdx.x == 0) reinterpret_cast<Meta*>(a.ws + kMetaOff)[blk] = meta;
}

// Joins the items that are cut between blocks: block (c, row) the one whose
// beginning is block c's last piece, with the first pieces of the blocks behind it.
// D / 4 threads read a piece's row; the 512 / D groups of them take the pieces in turn,
// and then each other's sums.  A launch waits for two loads, one after the other:
// every block's Meta, and then the pieces' rows with their maxima and sums.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4Args a) {
  constexpr int TPP = D / 4, GROUPS = 128 / TPP, AHEAD = 4;
  __shared__ int flags[kMaxBlocks];
  __shared__ __align__(16) float red[GROUPS][D];
  __shared__ __align__(8) float2 red_ml[GROUPS];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31;
  const int blocks = *reinterpret_cast<const int*>(a.ws);
  const Meta* meta = reinterpret_cast<const Meta*>(a.ws + kMetaOff);
  const Meta me = meta[c];
  // (Metas behind the last block are not written, and not looked at)
  for (int e = threadIdx.x; e < gridDim.x; e += 128) flags[e] = meta[e].flags;
  if (c >= blocks || !(me.flags & 4)) return;
  __syncthreads();
  // the chain: blocks c + 1 .. last (a block with no first piece in it has no units)
  int last = blocks - 1;
  for (int e0 = c + 1; e0 < blocks; e0 += 32) {
    const int e = e0 + lane;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, e < blocks && (flags[e] & 2) != 0);
    if (hit != 0) {
      last = e0 + __ffs(hit) - 1;
      break;
    }
  }
  const int n = last - c + 1;
  const int grp = threadIdx.x / TPP, d = 4 * (threadIdx.x % TPP);
  float top = kLeast, sum = 0.0f;
  float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int i0 = grp; i0 < n; i0 += AHEAD * GROUPS) {
    float4 x[AHEAD];
    float2 ml[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j * GROUPS;
      x[j] = make_float4(0, 0, 0, 0);
      ml[j] = make_float2(kLeast, 0.0f);
      if (i < n && (i == 0 || (flags[c + i] & 1) != 0)) {
        const float* p = piece_at(a.ws, D, c + i, i == 0 ? 1 : 0);
        x[j] = *reinterpret_cast<const float4*>(p + r * D + d);
        ml[j] = *reinterpret_cast<const float2*>(p + 16 * D + 2 * r);
      }
    }
    float most = top;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) most = fmaxf(most, ml[j].x);
    const float keep = ex2(top - most);
    top = most;
    sum *= keep;
    v = make_float4(v.x * keep, v.y * keep, v.z * keep, v.w * keep);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const float f = ex2(ml[j].x - top);
      sum = fmaf(f, ml[j].y, sum);
      v.x = fmaf(f, x[j].x, v.x);
      v.y = fmaf(f, x[j].y, v.y);
      v.z = fmaf(f, x[j].z, v.z);
      v.w = fmaf(f, x[j].w, v.w);
    }
  }
  *reinterpret_cast<float4*>(&red[grp][d]) = v;
  if (d == 0) red_ml[grp] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x >= TPP) return;
  const int row = me.rt * ROWS + r, tok = quot(row, a.by_g);
  if (tok >= me.n) return;
  float most = kLeast;
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) most = fmaxf(most, red_ml[i].x);
  v = make_float4(0, 0, 0, 0);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    const float f = ex2(red_ml[i].x - most);
    const float4 x = *reinterpret_cast<const float4*>(&red[i][d]);
    sum = fmaf(f, red_ml[i].y, sum);
    v.x = fmaf(f, x.x, v.x);
    v.y = fmaf(f, x.y, v.y);
    v.z = fmaf(f, x.z, v.z);
    v.w = fmaf(f, x.w, v.w);
  }
  const float inv = sum > 0.0f ? __frcp_rn(sum) : sum;
  uint16_t* dst = a.out + ((long long)(me.row0 + tok) * a.H + me.kvh * a.G + row - tok * a.G) * D + d;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
}

template <int D, int NT>
cudaError_t launch(const Kv4Args& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !done[dev]) {
    e = cudaFuncSetAttribute(kv4_attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  e = cudaLaunchKernelEx(&cfg, kv4_attn_kernel<D, NT>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)blocks, C::ROWS);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, C::ROWS>, a);
}

// Whether kv4_chunk.cu's tiles of 128 rows are the faster ones: where the batch's average
// request fills three quarters of one per kv head, and there are tiles for most of the SMs.
// 128 rows a request over 2400 keys, 16 kv heads of 128: 8 requests 68 us (104 here), 4 (64
// tiles) 43 (59), but over 600 keys 30 (27); 96 rows, 8 requests: 65 (82); 64 rows: 64 (62).
// 300 rows, 8 kv heads, 4 requests (96 tiles): 55 us over 2400 keys (66), 31 over 600 (29).
// A prompt of 2048 tokens, 8 kv heads of 4 query heads: 124 us (466).
// The host knows T and B only, so the average counts the rows of nobody, and one long request
// decides for all: a prompt of 2048 beside 31 requests of one row over 8192 tokens takes 389 us,
// in two calls 123 + 59; beside 63 of two query heads per kv head 525, in two calls 69 + 106.
bool by_chunks(int64_t T, int64_t B, int64_t H, int64_t Hkv) {
  const int64_t rows = H / Hkv * ((T + B - 1) / B);
  return rows >= 96 && B * Hkv * ((rows + 127) / 128) >= 96;
}

}  // namespace

size_t kv4_attention_workspace(int64_t D) {
  return kv4_chunk_workspace(D);  // (the larger one)
}

size_t kv4_attention_workspace(int64_t D, int64_t T, int64_t B, int64_t H, int64_t Hkv) {
  if (by_chunks(T, B, H, Hkv)) return kv4_chunk_workspace(D);
  return kPieceOff + 2 * kMaxBlocks * piece_floats((int)D) * sizeof(float);
}

cudaError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t H, const Kv4Req& req,
                                 const Kv4Cache& cache, float scale, int64_t window, int64_t sinks,
                                 uint16_t* out, void* workspace, int* err, cudaStream_t s) {
  Kv4Args a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.H = (int)H;
  a.G = (int)(H / cache.Hkv);
  a.by_g = fast_div(a.G);
  a.by_page = fast_div(cache.page / 16);
  a.req = req;
  a.cache = cache;
  a.sc = scale * 1.4426950408889634f;
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.out = out;
  a.ws = static_cast<uint8_t*>(workspace);
  a.err = err;
  // Rows of an item: 8 where the batch's average request has no more per kv head, else 16.
  // 16 requests of 8192 tokens, 4 kv heads of 128: with 8 rows 24.9 us (16 to an item: 31.5),
  // with 9 31.6 (8 to an item, twice the cache: 41.0), with 16 31.8 (41.0).  A chunk of 200 rows
  // over 2500 tokens, 16 kv heads: 33.4 (36.2).  (One row more than requests is an average of 2:
  // with 8 query heads per kv head 31.5 us instead of 24.5.)
  const int64_t rows = a.G * ((req.T + req.B - 1) / req.B);
  const bool wide = rows > 8;
  if (by_chunks(req.T, req.B, H, cache.Hkv)) return launch_kv4_chunk(a, s);
  if (cache.D == 64) return wide ? launch<64, 2>(a, s) : launch<64, 1>(a, s);
  return wide ? launch<128, 2>(a, s) : launch<128, 1>(a, s);
}

}  // namespace qk
