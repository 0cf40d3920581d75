// kv4_chunk.cu -- attention of many new tokens per request (chunks of prompts, whole
// prompts) over the 4-bit paged key/value cache, by tcgen05.  The formula, the masks and
// the precision are kv4_attn.cu's; it is for items of up to 128 query rows.
//
// Per block of 64 keys, with groups g of 64 dims and one 128 x 64 product each:
//     S_g = Q_g cK_g^T,     x = sum_g [ sK_g S_g + oK_g sum(q_g) ],    P = 2^(x R - m)
//     O_g += (P sV_g) cV_g,     l += sum P,     off_g += sum P oV_g
//     out = (O_g + off_g) / l
// The codes are operands as they are (whole numbers 0..15 in fp16, exact), the scales are
// applied in fp32 on either side; q is fp16 times a power of two per row (exact but for
// elements 2^-23 below the largest), and P sV is rounded to fp16 with a row reference that
// keeps the largest product below 2^15 (set into [2^5, 2^6)), as in kv4_attn.cu.
//
// Warps of a block (one per SM):
//  * 0-3 unpack a block of keys into K-major fp16 tiles of 128-byte rows (128-byte swizzle).
//    A word's nibbles n and n + 4 come out of one mask (and the fp16 exponents 1024 or 64
//    that an or puts over them out of one subtraction), so a K row holds its dims in the
//    order 0 4 1 5 2 6 3 7 of every 8, and so do the queries; a word of V codes holds two
//    tokens of one dim side by side, which is V^T's row.
//  * 4 issues the products: S_g of one block into the columns of one softmax group while the
//    other group works; P sV is read from tensor memory, over its own scores.
//  * 5 copies the records (bulk copies, four blocks ahead); 6 and 7 idle.
//  * 8-15 are two softmax groups: one takes the even blocks of an item, the other the odd
//    ones, each with sums, references and O of its own, joined at the item's end.  A thread
//    reads scores as 16 x 256 bit fragments: 4 rows of 16 keys, so that a key's scales are
//    read once for four rows, and what it writes back as 16 x 128 bit fragments is the
//    operand's layout.
// Items are cut between blocks like kv4_attn.cu's, in blocks of 64 keys; pieces are joined
// from the workspace, in the order of the keys, by kv4_chunk_join_kernel.  A new item costs a
// block about as much as 8 blocks of keys (queries, a first reference, the join of the two
// groups), and counts for that in the spans: without it a prompt's short first tiles, one
// after the other, took 410 us (2048 rows, 8 kv heads, 4 heads each) instead of 124.
//
// Bound: what the softmax groups issue and wait for.  148 items of 128 rows: 25.2 us over 512
// keys, and 1.2 us for every further 64 (a product of that size is 0.27 us at the tensor
// cores' rate; D = 64: 19.5 and 0.85 us).  Code that runs once an item is as dear as the code of eight
// blocks, mostly its instructions' fetch.  What kv4_attn.cu takes for the same: 47.4 us, and
// 2.6 us for every further 64 keys.
// Registers are short on both sides of the split: a thread spills 592 bytes of stores and 500 of
// loads (D = 64: 380 and 332), partly where the issuing and copying warps walk the items in 48
// registers.  Local memory takes 1.2 % of the instructions of 32 blocks of keys an item.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kv4_chunk.h"
#include "kv4_items.cuh"

namespace qk {
namespace {

constexpr int kRows = 128;             // of an item: lanes of tensor memory
constexpr int kKeys = 64, kLog = 6;    // of a block of keys
// what a new item counts for beside its blocks (5, 8, 12: 147, 131, 134 us for a prompt of 2048 rows, 8 kv
// heads of 4, when a block of keys still took longer)
constexpr int kPad = 8;
constexpr int kThreads = 512, kWarps = kThreads / 32;
// registers a thread: of kRegsLaunch at launch (the build checks it), for the unpacking, the issuing and
// two softmax groups
constexpr int kRegsLaunch = 128;
constexpr int kRegsUnpack = 96, kRegsIssue = 48, kRegsSoft = 184;
static_assert(kRegsUnpack + kRegsIssue + 2 * kRegsSoft <= 4 * kRegsLaunch, "register split");

template <int D>
struct Cfg {
  static constexpr int NG = D / 64;
  static constexpr int STAGES = 3;                            // unpacked blocks
  static constexpr int DEPTH = 4;                             // blocks on their way to be unpacked
  // a record as it was copied, with a pad that spreads the four over the banks
  static constexpr int RAW_REC = Kv4<D>::REC + 32, RAW = 4 * RAW_REC;
  static constexpr int TILE = kKeys * 128;                    // a group's K, or V^T: 64 rows of 128 bytes
  static constexpr int CONST = 2 * (kKeys / 2) * 16 * NG;      // K, V: per pair of keys and group (s, s, o, o)
  static constexpr int Q_SLAB = kRows * 128;
  static constexpr int SM_Q = 0;
  static constexpr int SM_K = SM_Q + NG * Q_SLAB;
  static constexpr int SM_V = SM_K + STAGES * NG * TILE;
  static constexpr int SM_C = SM_V + STAGES * NG * TILE;
  static constexpr int SM_RAW = SM_C + STAGES * CONST;
  static constexpr int SM_END = SM_RAW + DEPTH * RAW;         // per group and row: m, l, sum P oV_g
  static constexpr int SM_ROW = SM_END + 2 * kRows * 16;      // per row: sum(q_g), R, position
  static constexpr int SM_MAX = SM_ROW + kRows * 16;          // per stage and warp: largest V scale
  static constexpr int SM_FLAG = SM_MAX + STAGES * 16;        // per stage and warp, below
  static constexpr int SM_GONE = SM_FLAG + STAGES * 16;       // per block on its way: records without copy
  static constexpr int SM_BAR = SM_GONE + 4 * DEPTH;
  static constexpr int NBAR = 2 * STAGES + 2 * 3 + 1 + 2 * DEPTH;
  static constexpr int SM_SLOT = SM_BAR + NBAR * 8;
  static constexpr int SMEM = SM_SLOT + 16 + 1024;
  static_assert(SM_K % 1024 == 0 && SM_V % 1024 == 0, "swizzled tiles");
  static_assert(SM_RAW % 16 == 0 && SM_END % 16 == 0 && SM_ROW % 16 == 0 && SM_MAX % 16 == 0 && SM_BAR % 8 == 0, "alignment");
  static_assert(SMEM + (int)sizeof(Kv4Scan<kWarps>) + 64 <= 232448, "shared memory");
};

constexpr uint32_t kLast = 256;  // no block on its way: the span ends

// fp16 operands, fp32 sums, both K-major, N = 64, M = 128.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(64 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdesc), "r"(acc)
      : "memory");
}
// A from tensor memory: row = lane, two elements to a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdesc), "r"(acc)
      : "memory");
}

// 16 lanes x 16 columns: lane 4 i + t of the warp gets, per 8 columns, columns 2 t, 2 t + 1
// of row i and then of row i + 8.
__device__ __forceinline__ void ld_frag(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void st_frag(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 lanes x 8 columns of two 16-bit elements: per 4 columns, column t of row i and of row i + 8.
__device__ __forceinline__ void st_half(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], uint32_t at) {
  static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(at));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Two fp32 at once.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1,%2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0,%1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// Over the four lanes of a row.
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

// Codes of nibbles kAt and kAt + 4 of a word (kAt 0..3), two fp16.
template <int kAt>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  // 1024 + c, or 64 + c (the code 4 bits up)
  const uint32_t v = kAt >= 2 ? w >> 8 : w;
  const uint32_t b = kAt & 1 ? ((v & 0x00F000F0u) | 0x54005400u) : ((v & 0x000F000Fu) | 0x64006400u);
  const uint32_t off = kAt & 1 ? 0x54005400u : 0x64006400u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr float kNone = -1.0e30f;   // the reference maximum of a row that has seen nothing

// ---- workspace: the number of blocks with work, a Meta per block, two pieces per block (of
// its first item, where that began in an earlier block, and of its last)
struct Meta {
  int flags;  // 1: a first piece, 2: it ends its item, 4: a last piece, of
  int rt, kvh, row0, n;
  int pad[3];
};
constexpr size_t kMetaOff = 256;
constexpr size_t kPieceOff = kMetaOff + kMaxBlocks * sizeof(Meta);
__host__ __device__ constexpr size_t piece_floats(int D) { return (size_t)kRows * (D + 2); }
__device__ __forceinline__ float* piece_at(uint8_t* ws, int D, int block, int which) {
  return reinterpret_cast<float*>(ws + kPieceOff) + (size_t)(2 * block + which) * piece_floats(D);
}

// Scales and offsets of a pair of keys.  (fp32 in shared memory: as fp16, half the loads and
// two conversions for each of them, a block of 64 keys took a twelfth longer.)
template <int NG>
__device__ __forceinline__ void scales(uint32_t at, uint64_t (&sc)[NG], uint64_t (&of)[NG]) {
#pragma unroll
  for (int gr = 0; gr < NG; ++gr) {
    uint32_t h[4];
    lds(h, at + 16 * gr);
    sc[gr] = two(__uint_as_float(h[0]), __uint_as_float(h[1]));
    of[gr] = two(__uint_as_float(h[2]), __uint_as_float(h[3]));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const Kv4Args a) {
  using C = Cfg<D>;
  using L = Kv4<D>;
  constexpr int NG = C::NG, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  const uint32_t base = smem_u32(smem);
  __shared__ Kv4Scan<kWarps> scan;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int blk = blockIdx.x;
  auto full = [&](int s) { return base + C::SM_BAR + 8u * s; };             // a stage is unpacked
  auto empty = [&](int s) { return base + C::SM_BAR + 8u * (STAGES + s); };  // and read
  auto group_bar = [&](int w, int which) { return base + C::SM_BAR + 8u * (2 * STAGES + 3 * w + which); };
  const uint32_t qfull = base + C::SM_BAR + 8u * (2 * STAGES + 6);
  auto raw_full = [&](int s) { return qfull + 8u + 8u * s; };
  auto raw_empty = [&](int s) { return qfull + 8u + 8u * (C::DEPTH + s); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::SM_SLOT);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 4);
      mbar_init(empty(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(group_bar(w, 0), 1);  // scores are there
      mbar_init(group_bar(w, 1), 4);  // weights are written
      mbar_init(group_bar(w, 2), 1);  // and multiplied
    }
    mbar_init(qfull, 8);
    for (int s = 0; s < C::DEPTH; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 4);
    }
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  const int per = (a.req.B + kThreads - 1) / kThreads;
  scan_units<kRows, kLog, kPad>(a, scan, per, warp);
  const long long W = scan.pre[kThreads];
  // (no less than an item of four blocks of keys to a block: 1 item of 128 rows over 8192
  // keys 52 us with one block of keys each, 32 so)
  const int blocks = (int)min((long long)gridDim.x, W == 0 ? 0 : max(1ll, W / (kPad + 4)));
  if (blk == 0 && threadIdx.x == 0) *reinterpret_cast<int*>(a.ws) = blocks;
  if (blk >= blocks) return;  // the whole block

  // this block's span of W / blocks units (one more for the first W % blocks): from unit k of
  // item `it` up to unit stop_k of an item (stop_b, stop_rt, stop_kvh)
  const long long each = W / blocks;
  const int extra = (int)(W - each * blocks);
  Item it = {};
  int k = 0, stop_b = a.req.B, stop_rt = 0, stop_kvh = 0, stop_k = 0;
  const bool hours = each > 0x7FFFFF00ll;  // of work for one block
  if (hours) record_timeout(a.err);
  if (blk + 1 < blocks) {
    locate_unit<kRows, kLog, kPad>(a, scan, per, each * (blk + 1) + min(blk + 1, extra), it, stop_k);
    stop_b = it.b;
    stop_rt = it.rt;
    stop_kvh = it.kvh;
  }
  if (!locate_unit<kRows, kLog, kPad>(a, scan, per, each * blk + min(blk, extra), it, k) || hours) it.b = a.req.B;
  // Units of the segment that begins at unit k of `it`: 0 behind the span.
  auto segment = [&]() {
    if (it.b >= a.req.B) return 0;
    return (it.b == stop_b && it.rt == stop_rt && it.kvh == stop_kvh ? stop_k : it.cnt) - k;
  };

  if (warp == 4) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;  // scores of group w from column 128 w on, O from 256 + 128 w
  bool ok = true;               // a wait that ran out ends no loop: all that follows just does not wait
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, a.err));
  };

  if (warp < 4) {
    // ------------------------------------------------------------------ unpacking
    regs_dec<kRegsUnpack>();
    const int tid = threadIdx.x;
    // what this thread takes of a block: K: keys, 4 words; V: 8 keys of 4 dims a word
    constexpr int KL = NG;                          // 16-byte loads
    const int krow = NG == 2 ? tid >> 2 : tid >> 1; // + 32 per load (D = 128)
    const int kt = NG == 2 ? tid & 3 : tid & 1;     // 16-byte word of the row
    const int chunk = tid & 7, vg = (tid >> 3) & 7, sub = tid >> 6;  // sub: group (D = 128) or h (64)
    const int skey = NG == 2 ? tid >> 1 : tid & 63, sgrp = NG == 2 ? tid & 1 : 0;
    int place = 0, fresh = 0;  // of the block in the ring of copies, and the ring's phase
#pragma unroll 1
    for (int s = 0, phase = 0; ok;) {
      wait(raw_full(place), fresh);
      uint32_t kw[KL][4], vw[4][NG], sw[2][1];
      const uint32_t gone = *reinterpret_cast<const uint32_t*>(smem + C::SM_GONE + 4 * place);
      if (gone & kLast) break;
      {
        const uint32_t raw = base + C::SM_RAW + place * C::RAW;
#pragma unroll
        for (int i = 0; i < KL; ++i)
          lds(kw[i], raw + ((krow >> 4) + 2 * i) * C::RAW_REC + ((krow & 15) * (2 * NG) + kt) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          lds(vw[j], raw + (chunk >> 1) * C::RAW_REC + L::V_OFF + ((4 * (chunk & 1) + j) * 8 + vg) * 8 * NG + sub * 4 * NG);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          lds(sw[j], raw + (skey >> 4) * C::RAW_REC + L::KS_OFF + j * 16 * NG * 4 + ((skey & 15) * NG + sgrp) * 4);
          // (a record that was not copied: the codes are whatever was there, the scales 0)
          if ((gone >> (skey >> 4)) & 1u) sw[j][0] = 0;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(raw_empty(place));
      if (++place == C::DEPTH) {
        place = 0;
        fresh ^= 1;
      }
      wait(empty(s), phase ^ 1);
      uint8_t* tk = smem + C::SM_K + s * NG * C::TILE;
      uint8_t* tv = smem + C::SM_V + s * NG * C::TILE;
      // K: a word is a chunk of 8 dims of its key's row
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const int row = krow + 32 * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // D = 128: words (group, j) of t = kt; 64: words (t, j) of t = 2 kt, 2 kt + 1
          const int grp = NG == 2 ? j >> 1 : 0, ch = NG == 2 ? 2 * kt + (j & 1) : 4 * kt + j;
          const uint32_t w = kw[i][j];
          *reinterpret_cast<uint4*>(tk + grp * C::TILE + row * 128 + ((ch ^ (row & 7)) << 4)) =
              make_uint4(codes<0>(w), codes<1>(w), codes<2>(w), codes<3>(w));
        }
      }
      // V: nibble i of four words is a chunk of 8 keys of dim 8 g + 4 h + i
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int grp = NG == 2 ? sub : 0, h = NG == 2 ? j : sub;
        uint8_t* row0 = tv + grp * C::TILE + (8 * vg + 4 * h) * 128;
        auto put = [&](auto at) {
          constexpr int i = decltype(at)::value;
          // (dims 8 g + 4 h + i: the row within 8 is 4 h + i)
          *reinterpret_cast<uint4*>(row0 + i * 128 + ((chunk ^ (4 * h + i)) << 4)) =
              make_uint4(codes<i>(vw[0][j]), codes<i>(vw[1][j]), codes<i>(vw[2][j]), codes<i>(vw[3][j]));
        };
        put(std::integral_constant<int, 0>{});
        put(std::integral_constant<int, 1>{});
        put(std::integral_constant<int, 2>{});
        put(std::integral_constant<int, 3>{});
      }
      // scales: [pair of keys][group] (s, s, o, o), K's then V's
      float big = 0.0f;
      bool odd = false;  // a V scale or offset is not finite
      if (NG == 2 || tid < 64) {
        float* c = reinterpret_cast<float*>(smem + C::SM_C + s * C::CONST) + (skey >> 1) * 4 * NG + sgrp * 4 + (skey & 1);
        const float2 ks = unpack_f16(sw[0][0]), vs = unpack_f16(sw[1][0]);
        c[0] = ks.x;
        c[2] = ks.y;
        c[(kKeys / 2) * 4 * NG] = vs.x;
        c[(kKeys / 2) * 4 * NG + 2] = vs.y;
        if (vs.x < INFINITY) big = fmaxf(vs.x, 0.0f);
        odd = !(vs.x < INFINITY && fabsf(vs.y) < INFINITY);
      }
      odd = __any_sync(0xFFFFFFFFu, odd);
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big));
      if (lane == 0) {
        *reinterpret_cast<uint32_t*>(smem + C::SM_MAX + s * 16 + warp * 4) = top;
        *reinterpret_cast<uint32_t*>(smem + C::SM_FLAG + s * 16 + warp * 4) = gone >> 4 | (odd ? 16u : 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(s));
      if (++s == STAGES) {
        s = 0;
        phase ^= 1;
      }
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------------- products
    regs_dec<kRegsIssue>();
    if (warp == 5) {
      // the copies: lanes 0..3 take a record each; a unit's pages are looked up one unit ahead
      int left = segment();  // of the segment
      int id = 0, in = 0, kvh = 0;
      bool want = false;
      auto look = [&]() {
        const int rec = record_of(it, k) * 4 + (lane & 3);
        const int lo = max(it.p0 - a.window + 1, 0);
        want = lane < 4 && it.p1 >= 0 && rec * 16 <= it.p1 &&
               (a.window == 0 || rec * 16 + 15 >= lo || rec * 16 < a.sinks);  // (a row sees some of it)
        kvh = it.kvh;
        if (want) {
          const int page = quot(rec, a.by_page);
          in = rec - page * a.by_page.d;
          id = __ldg(a.req.page_table + (long long)it.b * a.req.max_pages + page);
        }
      };
      int last_s = 0, last_phase = 1;
      if (left > 0) look();
#pragma unroll 1
      for (int s = 0, phase = 1; left > 0;) {
        const bool bad = want && (id < 0 || id >= a.cache.num_pages);
        const bool there = want && !bad;
        const uint8_t* src =
            a.cache.base +
            (((unsigned long long)(uint32_t)id * (uint32_t)a.cache.Hkv + (uint32_t)kvh) * (uint32_t)a.by_page.d +
             (uint32_t)in) * L::REC;
        if (bad) record_index(a.err);
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, there), dead = __ballot_sync(0xFFFFFFFFu, bad);
        ++k;
        if (--left == 0 && k == it.cnt) {
          k = 0;
          next_item<kRows, kLog>(a, it);
          left = segment();
        }
        if (left > 0) look();
        wait(raw_empty(s), phase);
        if (lane == 0) {
          // records without a copy, and those of them that should have been there
          *reinterpret_cast<uint32_t*>(smem + C::SM_GONE + 4 * s) = (~have & 15u) | dead << 4;
          mbar_arrive_expect_tx(raw_full(s), (uint32_t)__popc(have) * L::REC);
        }
        __syncwarp();
        if (there && ok) bulk_load(base + C::SM_RAW + s * C::RAW + lane * C::RAW_REC, src, L::REC, raw_full(s));
        if (++s == C::DEPTH) {
          s = 0;
          phase ^= 1;
        }
        last_s = s;
        last_phase = phase;
      }
      wait(raw_empty(last_s), last_phase);
      if (lane == 0) {
        *reinterpret_cast<uint32_t*>(smem + C::SM_GONE + 4 * last_s) = kLast;
        mbar_arrive(raw_full(last_s));
      }
    }
    if (warp == 4) {
      int seg = 0;
      int ns = 0, np = 0;        // stage and its phase of the next scores
      int vs = 0, vp = 0;        // stage of the next weights, and its phase
      int last = -1, last_phase = 0;
      uint32_t turn[2] = {0, 0}; // blocks of each group whose weights were multiplied
#pragma unroll 1
      for (int n; (n = segment()) > 0;) {
        wait(qfull, seg & 1);
        tc_fence_after();
        auto scores = [&](int i) {
          wait(full(ns), np);
          tc_fence_after();
          if (elected()) {
            const uint32_t q = base + C::SM_Q, kk = base + C::SM_K + ns * NG * C::TILE;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_ss(tmem + 128 * (i & 1) + 64 * g, sw128_kmajor_desc(q + g * C::Q_SLAB + 32 * e),
                       sw128_kmajor_desc(kk + g * C::TILE + 32 * e), e);
            mma_commit(group_bar(i & 1, 0));
          }
          __syncwarp();
          if (++ns == STAGES) {
            ns = 0;
            np ^= 1;
          }
        };
        scores(0);
        if (n > 1) scores(1);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const int w = i & 1;
          wait(group_bar(w, 1), turn[w] & 1);
          ++turn[w];
          tc_fence_after();
          if (elected()) {
            const uint32_t vv = base + C::SM_V + vs * NG * C::TILE;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_ts(tmem + 256 + 128 * w + 64 * g, tmem + 128 * w + 64 * g + 8 * e,
                       sw128_kmajor_desc(vv + g * C::TILE + 32 * e), i > 1 || e > 0);
            mma_commit(group_bar(w, 2));
            mma_commit(empty(vs));
          }
          __syncwarp();
          last = vs;
          last_phase = vp;
          if (++vs == STAGES) {
            vs = 0;
            vp ^= 1;
          }
          if (i + 2 < n) scores(i + 2);
        }
        ++seg;
        if (k + n < it.cnt) break;
        k = 0;
        next_item<kRows, kLog>(a, it);
      }
      if (last >= 0) wait(empty(last), last_phase);  // (no arrival is on its way when the block ends)
    }
  } else {
    // -------------------------------------------------------------------- softmax
    regs_inc<kRegsSoft>();
    const int tid = threadIdx.x - 256, w = tid >> 7, quarter = warp & 3;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t t_s = tmem + ((uint32_t)(32 * quarter) << 16) + 128 * w, t_o = t_s + 256;
    constexpr uint32_t kDown = 16u << 16;  // 16 lanes
    int begin = 0;            // blocks up to the segment
    int turn = 0;             // blocks of this group
    bool first_piece = k > 0;
    Meta meta = {};
    float4* send = reinterpret_cast<float4*>(smem + C::SM_END);
    float4* srow = reinterpret_cast<float4*>(smem + C::SM_ROW);
#pragma unroll 1
    for (int n; (n = segment()) > 0;) {
      const bool ends = k + n == it.cnt;
      // ---- queries: two threads a row
      {
        constexpr int N = 4 * NG;  // chunks of 8 dims
        const int r = tid >> 1, half = tid & 1, row = it.rt * kRows + r, tok = quot(row, a.by_g);
        const bool live = tok < it.n;
        const uint16_t* src = a.q + (long long)(it.row0 + (live ? tok : 0)) * a.q_stride +
                              (long long)(it.kvh * a.G + row - tok * a.G) * D + 8 * N * half;
        uint4 raw[N];
        float top = 0.0f, sum = 0.0f;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          raw[c] = make_uint4(0, 0, 0, 0);
          if (live) raw[c] = *reinterpret_cast<const uint4*>(src + 8 * c);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf_lo(v[i])), fabsf(bf_hi(v[i]))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        // times 2^-e, the largest element comes into [2^13, 2^14)
        const int e = min(max(top == 0.0f ? 0 : exponent(top) - 13, -113), 113);
        const float f = pow2(-e);
        // (in the queries' unit: of rows near the largest bf16 the sum may leave fp32's range)
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += fmaf(bf_lo(v[i]), f, bf_hi(v[i]) * f);
        }
        const float other = __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        uint8_t* dst = smem + C::SM_Q + (NG == 2 ? half * C::Q_SLAB : 0) + r * 128;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const int ch = NG == 2 ? c : 4 * half + c;
          const uint4 v = raw[c];  // dims 0 .. 7 in the order 0 4 1 5 2 6 3 7
          *reinterpret_cast<uint4*>(dst + ((ch ^ (r & 7)) << 4)) =
              make_uint4(pack_f16(bf_lo(v.x) * f, bf_lo(v.z) * f), pack_f16(bf_hi(v.x) * f, bf_hi(v.z) * f),
                         pack_f16(bf_lo(v.y) * f, bf_lo(v.w) * f), pack_f16(bf_hi(v.y) * f, bf_hi(v.w) * f));
        }
        if (half == 0)
          srow[r] = make_float4(NG == 2 ? sum : sum + other, other,
                                // (neither 0 nor infinite: a masked score is -inf, one of 0 stays 0)
                                fminf(fmaxf(a.sc * pow2(e), 1.0e-35f), 3.0e38f),
                                __int_as_float(live ? it.len - it.n + tok : -1));
        fence_proxy_async_smem();
        named_bar_sync(1, 256);
        if (lane == 0) mbar_arrive(qfull);
      }
      // rows 32 quarter + 8 i + g, i = 0..3
      float R[4], nm[4], lim[4], room[4];  // room: 2^8 in the scores' unit
      int pos[4];
      uint64_t qs[4][NG], l2[4], off2[4][NG];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = srow[32 * quarter + 8 * i + g];
        qs[i][0] = two(v.x, v.x);
        if constexpr (NG == 2) qs[i][NG - 1] = two(v.y, v.y);
        R[i] = v.z;
        pos[i] = __float_as_int(v.w);
        nm[i] = -fmaxf(kNone * R[i], kLeast);
        lim[i] = kNone;
        room[i] = 8.0f / R[i];
        l2[i] = two(0.0f, 0.0f);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) off2[i][gr] = two(0.0f, 0.0f);
      }
      bool fresh = true;
      // One block of keys.  `part`: a row may not see all of them; kOdd: and there are V scales
      // or offsets that are not finite among them.
      auto block = [&](auto odd, bool part, int key0, int dead, int s) {
        constexpr bool kOdd = decltype(odd)::value;
        const uint32_t kc = base + C::SM_C + s * C::CONST + t * 16 * NG, vc = kc + (kKeys / 2) * 16 * NG;
        // x[i][2 m], x[i][2 m + 1]: keys 8 m + 2 t, and the one behind it
        float x[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 keys
          uint32_t v[2][NG][8];
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) ld_frag(t_s + d * kDown + 64 * gr + 16 * c, v[d][gr]);
          tmem_ld_wait();
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint64_t sc[NG], of[NG];
            scales(kc + (8 * c + 4 * m) * 16 * NG, sc, of);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint64_t y = mul2(of[0], qs[i][0]);
              if constexpr (NG == 2) y = fma2(of[NG - 1], qs[i][NG - 1], y);
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) {
                const uint32_t* f = &v[i >> 1][gr][4 * m + 2 * (i & 1)];
                y = fma2(two(__uint_as_float(f[0]), __uint_as_float(f[1])), sc[gr], y);
              }
              const float2 z = apart(y);
              x[i][4 * c + 2 * m] = z.x;
              x[i][4 * c + 2 * m + 1] = z.y;
            }
          }
        }
        if (part) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // of the keys key0 + 2 t + in: up to `last`, and behind `before` or in front of `sinks`
            const int at = key0 + 2 * t, last = pos[i] - at;
            const int before = a.window > 0 ? last - a.window : -1, sinks = a.window > 0 ? a.sinks - at : 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int in = 8 * (j >> 1) + (j & 1);
              const bool hidden = (in > last) | ((in <= before) & (in >= sinks));
              x[i][j] = hidden ? -INFINITY : x[i][j];
            }
          }
          if (dead != 0)
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i][j] = (dead >> (j >> 2)) & 1 ? -INFINITY : x[i][j];
        }
        // ---- a row's reference moves where a score passes the last maximum by 2^8, or a
        // product may come to 2^15
        const float4 tops = *reinterpret_cast<const float4*>(smem + C::SM_MAX + s * 16);
        const float heaviest = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
        float most[4];
        bool move = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          most[i] = x[i][0];
#pragma unroll
          for (int j = 1; j < 16; ++j) most[i] = fmaxf(most[i], x[i][j]);
          move |= (most[i] > lim[i]) | (ex2(fmaf(most[i], R[i], nm[i])) * heaviest >= 0x1p15f);
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
          float alpha[4], heavy[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < 4; ++i) most[i] = quad_max(most[i]);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            float s0 = 0.0f, s1 = 0.0f;  // the largest finite scale of a key
            uint64_t sc[NG], of[NG];
            scales(vc + 4 * m * 16 * NG, sc, of);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const float2 v4 = apart(sc[gr]);
              s0 = v4.x < INFINITY ? fmaxf(s0, v4.x) : s0;
              s1 = v4.y < INFINITY ? fmaxf(s1, v4.y) : s1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              heavy[i] = fmaxf(heavy[i], fmaxf(ex2((x[i][2 * m] - most[i]) * R[i]) * s0,
                                               ex2((x[i][2 * m + 1] - most[i]) * R[i]) * s1));
          }
          bool any = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            heavy[i] = quad_max(heavy[i]);
            const float was = nm[i];
            const float set = reference(most[i] * R[i], heavy[i]);
            // (or products of 2^13 and more)
            const bool above = most[i] > lim[i];
            nm[i] = above | ((most[i] > -INFINITY) & (set < was - 8.0f)) ? set : was;
            lim[i] = above ? most[i] + room[i] : lim[i];
            alpha[i] = ex2(nm[i] - was);
            any |= nm[i] != was;
          }
          if (!fresh && __any_sync(0xFFFFFFFFu, any)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t f = two(alpha[i], alpha[i]);
              l2[i] = mul2(l2[i], f);
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) off2[i][gr] = mul2(off2[i][gr], f);
            }
            wait(group_bar(w, 2), (turn - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int e = 0; e < D / 16; ++e) {
              uint32_t o[2][8];
              ld_frag(t_o + 16 * e, o[0]);
              ld_frag(t_o + kDown + 16 * e, o[1]);
              tmem_ld_wait();
#pragma unroll
              for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int m = 0; m < 8; ++m)
                  o[d][m] = __float_as_uint(__uint_as_float(o[d][m]) * alpha[2 * d + ((m >> 1) & 1)]);
              st_frag(t_o + 16 * e, o[0]);
              st_frag(t_o + kDown + 16 * e, o[1]);
            }
          }
        }
        fresh = false;
        // ---- weights, and times scales, over the scores
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[2][NG][4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint64_t sc[NG], of[NG];
            scales(vc + (8 * c + 4 * m) * 16 * NG, sc, of);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 4 * c + 2 * m;
              const float2 arg = apart(fma2(two(x[i][j], x[i][j + 1]), two(R[i], R[i]), two(nm[i], nm[i])));
              const float y0 = ex2(arg.x), y1 = ex2(arg.y);
              const uint64_t y = two(y0, y1);
              l2[i] = add2(l2[i], y);
              if constexpr (kOdd) {  // a key that a row does not see has weight 0 whatever its record holds
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                  const float2 s2 = apart(sc[gr]), o2 = apart(of[gr]);
                  p[i >> 1][gr][2 * m + (i & 1)] = pack_f16(y0 == 0.0f ? 0.0f : y0 * s2.x, y1 == 0.0f ? 0.0f : y1 * s2.y);
                  off2[i][gr] = add2(off2[i][gr], two(y0 == 0.0f ? 0.0f : y0 * o2.x, y1 == 0.0f ? 0.0f : y1 * o2.y));
                }
              } else {
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                  const float2 z = apart(mul2(y, sc[gr]));
                  p[i >> 1][gr][2 * m + (i & 1)] = pack_f16(z.x, z.y);
                  off2[i][gr] = fma2(y, of[gr], off2[i][gr]);
                }
              }
            }
          }
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) st_half(t_s + d * kDown + 64 * gr + 8 * c, p[d][gr]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(group_bar(w, 1));
      };
#pragma unroll 1
      for (int i = w; i < n; i += 2) {
        const int s = (begin + i) % STAGES, u = k + i;
        wait(group_bar(w, 0), turn & 1);
        tc_fence_after();
        // (the scores come behind the stage's unpacking: its scales are there)
        wait(full(s), ((begin + i) / STAGES) & 1);
        const uint4 flag = *reinterpret_cast<const uint4*>(smem + C::SM_FLAG + s * 16);
        const int dead = flag.x & 15;
        const bool part = u < it.whole0 || u >= it.whole1 || dead != 0;
        if (part && ((flag.x | flag.y | flag.z | flag.w) & 16u) != 0)
          block(std::true_type{}, true, record_of(it, u) * kKeys, dead, s);
        else
          block(std::false_type{}, part, record_of(it, u) * kKeys, dead, s);
        ++turn;
      }
      // ---- the segment's sums: each group tells the other its rows' m, l and offsets' part,
      // and joins half of the columns of both O
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = apart(l2[i]), o0 = apart(off2[i][0]), o1 = apart(off2[i][NG - 1]);
        const float l = quad_sum(v.x + v.y), off0 = quad_sum(o0.x + o0.y), off1 = quad_sum(o1.x + o1.y);
        if (t == 0)
          send[w * kRows + 32 * quarter + 8 * i + g] = make_float4(w < n ? -nm[i] : kLeast, l, off0, off1);
      }
      if (w < n) wait(group_bar(w, 2), (turn - 1) & 1);
      tc_fence_before();
      named_bar_sync(1, 256);
      tc_fence_after();
      {
        const bool both = n > 1, whole = ends && !first_piece;
        const int from = w * (D / 2);  // this group's columns
        float f0[4], f1[4], plus[4];
        uint16_t* dst[4];  // the row's place in the output, or null
        float* part = piece_at(a.ws, D, blk, first_piece ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * quarter + 8 * i + g, row = it.rt * kRows + r, tok = quot(row, a.by_g);
          const float4 e0 = send[r], e1 = send[kRows + r];
          const float top = fmaxf(e0.x, e1.x);
          f0[i] = ex2(e0.x - top);
          f1[i] = both ? ex2(e1.x - top) : 0.0f;
          const float sum = fmaf(f1[i], e1.y, f0[i] * e0.y);
          dst[i] = tok < it.n ? a.out + ((long long)(it.row0 + tok) * a.H + it.kvh * a.G + row - tok * a.G) * D : nullptr;
          if (whole) {
            const float inv = sum > 0.0f ? __frcp_rn(sum) : sum;  // (0, or NaN)
            f0[i] *= inv;
            f1[i] *= inv;
          } else if (t == 0 && w == 0) {
            *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(top, sum);
          }
          const bool second = NG == 2 && w == 1;  // (of the groups of 64 dims)
          plus[i] = f0[i] * (second ? e0.w : e0.z);
          if (both) plus[i] = fmaf(f1[i], second ? e1.w : e1.z, plus[i]);
        }
        const uint32_t t_0 = tmem + ((uint32_t)(32 * quarter) << 16) + 256 + from, t_1 = t_0 + 128;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[2][8], o[2][8] = {};
#pragma unroll
          for (int d = 0; d < 2; ++d) ld_frag(t_0 + d * kDown + 16 * c, v[d]);
          if (both) {
#pragma unroll
            for (int d = 0; d < 2; ++d) ld_frag(t_1 + d * kDown + 16 * c, o[d]);
          }
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float z[4];  // columns 2 t, 2 t + 1 of the first 8 and of the second
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 4 * (e >> 1) + 2 * (i & 1) + (e & 1);
              z[e] = fmaf(f0[i], __uint_as_float(v[i >> 1][at]), plus[i]);
              z[e] = fmaf(f1[i], __uint_as_float(o[i >> 1][at]), z[e]);
            }
            if (whole) {
              // (an even lane takes four columns of the first 8, an odd one of the second)
              const uint32_t p0 = pack_bf16(z[0], z[1]), p1 = pack_bf16(z[2], z[3]);
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, t & 1 ? p0 : p1, 1);
              const uint2 y = t & 1 ? make_uint2(got, p1) : make_uint2(p0, got);
              if (dst[i] != nullptr)
                *reinterpret_cast<uint2*>(dst[i] + from + 16 * c + 8 * (t & 1) + 4 * (t >> 1)) = y;
            } else {
              float* at = part + (32 * quarter + 8 * i + g) * D + from + 16 * c + 2 * t;
              *reinterpret_cast<float2*>(at) = make_float2(z[0], z[1]);
              *reinterpret_cast<float2*>(at + 8) = make_float2(z[2], z[3]);
            }
          }
        }
      }
      tc_fence_before();
      if (!(ends && !first_piece)) {
        if (first_piece) {
          meta.flags |= ends ? 3 : 1;
        } else {
          meta.flags |= 4;
          meta.rt = it.rt;
          meta.kvh = it.kvh;
          meta.row0 = it.row0;
          meta.n = it.n;
        }
      }
      first_piece = false;
      begin += n;
      if (!ends) break;
      k = 0;
      next_item<kRows, kLog>(a, it);
    }
    if (tid == 0) reinterpret_cast<Meta*>(a.ws + kMetaOff)[blk] = meta;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, 512);
}

// Joins the items that are cut between blocks: block (c, y) the one whose beginning is
// block c's last piece, a warp to a row (or two, D = 64).
constexpr int kJoinWarps = 8, kJoinParts = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) kv4_chunk_join_kernel(const Kv4Args a) {
  constexpr int LPR = D / 4, RPW = 32 / LPR, AHEAD = 4;
  __shared__ int flags[kMaxBlocks];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = *reinterpret_cast<const int*>(a.ws);
  const Meta* meta = reinterpret_cast<const Meta*>(a.ws + kMetaOff);
  if (c >= blocks) return;
  const Meta me = meta[c];
  if (!(me.flags & 4)) return;
  for (int e = threadIdx.x; e < blocks; e += 32 * kJoinWarps) flags[e] = meta[e].flags;
  __syncthreads();
  int last = blocks - 1;
  for (int e0 = c + 1; e0 < blocks; e0 += 32) {
    const int e = e0 + lane;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, e < blocks && (flags[e] & 2) != 0);
    if (hit != 0) {
      last = e0 + __ffs(hit) - 1;
      break;
    }
  }
  const int n = last - c + 1, d = 4 * (lane % LPR);
  for (int r = (blockIdx.y * kJoinWarps + warp) * RPW + lane / LPR; r < kRows; r += kJoinParts * kJoinWarps * RPW) {
    const int row = me.rt * kRows + r, tok = quot(row, a.by_g);
    if (tok >= me.n) continue;
    float top = kLeast, sum = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
      float4 x[AHEAD];
      float2 ml[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = i0 + j;
        x[j] = make_float4(0, 0, 0, 0);
        ml[j] = make_float2(kLeast, 0.0f);
        if (i < n && (i == 0 || (flags[c + i] & 1) != 0)) {
          const float* p = piece_at(a.ws, D, c + i, i == 0 ? 1 : 0);
          x[j] = *reinterpret_cast<const float4*>(p + r * D + d);
          ml[j] = *reinterpret_cast<const float2*>(p + kRows * D + 2 * r);
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
    const float inv = sum > 0.0f ? __frcp_rn(sum) : sum;
    uint16_t* dst = a.out + ((long long)(me.row0 + tok) * a.H + me.kvh * a.G + row - tok * a.G) * D + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  }
}

template <int D>
cudaError_t launch(const Kv4Args& a, cudaStream_t s) {
  using C = Cfg<D>;
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !done[dev]) {
    e = cudaFuncSetAttribute(kv4_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;  // the register split is of what the block is launched with
    if ((e = cudaFuncGetAttributes(&fa, kv4_chunk_kernel<D>)) != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
    done[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int blocks = num_sms() < kMaxBlocks ? num_sms() : kMaxBlocks;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_chunk_kernel<D>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)blocks, kJoinParts);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_chunk_join_kernel<D>, a);
}

}  // namespace

size_t kv4_chunk_workspace(int64_t D) {
  return kPieceOff + 2 * kMaxBlocks * piece_floats((int)D) * sizeof(float);
}

cudaError_t launch_kv4_chunk(const Kv4Args& a, cudaStream_t s) {
  return a.cache.D == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace qk
