// kv4.cuh -- the 4-bit key/value cache: its layout, and how a request's rows are
// found.  Shared by the kernels that write it (kv4_cache.cu) and read it.
//
// The cache is [num_pages, Hkv, page, D + D / 8] bytes, page a multiple of 16:
// per page and kv head one record for every 16 tokens (18 D bytes),
//   K codes  [row 16][t 4][group NG][j 2] words of 4 bytes, NG = D / 64,
//            nibble i of a word = dim 64 group + 16 t + 8 j + i of token `row`;
//   V codes  [pair 8][g 8][group NG][h 2] words, the low half token 2 pair, the
//            high half token 2 pair + 1, nibble i of a half = dim
//            64 group + 8 g + 4 h + i;
//   K scales [token 16][group NG] fp16 (scale, offset), then V scales alike.
// It is the order in which a warp's mma.m16n8k16 fragments take them: lane
// 4 g + t of the attention reads its K codes (16 D / 128 bytes of token g) and
// its V codes (tokens 2 t, 2 t + 1) with one load each and no lane exchanges
// anything; 16 tokens are one contiguous copy.
#pragma once

#include <cstdint>

#include "qk.h"
#include "qk_internal.h"

namespace qk {

template <int D>
struct Kv4 {
  static constexpr int NG = D / 64;
  static constexpr int K_BYTES = 16 * D / 2;
  static constexpr int V_OFF = K_BYTES;
  static constexpr int KS_OFF = 2 * K_BYTES;
  static constexpr int VS_OFF = KS_OFF + 16 * NG * 4;
  static constexpr int REC = VS_OFF + 16 * NG * 4;
  static_assert(REC == 18 * D && REC % 16 == 0, "record size");
};

// A wrong length, row bound or page id met by a kernel: recorded, and the access skipped.
__device__ __forceinline__ void record_index(int* err) { atomicCAS(err, 0, QK_ERR_INDEX); }

struct Kv4Seq {
  int row0;  // first row of the request's tokens
  int n;     // its rows
  int len;   // tokens in the cache, the rows' own included
};

// Request b's rows and length, held inside the buffers' bounds.  Where they are out of range the
// request is skipped: its length is 0, so that its rows lie in front of the first token.  (With
// the clamped length or number of rows they would be rows of other positions.)
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Req& r, int b, int* err) {
  Kv4Seq s;
  s.len = __ldg(r.kv_lens + b);
  int end;
  if (r.cu != nullptr) {
    s.row0 = __ldg(r.cu + b);
    end = __ldg(r.cu + b + 1);
    s.n = (int)((uint32_t)end - (uint32_t)s.row0);
  } else {
    s.n = r.T / r.B;
    s.row0 = b * s.n;
    end = s.row0 + s.n;
  }
  // (as unsigned numbers, the negative ones are too large)
  if ((uint32_t)s.len > (uint32_t)r.max_len || (uint32_t)s.row0 > (uint32_t)end || (uint32_t)end > (uint32_t)r.T) {
    s.row0 = min(max(s.row0, 0), r.T);
    s.n = max(min(end, r.T) - s.row0, 0);
    s.len = 0;
    record_index(err);
  }
  return s;
}

}  // namespace qk
