// kv4.h -- the 4-bit key / value cache of libsvdq: how a page is laid out.
//
// A cache is `pages` pages of P tokens.  Per page and head the tokens form
// runs of 16, the rows of one product of the matrix cores; D = channels per
// head, g = 64 (INT4) / 32 (MXFP4):
//   k_codes   [P / 16][4][16][D / 8] bytes: run, part b, token, bytes
//   v_codes   [P / 16][4][16][D / 32][4] bytes: run, part b, j, block k,
//             token 4 b + i of the run: channel 32 k + j in the low, 32 k + 16
//             + j in the high nibble
//   scales    [P / 16][D / g][16]: fp32 (INT4) or E8M0 bytes (MXFP4)
// Both kinds of codes are stored in the order in which a wave's lanes (part b
// = lane / 16, j = lane % 16) take them, so that a run is one load of
// consecutive 16 (D = 64: 8) bytes per lane:
//   K: lane (b, token) has part b of the token's channels, dword s for product
//      step s.  MXFP4: channels D / 4 b + .., channel c in byte c / 2, nibble c
//      % 2.  INT4: dword 2 G + s holds channels 64 G + 16 b + 8 s + i, i < 8,
//      in byte i % 4, nibble i / 4: every step stays within one 64-channel
//      group, whose scale multiplies the step's sums.
//   V: lane (b, j) has tokens 4 b .. 4 b + 3 of channels 32 k + j and 32 k + 16
//      + j for every k: the sums over tokens need no transposition.
// One token's bytes are its own, so appending it touches no other token.
#pragma once

#include "svdq_internal.h"
#include "svdq_quant.h"

namespace svdq {

// Byte offset, inside a run, of the dword of K channels c .. c + 7 (c % 8 ==
// 0) of token r.
template <bool INT4>
__host__ __device__ __forceinline__ int kv4_k_offset(int r, int c, int D)
{
    const int b = INT4 ? (c >> 4) & 3 : c / (D / 4);
    const int dw = INT4 ? 2 * (c >> 6) + ((c >> 3) & 1) : (c % (D / 4)) >> 3;
    return (16 * b + r) * (D / 8) + 4 * dw;
}

// Byte offset, inside a run, of V channels 32 k + j and 32 k + 16 + j of token
// r.
__host__ __device__ __forceinline__ int kv4_v_offset(int r, int k, int j, int D)
{
    return (16 * (r >> 2) + j) * (D / 8) + 4 * k + (r & 3);
}

// The fp32 scale of an E8M0 byte: 2^(e - 127), 2^-127 being subnormal.
__host__ __device__ __forceinline__ float kv4_e8m0(uint32_t e) { return bits_f32(e ? e << 23 : 0x00400000u); }

}  // namespace svdq
