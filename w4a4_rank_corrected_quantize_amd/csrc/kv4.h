// kv4.h -- the 4-bit key / value cache of libsvdq: how a page is laid out.
//
// A cache is `pages` pages of P tokens; a page holds, head by head,
//   k_codes   [P][D / 2] bytes     a token's row: D codes
//   k_scales  [D / g][P]           fp32 (INT4, g = 64) or E8M0 bytes (MXFP4, g = 32)
//   v_codes   [D / 2][P] bytes     a token's column: byte row 16 k + j holds
//                                  channel 32 k + j (low nibble) and
//                                  32 k + 16 + j (high nibble)
//   v_scales  [D / g][P]
// A K row is stored in the order in which the matrix instruction takes it
// (its lanes fall into four parts b = lane / 16; part b reads D / 8
// consecutive bytes of a row, dword s of them for step s):
//   MXFP4  natural order, channel c in byte c / 2, nibble c % 2;
//   INT4   channel c = 64 g + 16 b + 8 s + i lies in byte b D / 8 + 8 g + 4 s
//          + i % 4, nibble i / 4: every step stays within one 64-channel
//          group, whose scale multiplies the step's sums.
// V is stored by channel because its product sums over tokens: a lane then
// reads 16 tokens of two channels as 16 bytes.  One token is one byte column,
// so appending a token writes no byte that another token shares.
#pragma once

#include "svdq_internal.h"
#include "svdq_quant.h"

namespace svdq {

// Dword offset inside a K row of channels c .. c + 7 (c % 8 == 0).
template <bool INT4>
__host__ __device__ __forceinline__ int kv4_k_dword(int c, int D)
{
    if (!INT4) return c >> 3;
    return ((c >> 4) & 3) * (D >> 5) + (c >> 6) * 2 + ((c >> 3) & 1);
}

// The fp32 scale of an E8M0 byte: 2^(e - 127), 2^-127 being subnormal.
__host__ __device__ __forceinline__ float kv4_e8m0(uint32_t e) { return bits_f32(e ? e << 23 : 0x00400000u); }

}  // namespace svdq
