// Rows in MXFP4 (OCP Microscaling Formats 1.0): e2m1 codes, the even channel in
// a byte's low half, and for every 32 channels an exponent byte e; a value is
// code * 2^(e - 127), and all values of a block with e = 255 are NaN (here with
// any e past 252, under which the largest code would pass bf16's range).  Every
// other value is a bf16 number, so that reading rounds nothing.
#pragma once

#include "gdn_device.h"

namespace gdn {

constexpr int kMxBlock = 32;             // channels of an exponent
constexpr int kMxLeast = 25, kMxMost = 252, kMxNan = 255;    // exponent bytes that are written

__device__ __forceinline__ float mx_scale(uint32_t e) { return e > kMxMost ? NAN : __uint_as_float(e << 23); }

// Byte B (0..3) of 8 codes: two channels in bf16.
template <int B>
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, B));
}
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale, int b)      // b known when compiled
{
    return b == 0 ? mx_pair<0>(codes, scale) : b == 1 ? mx_pair<1>(codes, scale) : b == 2 ? mx_pair<2>(codes, scale) : mx_pair<3>(codes, scale);
}
// 8 codes: 8 channels
__device__ __forceinline__ uint4 mx_values8(uint32_t codes, float scale)
{
    return make_uint4(mx_pair<0>(codes, scale), mx_pair<1>(codes, scale), mx_pair<2>(codes, scale), mx_pair<3>(codes, scale));
}

}  // namespace gdn
