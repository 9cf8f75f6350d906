// 16-byte loads and stores of what passes through once: nothing of it is kept
// in the XCD's cache for longer than it has to be.
#pragma once

#include "gdn_device.h"

namespace gdn {

__device__ __forceinline__ uint4 load_once(const void *p)
{
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(static_cast<const f4v *>(p)));
}
__device__ __forceinline__ void store_once(void *p, uint4 x)
{
    __builtin_nontemporal_store(__builtin_bit_cast(f4v, x), static_cast<f4v *>(p));
}

}  // namespace gdn
