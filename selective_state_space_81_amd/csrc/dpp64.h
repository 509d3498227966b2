// dpp64.h -- sums of fp64 values over a wave with DPP moves, a few cycles each
// where a shuffle is a trip through LDS.  Included only by .hip files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msscan {
namespace dev {

// Sums over the lanes up to each; lane 63 has the whole wave's.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double x) {  // 0 where no lane gives anything
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double scan64(double x) {
    x += dpp64<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: within 16 lanes
    x += dpp64<0x112, 0xf>(x);
    x += dpp64<0x114, 0xf>(x);
    x += dpp64<0x118, 0xf>(x);
    x += dpp64<0x142, 0xa>(x);  // lane 15 of a row to the next one, lane 31 to the upper half
    x += dpp64<0x143, 0xc>(x);
    return x;
}
// The same from lane `first` (of each lane's own run of neighbours, or below 0) on.
__device__ __forceinline__ double scan64_from(double x, int first) {
    const int i = threadIdx.x & 63;
    double y;
    y = dpp64<0x111, 0xf>(x), x += i - 1 >= first ? y : 0.0;
    y = dpp64<0x112, 0xf>(x), x += i - 2 >= first ? y : 0.0;
    y = dpp64<0x114, 0xf>(x), x += i - 4 >= first ? y : 0.0;
    y = dpp64<0x118, 0xf>(x), x += i - 8 >= first ? y : 0.0;
    y = dpp64<0x142, 0xa>(x), x += (i & 48) - 1 >= first ? y : 0.0;
    y = dpp64<0x143, 0xc>(x), x += 31 >= first ? y : 0.0;
    return x;
}
__device__ __forceinline__ double lane64(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

}  // namespace dev
}  // namespace msscan
