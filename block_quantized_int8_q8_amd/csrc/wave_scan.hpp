// wave_scan.hpp -- scans over the 64 lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>

namespace mmq {

// Inclusive scans of numbers >= 0 over the lanes of a wave, by DPP: shifts
// within the rows of 16 lanes, then each row's last lane to the rows behind.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_0(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int scan_sum(int v) {
    v += dpp_or_0<0x111, 0xf>(v);      // row_shr:1
    v += dpp_or_0<0x112, 0xf>(v);
    v += dpp_or_0<0x114, 0xf>(v);
    v += dpp_or_0<0x118, 0xf>(v);
    v += dpp_or_0<0x142, 0xa>(v);      // row_bcast:15 into rows 1 and 3
    v += dpp_or_0<0x143, 0xc>(v);      // row_bcast:31 into rows 2 and 3
    return v;
}
__device__ __forceinline__ int scan_max(int v) {
    v = max(v, dpp_or_0<0x111, 0xf>(v));
    v = max(v, dpp_or_0<0x112, 0xf>(v));
    v = max(v, dpp_or_0<0x114, 0xf>(v));
    v = max(v, dpp_or_0<0x118, 0xf>(v));
    v = max(v, dpp_or_0<0x142, 0xa>(v));
    v = max(v, dpp_or_0<0x143, 0xc>(v));
    return v;
}
// The lane before's v; `first` in lane 0.
__device__ __forceinline__ int lane_before(int v, int first) {
    return __builtin_amdgcn_update_dpp(first, v, 0x138, 0xf, 0xf, false);      // wave_shr:1
}

}  // namespace mmq
