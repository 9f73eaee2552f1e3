// i8_codes.hpp -- the int8 row code shared by the quantizers: a row's scale
// is amax / 127 and its codes are the values over it, rounded half away from
// zero.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmq {

// What a row's largest magnitude (as integer bits: NaN > infinity > any
// finite) says of its codes.
struct RowCode {
    bool finite;
    float d, id;              // scale, and its reciprocal (0 where codes are 0)
    __device__ __forceinline__ explicit RowCode(uint32_t am) {
        finite = am < 0x7f800000u;
        d = __uint_as_float(am) / 127.0f;                                // correctly rounded
        id = (finite && d != 0.0f) ? 1.0f / d : 0.0f;
        if (__builtin_isinf(id)) id = 0.0f;
    }
    __device__ __forceinline__ float scale() const { return finite ? d : __uint_as_float(0x7fc00000u); }
};

// Codes of eight values, a byte each.  |v * id| <= 127 (1 + 2^-21), so the
// rounded code needs no clamp.
__device__ __forceinline__ uint2 encode8(const float (&w)[8], const RowCode &c) {
    uint32_t pk[2];
#pragma unroll
    for (int g = 0; g < 2; g++) {
        int k[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            // half away from zero: adding the number below 1/2 carries exactly the halves and what is above them
            const float y = w[4 * g + i] * c.id;
            k[i] = c.finite ? int(y + __builtin_copysignf(0x1.fffffep-2f, y)) : 0;
        }
        const uint32_t lo = __builtin_amdgcn_perm(k[1], k[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(k[3], k[2], 0x0c0c0400u);
        pk[g] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    return make_uint2(pk[0], pk[1]);
}

}  // namespace mmq
