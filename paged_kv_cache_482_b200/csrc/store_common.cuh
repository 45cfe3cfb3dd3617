// store_common.cuh -- helpers shared by the kernels that write cache rows:
// the largest magnitude of a row's chunk, the per-token scale, the E4M3
// quantisation, and the shuffles between interleaved and split rotary pairs.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// Largest |x| of 8 bf16 elements.
__device__ __forceinline__ float amax8(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(bf16lo(w[j])), fabsf(bf16hi(w[j]))));
    return m;
}

// Per-token scale: the row's largest magnitude / 448 (one IEEE division), at
// least the smallest normal binary32 so that an all-zero row encodes as zeros.
__device__ __forceinline__ float token_scale(float amax) { return fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f); }

__device__ __forceinline__ uint2 quantise8(uint4 x, float scale) {
    // E4M3 of x / scale for 8 bf16 elements: one IEEE fp32 division each, then
    // round-to-nearest-even with saturation to +-448 (CUDA's conversion).
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = __fdiv_rn(bf16lo(w[j]), scale);
        const float b = __fdiv_rn(bf16hi(w[j]), scale);
        const uint32_t ca = __nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t cb = __nv_cvt_float_to_fp8(b, __NV_SATFINITE, __NV_E4M3);
        out[j >> 1] |= (ca | (cb << 8)) << ((j & 1) * 16);
    }
    return make_uint2(out[0], out[1]);
}

// Interleaved pairs: 16 consecutive elements (two 16-byte chunks a, b) ->
// the 8 first elements of the pairs (x) and the 8 second ones (y), and back.
__device__ __forceinline__ void deinterleave(const uint4 &a, const uint4 &b, uint4 &x, uint4 &y) {
    x = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410), __byte_perm(b.x, b.y, 0x5410),
                   __byte_perm(b.z, b.w, 0x5410));
    y = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632), __byte_perm(b.x, b.y, 0x7632),
                   __byte_perm(b.z, b.w, 0x7632));
}
__device__ __forceinline__ void interleave(const uint4 &x, const uint4 &y, uint4 &a, uint4 &b) {
    a = make_uint4(__byte_perm(x.x, y.x, 0x5410), __byte_perm(x.x, y.x, 0x7632), __byte_perm(x.y, y.y, 0x5410),
                   __byte_perm(x.y, y.y, 0x7632));
    b = make_uint4(__byte_perm(x.z, y.z, 0x5410), __byte_perm(x.z, y.z, 0x7632), __byte_perm(x.w, y.w, 0x5410),
                   __byte_perm(x.w, y.w, 0x7632));
}

}  // namespace pkv
