// pa_rope.cuh -- the angle of a rotary pair at a position, shared by the kernels
// that rotate (pa_rope.cu, pa_write8.cu).
#pragma once

#include <cstdint>

#include "pa_device.cuh"

namespace pa {

// freq / 2 pi mod 1 in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
    const double t = freq * 0.15915494309189535;  // 1 / (2 pi)
    return (unsigned long long)((t - floor(t)) * 0x1p64);  // the conversion saturates at 2^64 - 1
}

// (cos, sin) of pos steps of that fraction, times mscale.
__device__ __forceinline__ float2 turn_at(unsigned long long fraction, int pos, float mscale) {
    const int t = (int)((fraction * (unsigned long long)(long long)pos) >> 32);  // turns mod 1, signed, in 2^-32
    float s, c;
    sincospif((float)t * 0x1p-31f, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

// The pair (a, b) turned by c.  Which product of a sum is rounded is written out, as a compiler may choose either: a
// layout's bits then do not depend on which kernel takes it, nor on the cache that the keys go to.
__device__ __forceinline__ float2 turned(float a, float b, float2 c) {
    const float y = fmaf(a, c.y, __fmul_rn(b, c.x));   // first: in this order the 8-bit write spills less (8192 tokens 39.4 us, 40.6)
    return make_float2(fmaf(a, c.x, -__fmul_rn(b, c.y)), y);
}

// The position by which pair p of token t turns: that of its axis, or 0 (flagged) if the axis is none of the call's.
template <typename Args>
__device__ __forceinline__ int pair_position(const Args &a, int t, int p) {
    if (!a.pair_axis) return a.positions[t];
    const int axis = a.pair_axis[p];
    if ((unsigned)axis >= (unsigned)a.num_axes) {
        set_error(a.err, PA_DEVERR_BAD_AXIS);
        return 0;
    }
    return a.positions[(size_t)axis * a.T + t];
}

}  // namespace pa
