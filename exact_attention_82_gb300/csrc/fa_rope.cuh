// fa_rope.cuh -- rotary positions: angles, and the rotation of 16 elements of a head
// by one thread.  Used by fa_rope (fa_rope.cu) and fa_kv_append_rope (fa_kv_append_rope.cu).
//
// A pair's frequency is a whole number of 2^-64 turns a position (its phase), so the
// angle at a position is the low 64 bits of position * phase: whole turns drop out of an
// integer product exactly, however far the position, where fp32 (and at 10^6 positions
// even the frequency alone in fp32) would lose the angle's leading digits.  The upper
// 32 bits, a signed number of 2^-31 half turns, then go to fp32: the angle is off by
// at most 2^-25 half turns, 10^-7 radians.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

namespace fa {

// amplitude * cos and sin of the angle of `phase` at `position`
__device__ __forceinline__ float2 rope_factor(unsigned long long phase, int position, float amplitude) {
    const unsigned long long turns = phase * (unsigned long long)(long long)position;
    float s, c;
    sincospif((float)(int)(uint32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

// (a, b) rotated: a c - b s, a s + b c
__device__ __forceinline__ void rope_turn(float &a, float &b, const float2 f) {
    const float x = fmaf(a, f.x, -(b * f.y)), y = fmaf(a, f.y, b * f.x);
    a = x, b = y;
}

// The two 8-element pieces of a head that thread `sub` of D / 16 holds.  Half layout: a piece
// and its partner rot / 2 behind; neighbouring pairs, and behind the rotated part: two
// pieces in a row.  Either way its pairs are the eight 8 sub .. 8 sub + 7.
__device__ __forceinline__ int2 rope_pieces(int sub, int rot, bool interleaved) {
    const bool half = !interleaved && sub < rot / 16;
    return half ? make_int2(sub, sub + rot / 16) : make_int2(2 * sub, 2 * sub + 1);
}

__device__ __forceinline__ void bf16x8_to_float(const uint4 w, float *f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 float_to_bf16x8(const float *f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The 16 elements of two pieces, x[0 .. 7] and x[8 .. 15], rotated by eight factors.
template <bool INTER>
__device__ __forceinline__ void rope_turn16(float (&x)[16], const float2 (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (INTER)
            rope_turn(x[2 * j], x[2 * j + 1], f[j]);
        else
            rope_turn(x[j], x[j + 8], f[j]);
    }
}

}  // namespace fa
