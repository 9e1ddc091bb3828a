// fa_rope.cuh -- rotary positions: angles, and the rotation of 16 elements of a head
// by one thread.  Used by fa_rope (fa_rope.cu) and fa_kv_append_rope (fa_kv_append_rope.cu).
//
// A pair's frequency is a whole number of 2^-64 turns a position (its phase), so the
// angle at a position is the low 64 bits of position * phase: whole turns drop out of an
// integer product exactly, however far the position, where fp32 (and at 10^6 positions
// even the frequency alone in fp32) would lose the angle's leading digits.  Of its upper
// 32 bits the quarter turn that is nearest is taken off, in integers too; what remains, at most
// an eighth of a turn, goes to fp32 (rounded by 2^-27 of a turn), and its sine and cosine are
// Taylor sums: behind the terms that are kept (to r^9 and r^8, r in turns) the next are
// (pi/4)^11 / 11! = 2e-9 and (pi/4)^10 / 10! = 2.5e-8.  The quarter turns swap the two and set their signs.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

namespace fa {

// amplitude * cos and sin of the angle of `phase` at `position`
__device__ __forceinline__ float2 rope_factor(unsigned long long phase, int position, float amplitude) {
    // bits 32-63 of phase * position (a negative position counts 2^32 too many, so phase's lower half comes off)
    const uint32_t lo = (uint32_t)phase, hi = (uint32_t)(phase >> 32);
    const uint32_t turns = __umulhi(lo, (uint32_t)position) + hi * (uint32_t)position - (position < 0 ? lo : 0u);
    const uint32_t quarter = (turns + 0x20000000u) >> 30;
    const float r = (float)(int)(turns - (quarter << 30)) * 0x1p-32f, u = r * r;
    const float s = r * fmaf(u, fmaf(u, fmaf(u, fmaf(u, 42.05869394f, -76.70585975f), 81.60524928f), -41.34170224f), 6.283185307f);
    const float c = fmaf(u, fmaf(u, fmaf(u, fmaf(u, 60.24464137f, -85.45681721f), 64.93939402f), -19.7392088f), 1.f);
    const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;  // cos and sin of r + quarter, but for their signs
    const uint32_t flip_x = (quarter + 1u) << 30 & 0x80000000u, flip_y = quarter << 30 & 0x80000000u;
    return make_float2(__uint_as_float(__float_as_uint(x) ^ flip_x) * amplitude, __uint_as_float(__float_as_uint(y) ^ flip_y) * amplitude);
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
