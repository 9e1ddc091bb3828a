// fa_kv_append.cuh -- what fa_kv_append (fa_kv_cache.cu) and fa_kv_append_rope
// (fa_kv_append_rope.cu) share: teams of warps for a page, and e4m3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

namespace fa {

constexpr int kWindow = 64;  // tokens whose runs one set of blocks shares

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

__device__ __forceinline__ void decode8(const uint2 w, float (&f)[8]) {
    const float2 a = e4m3x2_to_float2(w.x & 0xffffu), b = e4m3x2_to_float2(w.x >> 16);
    const float2 c = e4m3x2_to_float2(w.y & 0xffffu), d = e4m3x2_to_float2(w.y >> 16);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
}

// f += the values of eight codes
__device__ __forceinline__ void add8(const uint2 w, float (&f)[8]) {
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(u[i / 2] >> 16 * (i & 1))));
        asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; add.rn.f32.f16 %0, lo, %0; add.rn.f32.f16 %1, hi, %1;}"
            : "+f"(f[2 * i]), "+f"(f[2 * i + 1])
            : "r"(h));
    }
}

// NaN codes (0x7f and 0xff) as 0
__device__ __forceinline__ uint32_t without_nan(uint32_t c) {
    const uint32_t nan = ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return nan ? c & ~((nan >> 7) * 0xffu) : c;
}
__device__ __forceinline__ uint2 without_nan(uint2 c) { return make_uint2(without_nan(c.x), without_nan(c.y)); }

__device__ __forceinline__ uint2 encode8(const float (&f)[8]) {
    return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

__device__ __forceinline__ void bf16x8(const uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// eight bf16 numbers times another one, in fp32
__device__ __forceinline__ void scaled8(const uint4 w, uint16_t by, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; fma.rn.f32.bf16 %0, lo, %3, %4; fma.rn.f32.bf16 %1, hi, %3, %4;}"
            : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
            : "r"(u[i]), "h"(by), "f"(-0.f));
    }
}

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), its
// exponent held to [-100, 120]; 1 for amax = 0.  amax is finite.
__device__ __forceinline__ float pow2_scale(float amax) {
    if (!(amax > 0.f)) return 1.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(-100, min(120, e)) + 127) << 23);
}

// PER: elements a thread holds at most
template <int D, int PAGE, int PER = 64>
struct AppendCfg {
    static constexpr int TEAM = PAGE * D < 32 * PER ? 1 : PAGE * D / (32 * PER);  // warps
    static constexpr int WARPS = TEAM > 4 ? TEAM : 4;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int TEAMS = WARPS / TEAM;
    static_assert(TEAM == 1 || TEAMS <= 2, "");
    static constexpr int TPT = D / 8;                                 // threads a token
    static constexpr int ROWS = 32 * TEAM / TPT;                      // tokens a pass
    static constexpr int PASSES = PAGE / ROWS;
    // Blocks an SM that the registers are held to.  A team waits for memory three times
    // (slots, rows, and to be written), so more of them side by side is faster, until they
    // spill much.  At 10 all forms have 48 registers and spill 140 to 244 bytes, but for D = 64 with
    // pages of 16.  A 16384-token prompt with 8, 9, 10 and 12 blocks, pages of 16, 32, 64, 128:
    //   D = 128  18.2 18.6 18.1 20.3,  18.4 18.7 17.7 20.3,  18.6 18.8 17.4 19.1,  20.3 20.6 20.5 21.5 us;
    //   D = 64   12.3 12.0 12.1 11.7,  12.2 11.9 11.9 11.6,  11.8 11.6 11.6 11.2,  11.9 12.3 12.4 12.6;
    // ragged prompts at 16 rows a page, D = 64, 14.5, 14.3, 13.7 and 14.1.
    static constexpr int BLOCKS = 10 * 128 / THREADS;
};

}  // namespace fa
