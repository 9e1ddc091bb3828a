// fa_kv_append.cuh -- what fa_kv_append (fa_kv_cache.cu) and fa_kv_append_rope
// (fa_kv_append_rope.cu) share: teams of warps for a page, e4m3 codes, a run's rows into
// its page, and the page's mean.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"
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
    // spill much.  At 10 all forms have 48 registers and spill 68 to 236 bytes, but for D = 64 with
    // pages of 16.  A 16384-token prompt with 8, 9, 10 and 12 blocks, pages of 16, 32, 64, 128:
    //   D = 128  18.2 18.6 18.1 20.3,  18.4 18.7 17.7 20.3,  18.6 18.8 17.4 19.1,  20.3 20.6 20.5 21.5 us;
    //   D = 64   12.3 12.0 12.1 11.7,  12.2 11.9 11.9 11.6,  11.8 11.6 11.6 11.2,  11.9 12.3 12.4 12.6;
    // ragged prompts at 16 rows a page, D = 64, 14.5, 14.3, 13.7 and 14.1.
    static constexpr int BLOCKS = 10 * 128 / THREADS;
};

// What the teams of a block share.
template <int D, int PAGE, class C>
struct AppendShared {
    int slot_of[kWindow + PAGE];   // the window's slots and those that its last run may reach
    uint32_t starts[kWindow / 32];
    uint32_t amax[2][C::WARPS];
    int sums[C::WARPS][D];
};

// A run: its first token in the window, that token's slot, and how many tokens it has.
struct AppendRun {
    int i0, slot, n;
};

// A thread in its team, and what a team does with a run of the window of tokens from t0 on.  (The search for the runs is written out in
// both kernels: as a function of this struct it took fa_kv_append from 9.6 to 10.05 us for 16384 tokens, D = 64, pages of 64.)
template <int D, int PAGE, class C>
struct AppendTeam {
    const AppendParams &p;
    AppendShared<D, PAGE, C> &sm;
    int lane, warp, team, first_warp, tt, t0;

    __device__ __forceinline__ void sync() const {
        if (C::TEAM == 1)
            __syncwarp();
        else if (C::TEAMS == 1 || team == 0)  // by constant numbers: a block that may mean any of the 16
            named_bar_sync(1, C::TEAM * 32);  // barriers has them all, and few fit an SM (24.2 -> 14.3 us)
        else
            named_bar_sync(2, C::TEAM * 32);
    }

    // The largest of the team's magnitudes; a barrier of the team.
    __device__ __forceinline__ uint32_t join_max(uint32_t am) const {
        am = __reduce_max_sync(0xffffffffu, am);
        if (C::TEAM > 1) {
            if (lane == 0) sm.amax[0][warp] = am;
            sync();
#pragma unroll
            for (int v = 0; v < C::TEAM; ++v) am = max(am, sm.amax[0][first_warp + v]);
        } else {
            sync();
        }
        return am;
    }

    // The mean of the first `rows` rows of page and head ph, from the warps' sums in units of 2^-9 (integers: the same in any order).
    __device__ __forceinline__ void write_mean(long long ph, float scale, int rows) const {
        sync();
        constexpr int PER = D > 32 * C::TEAM ? D / (32 * C::TEAM) : 1;  // columns a thread
        int total[PER], a = 0;
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            const int d = tt + c * 32 * C::TEAM;
            total[c] = 0;
            if (d < D)
#pragma unroll
                for (int v = 0; v < C::TEAM; ++v) total[c] += sm.sums[first_warp + v][d];
            a = max(a, abs(total[c]));
        }
        a = (int)__reduce_max_sync(0xffffffffu, (unsigned)a);
        if (C::TEAM > 1) {
            if (lane == 0) sm.amax[1][warp] = (uint32_t)a;
            sync();
#pragma unroll
            for (int v = 0; v < C::TEAM; ++v) a = max(a, (int)sm.amax[1][first_warp + v]);
        }
        const float af = (float)a, inv = a > 0 ? 127.f / af : 0.f;
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            const int d = tt + c * 32 * C::TEAM;
            if (d < D) p.mean[ph * D + d] = (int8_t)__float2int_rn((float)total[c] * inv);
        }
        if (tt == 0) p.mean_scale[ph] = (af * (scale * 0.001953125f)) / (float)(127 * rows);
    }

    // A run of one head, as it is (not rotated), into its page.  W: a whole page, the usual run of a prompt, which does without what
    // the ends of others need and always has a power of two for its scale.  MEANS: whether the call may keep means at all.
    template <bool W, bool MEANS>
    __device__ __forceinline__ void append(const AppendRun &run, int h, bool keys, const __nv_bfloat16 *x_of, long long stride, uint8_t *pages_of, float *scale_of) const {
        const int i0 = run.i0, off = run.slot % PAGE, pg = run.slot / PAGE, n = run.n;
        // ---- everything that is read, at once: row r0 + i ROWS of the page in slot i
        const int sub = tt % C::TPT, r0 = tt / C::TPT;
        const long long ph = (long long)pg * p.Hkv + h;
        const float was = W ? 0.f : scale_of[ph];
        uint8_t *const codes = pages_of + ph * PAGE * D + sub * 8;
        const __nv_bfloat16 *const x = x_of + (long long)(t0 + i0 - off) * stride + sub * 8;  // row 0's token
        const bool mean = MEANS && keys && p.mean != nullptr;
        uint4 w[C::PASSES];
#pragma unroll
        for (int i = 0; i < C::PASSES; ++i) {
            const int r = r0 + i * C::ROWS;
            if (!W) w[i] = make_uint4(0, 0, 0, 0);
            if (W || (r >= off && r < off + n)) {
                w[i] = __ldg(reinterpret_cast<const uint4 *>(x + r * stride));
            } else if (mean && r < off) {
                const uint2 c = *reinterpret_cast<const uint2 *>(codes + r * D);
                w[i].x = c.x, w[i].y = c.y;
            }
        }
        // magnitudes of bf16 compare as integers, two at a time
        uint32_t am2 = 0;
#pragma unroll
        for (int i = 0; i < C::PASSES; ++i) {
            uint32_t u = __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                  __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
            if (!W && r0 + i * C::ROWS < off) u = 0;
            am2 = __vmaxu2(am2, u);
        }
        uint32_t am = max(am2 & 0xffffu, am2 >> 16);
        const bool special = am >= 0x7f80u;
        if (special) {  // infinities and NaN do not count
            am = 0;
#pragma unroll
            for (int i = 0; i < C::PASSES; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t lo = u[c] & 0x7fffu, hi = (u[c] >> 16) & 0x7fffu;
                    if (W || r0 + i * C::ROWS >= off) am = max(am, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
        }
        am = join_max(am);
        float scale = pow2_scale(__uint_as_float(am << 16));
        if (!W && off > 0) scale = fmaxf(scale, was);
        if (tt == 0) scale_of[ph] = scale;  // every thread has read it (the barrier above)
        // x / scale is x * (1 / scale) exactly where the scale is a power of two (always,
        // unless the caller put another one there; the remainder corrects it then)
        const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
        const float inv_scale = 1.f / scale, shrink = was / scale;
        const uint16_t inv_bf16 = (uint16_t)(__float_as_uint(inv_scale) >> 16);  // exact, where it is used
        const bool grown = !W && off > 0 && scale != was;  // the rows before the run are rounded again
        // the codes' sums: multiples of 2^-9, at most 8 of them of at most 448 a thread, are exact in fp32
        static_assert(C::PASSES <= 8, "");
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < C::PASSES; ++i) {
            const int r = r0 + i * C::ROWS;
            if (!W && (r < off || r >= off + n)) continue;
            float y[8];
            if (W || pow2) {
                scaled8(w[i], inv_bf16, y);
            } else {
                bf16x8(w[i], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = y[j];
                    y[j] = x * inv_scale;
                    if (fabsf(x) < INFINITY) y[j] = fmaf(fmaf(-y[j], scale, x), inv_scale, y[j]);
                }
            }
            const uint2 c = encode8(y);
            *reinterpret_cast<uint2 *>(codes + r * D) = c;
            if (mean) {
                add8(special ? without_nan(c) : c, sum);
            }
        }
        if (!W && off > 0 && (mean || grown)) {  // apart, so that prompts' whole pages skip it
#pragma unroll
            for (int i = 0; i < C::PASSES; ++i) {
                const int r = r0 + i * C::ROWS;
                if (r >= off) continue;
                uint2 c = make_uint2(w[i].x, w[i].y);
                float y[8];
                if (grown) {
                    if (!mean) c = *reinterpret_cast<const uint2 *>(codes + r * D);
                    decode8(c, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= shrink;
                    c = encode8(y);
                    *reinterpret_cast<uint2 *>(codes + r * D) = c;
                }
                decode8(without_nan(c), y);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += y[j];
            }
        }
        if (mean) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                int x = (int)(sum[j] * 512.f);
#pragma unroll
                for (int d = C::TPT; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (lane < C::TPT) sm.sums[warp][lane * 8 + j] = x;
            }
            write_mean(ph, scale, W ? PAGE : off + n);
        }
    }
};

}  // namespace fa
