// fa_kv_cache.cu -- what fills the paged 8-bit key/value cache on GB300
// (sm_103a): fa_kv_plan (block tables and slot maps from request lengths) and
// fa_kv_append (rounds a step's keys and values into pages).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_kv_cache = 0;

// -------------------------------------------------------------------- plan
// With held_b = ceil(cached_b / page) and need_b = ceil((cached_b + new_b) / page)
// - held_b, request b is served iff its lengths are valid and need_b = 0 or
// need_0 + .. + need_b <= free.  Every request before a served one that needs
// pages is served too (the sums only grow), so the running sum of the needs is
// also the number of the first page that request b takes.
//
// Bound by latency, not by bytes: a few hundred KB at most move.  So there is
// one launch and no value passes between CTAs: each CTA scans the lengths
// itself (8 bytes a request, from L2) into shared memory and then writes its
// share of the slots and of the new table entries, finding a token's or a page's
// request by bisection of the sums.  What a slot needs of the table (pages held
// before) is never written by this launch, and new pages come from the free list.
// 8 requests 3.0 us, back to back; 256 prompts (115,181 tokens) 4.3 us.
constexpr int kPlanThreads = 256;

struct Request {
    int cached, fresh, held, need;
    bool valid;
};

__device__ __forceinline__ Request plan_request(const PlanParams &p, int b) {
    Request r;
    r.cached = p.cached[b];
    r.fresh = p.fresh[b];
    const long long page = 1ll << p.page_log2, end = (long long)r.cached + r.fresh;
    r.valid = r.cached >= 0 && r.fresh >= 0 && end <= (long long)p.max_pages * page;
    r.cached = max(r.cached, 0);
    r.fresh = max(r.fresh, 0);
    r.held = (int)(((long long)r.cached + page - 1) >> p.page_log2);
    r.need = r.valid ? (int)((end + page - 1) >> p.page_log2) - r.held : 0;
    return r;
}

__device__ __forceinline__ int clamp_int(long long x, int most) { return (int)(x < most ? x : most); }

// Inclusive sum over the block's threads.
__device__ __forceinline__ long long block_scan(long long x, long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += warp_sums[w];
    __syncthreads();
    return x;
}

// How many of a[0 .. n-1] (ascending) are <= x.
__device__ __forceinline__ int count_le(const int *a, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) fa_kv_plan_kernel(const __grid_constant__ PlanParams p) {
    grid_wait();
    extern __shared__ int sm_plan[];
    __shared__ long long warp_sums[kPlanThreads / 32];
    int *cu = sm_plan;              // [B+1] first token of each request, at most T
    int *pc = sm_plan + p.B + 1;    // [B+1] running sums of the needs
    const int tid = threadIdx.x;
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long tokens = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = plan_request(p, b);
        tokens += r.fresh;
        pages += r.need;
    }
    const int free_count = max(0, min(p.free_count[0], p.num_free));
    long long t = block_scan(tokens, warp_sums) - tokens, g = block_scan(pages, warp_sums) - pages;
    for (int b = b0; b < b1; ++b) {
        const Request r = plan_request(p, b);
        cu[b] = clamp_int(t, p.T);
        pc[b] = clamp_int(g, INT_MAX);
        t += r.fresh;
        g += r.need;
        if (blockIdx.x == 0) {
            const bool served = r.valid && (r.need == 0 || g <= free_count);
            p.cu_q[b + 1] = clamp_int(t, p.T);
            p.seq_lens[b] = served ? r.cached + r.fresh : 0;
        }
    }
    if (b1 == p.B && b0 < b1) {  // the thread of the last request
        cu[p.B] = clamp_int(t, p.T);
        pc[p.B] = clamp_int(g, INT_MAX);
    }
    __syncthreads();
    const int step = gridDim.x * kPlanThreads, me = blockIdx.x * kPlanThreads + tid;
    if (me == 0) {
        p.cu_q[0] = 0;
        // pages taken: the largest running sum that the free pages hold
        p.free_left[0] = free_count - pc[count_le(pc, p.B + 1, free_count) - 1];
    }
    const int page = 1 << p.page_log2;
    for (int i = me; i < p.T; i += step) {
        int slot = -1;
        if (i < cu[p.B]) {
            const int b = count_le(cu + 1, p.B, i);
            const Request r = plan_request(p, b);
            if (r.valid && (r.need == 0 || (long long)pc[b] + r.need <= free_count)) {
                const int pos = r.cached + (i - cu[b]), ord = pos >> p.page_log2;
                // (in range, unless the caller changes the lengths during the call)
                const int of = free_count - 1 - (pc[b] + ord - r.held);
                int pg = -1;
                if (ord < r.held && ord < p.max_pages)
                    pg = p.table[(long long)b * p.max_pages + ord];
                else if (of >= 0 && of < free_count)
                    pg = p.free_pages[of];
                if (pg >= 0 && pg < p.num_pages) slot = pg * page + (pos & (page - 1));
            }
        }
        p.slots[i] = slot;
    }
    for (int i = me; i < min(pc[p.B], free_count); i += step) {
        const int b = count_le(pc + 1, p.B, i);
        const Request r = plan_request(p, b);
        if ((long long)pc[b] + r.need <= free_count && r.held + (i - pc[b]) < p.max_pages)
            p.table[(long long)b * p.max_pages + r.held + (i - pc[b])] = p.free_pages[free_count - 1 - i];
    }
}

cudaError_t launch_kv_plan(const PlanParams &p, int num_sms, cudaStream_t stream) {
    const long long entries = (long long)p.B * p.max_pages;
    const long long most = p.T > p.num_free ? p.T : (p.num_free < entries ? p.num_free : entries);
    long long grid = ((most > p.T ? most : p.T) + kPlanThreads - 1) / kPlanThreads;
    if (grid > 4ll * num_sms) grid = 4ll * num_sms;
    const int smem = 2 * (p.B + 1) * (int)sizeof(int);
    if (smem > 48 * 1024) {  // beyond what a kernel may have without asking
        // always the most: the limit is the function's, and another thread's call would lower one set to this call's size
        const cudaError_t e = cudaFuncSetAttribute(fa_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * (kMaxSequences + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    return launch_early(fa_kv_plan_kernel, dim3((unsigned)grid), kPlanThreads, smem, stream, 1, p);
}

// ------------------------------------------------------------------ append
// Bound by HBM: 4 bytes of bf16 read and 2 bytes of codes written for a key and
// a value element.  A team of 1 to 8 warps takes one run (consecutive tokens in one
// page: a whole page of a prompt, or one token of a decode step) of one head, of K or
// of V.  The page's rows are spread over its threads, eight elements each, eight times
// at most, and stay in registers between the pass that takes the largest magnitude and
// the one that writes codes: the run's rows as bf16, and where the page's mean is kept the
// rows before them as codes, so that everything a team reads is asked for at once.
// The size of the team follows from the page's: small pages go to single warps, which
// meet no barrier.
//
// A prompt of 16384 tokens, 8 heads, D = 128: 17.3 us, 5,840 GB/s of reads and writes (87% of
// the copy rate); D = 64 11.6 us; 64 single tokens 4.5 us, three latencies after one
// another.  It issues more than 2.5 instructions a cycle of 4, so what an element costs
// counts: bf16 times the inverse scale and fp16 plus a sum are instructions of mixed
// precision (22.4 -> 21.4 us with both), NaN among the codes is looked for only where the
// row had one (20.9 us), and whole pages have a pass of their own.
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

template <int D, int PAGE>
struct AppendCfg {
    static constexpr int TEAM = PAGE * D < 2048 ? 1 : PAGE * D / 2048;  // warps
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

template <int D, int PAGE>
__global__ void __launch_bounds__(AppendCfg<D, PAGE>::THREADS, AppendCfg<D, PAGE>::BLOCKS) fa_kv_append_kernel(const __grid_constant__ AppendParams p, int share) {
    using C = AppendCfg<D, PAGE>;
    grid_wait();
    __shared__ int slot_of[kWindow + PAGE];   // the window's slots and those that its last run may reach
    __shared__ uint32_t starts[kWindow / 32];
    __shared__ uint32_t amax_sm[2][C::WARPS];
    __shared__ int sums[C::WARPS][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / C::TEAM, first_warp = team * C::TEAM, tt = tid - first_warp * 32;
    const int h = blockIdx.y, kv = blockIdx.z;
    const int win = blockIdx.x / share, part = blockIdx.x % share;
    const int t0 = win * kWindow;
    const int limit = p.num_pages * PAGE;  // fewer than 2^31
    const __nv_bfloat16 *const x_of = static_cast<const __nv_bfloat16 *>(kv ? p.x[1] : p.x[0]) + h * D;
    const long long stride = kv ? p.stride[1] : p.stride[0];
    float *const scale_of = kv ? p.scale[1] : p.scale[0];
    uint8_t *const pages_of = kv ? p.pages[1] : p.pages[0];
    auto team_sync = [&]() {
        if (C::TEAM == 1)
            __syncwarp();
        else if (C::TEAMS == 1 || team == 0)  // by constant numbers: a block that may mean any of the 16
            named_bar_sync(1, C::TEAM * 32);  // barriers has them all, and few fit an SM (24.2 -> 14.3 us)
        else
            named_bar_sync(2, C::TEAM * 32);
    };

    // ---- the runs that begin in the window
    for (int i = tid; i < kWindow + PAGE; i += C::THREADS) slot_of[i] = t0 + i < p.T ? p.slots[t0 + i] : -1;
    int before = -2;
    if (tid == 0 && t0 > 0) before = p.slots[t0 - 1];
    __syncthreads();
    for (int i = warp * 32; i < kWindow; i += C::THREADS) {
        const int s = slot_of[i + lane], prev = i + lane > 0 ? slot_of[i + lane - 1] : before;
        const bool start = s >= 0 && s < limit && (prev != s - 1 || s % PAGE == 0);
        if (s >= limit) atomicExch(&g_status_kv_cache, (int)FA_ERR_BAD_PAGE);
        const uint32_t m = __ballot_sync(0xffffffffu, start);
        if (lane == 0) starts[i / 32] = m;
    }
    __syncthreads();
    // this lane's two tokens, and how many runs begin before each
    const uint32_t s0 = starts[0], s1 = starts[1], lt = (1u << lane) - 1;
    const int rank0 = (s0 >> lane) & 1u ? __popc(s0 & lt) : -1, rank1 = (s1 >> lane) & 1u ? __popc(s0) + __popc(s1 & lt) : -1;
    const int runs = __popc(s0) + __popc(s1);
    for (int run = part * C::TEAMS + team; run < runs; run += share * C::TEAMS) {
        const uint32_t m0 = __ballot_sync(0xffffffffu, rank0 == run), m1 = __ballot_sync(0xffffffffu, rank1 == run);
        const int i0 = m0 ? __ffs((int)m0) - 1 : 31 + __ffs((int)m1);
        const int slot = slot_of[i0], off = slot % PAGE, pg = slot / PAGE;
        int n = 0;  // tokens of the run
#pragma unroll
        for (int w = 0; w < (PAGE + 31) / 32; ++w) {
            const int i = w * 32 + lane;
            const uint32_t m = __ballot_sync(0xffffffffu, i < PAGE - off && slot_of[i0 + min(i, PAGE - 1)] == slot + i);
            if (n == 32 * w) n += m == 0xffffffffu ? 32 : __ffs((int)~m) - 1;
        }

        // A whole page, the usual run of a prompt, does without what the ends of others need
        // (20.9 -> 18.1 us) and always has a power of two for its scale (17.6 us).
        auto append = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
            // ---- everything that is read, at once: row r0 + i ROWS of the page in slot i
            const int sub = tt % C::TPT, r0 = tt / C::TPT;
            const long long ph = (long long)pg * p.Hkv + h;
            const float was = W ? 0.f : scale_of[ph];
            uint8_t *const codes = pages_of + ph * PAGE * D + sub * 8;
            const __nv_bfloat16 *const x = x_of + (long long)(t0 + i0 - off) * stride + sub * 8;  // row 0's token
            const bool mean = kv == 0 && p.mean != nullptr;
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
            am = __reduce_max_sync(0xffffffffu, am);
            if (C::TEAM > 1) {
                if (lane == 0) amax_sm[0][warp] = am;
                team_sync();
#pragma unroll
                for (int v = 0; v < C::TEAM; ++v) am = max(am, amax_sm[0][first_warp + v]);
            } else {
                team_sync();
            }
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
            if (mean) {  // integer sums: the same in any order
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    int x = (int)(sum[j] * 512.f);
#pragma unroll
                    for (int d = C::TPT; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    if (lane < C::TPT) sums[warp][lane * 8 + j] = x;
                }
                team_sync();
                constexpr int PER = D > 32 * C::TEAM ? D / (32 * C::TEAM) : 1;  // columns a thread
                int total[PER], a = 0;
#pragma unroll
                for (int c = 0; c < PER; ++c) {
                    const int d = tt + c * 32 * C::TEAM;
                    total[c] = 0;
                    if (d < D)
#pragma unroll
                        for (int v = 0; v < C::TEAM; ++v) total[c] += sums[first_warp + v][d];
                    a = max(a, abs(total[c]));
                }
                a = (int)__reduce_max_sync(0xffffffffu, (unsigned)a);
                if (C::TEAM > 1) {
                    if (lane == 0) amax_sm[1][warp] = (uint32_t)a;
                    team_sync();
#pragma unroll
                    for (int v = 0; v < C::TEAM; ++v) a = max(a, (int)amax_sm[1][first_warp + v]);
                }
                const float af = (float)a, inv = a > 0 ? 127.f / af : 0.f;
#pragma unroll
                for (int c = 0; c < PER; ++c) {
                    const int d = tt + c * 32 * C::TEAM;
                    if (d < D) p.mean[ph * D + d] = (int8_t)__float2int_rn((float)total[c] * inv);
                }
                if (tt == 0) p.mean_scale[ph] = (af * (scale * 0.001953125f)) / (float)(127 * (W ? PAGE : off + n));
            }
        };
        if (n == PAGE)
            append(std::true_type());
        else
            append(std::false_type());
        team_sync();  // the next run overwrites the shared words
    }
}

template <int D, int PAGE>
static cudaError_t launch_append(const AppendParams &p, int num_sms, cudaStream_t stream) {
    const int windows = (p.T + kWindow - 1) / kWindow;
    // Blocks that share a window's runs: as many as a decode step has (64 of one
    // token each) while there are few windows, one where a prompt fills the chip.
    const long long per = (long long)windows * p.Hkv * 2;
    constexpr int most = kWindow / AppendCfg<D, PAGE>::TEAMS;
    long long share = 32ll * num_sms / per;
    share = share < 1 ? 1 : (share > most ? most : share);
    const dim3 grid((unsigned)(windows * share), p.Hkv, 2);
    return launch_early(fa_kv_append_kernel<D, PAGE>, grid, AppendCfg<D, PAGE>::THREADS, 0, stream, 1, p, (int)share);
}

template <int D>
static cudaError_t launch_append_page(const AppendParams &p, int num_sms, cudaStream_t stream) {
    switch (p.page_log2) {
        case 4: return launch_append<D, 16>(p, num_sms, stream);
        case 5: return launch_append<D, 32>(p, num_sms, stream);
        case 6: return launch_append<D, 64>(p, num_sms, stream);
        default: return launch_append<D, 128>(p, num_sms, stream);
    }
}

cudaError_t launch_kv_append(int D, const AppendParams &p, int num_sms, cudaStream_t stream) {
    return D == 64 ? launch_append_page<64>(p, num_sms, stream) : launch_append_page<128>(p, num_sms, stream);
}

cudaError_t kv_cache_status_read_and_clear(int *out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_kv_cache, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status_kv_cache, &zero, sizeof(int));
    *out = v;
    return e;
}

}  // namespace fa
