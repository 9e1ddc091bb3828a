// fa_kv_cache.cu -- what fills the paged 8-bit key/value cache on GB300
// (sm_103a): fa_kv_plan (block tables and slot maps from request lengths) and
// fa_kv_append (rounds a step's keys and values into pages).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

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

__global__ void __launch_bounds__(kPlanThreads) fa_kv_plan_kernel(const PlanParams p) {
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
    const cudaError_t e =
        cudaFuncSetAttribute(fa_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    fa_kv_plan_kernel<<<(unsigned)grid, kPlanThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ append
// Bound by HBM: 4 bytes of bf16 read and 2 bytes of codes written for a key and
// a value element.  One CTA takes one run (consecutive tokens in one page: a
// whole page of a prompt, or one token of a decode step) of one head, of K or of
// V: its tokens stay in registers between the pass that takes the largest
// magnitude and the one that writes codes, so that they are read once.  Eight
// elements a thread: 16-byte loads, 8-byte stores.
constexpr int kAppendThreads = 128;
constexpr int kWindow = 64;  // tokens whose runs one set of CTAs shares

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

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), its
// exponent held to [-100, 120]; 1 for amax = 0.  amax is finite.
__device__ __forceinline__ float pow2_scale(float amax) {
    if (!(amax > 0.f)) return 1.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(-100, min(120, e)) + 127) << 23);
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) fa_kv_append_kernel(const AppendParams p, int share) {
    constexpr int TPT = D / 8;                     // threads a token
    constexpr int ROWS = kAppendThreads / TPT;     // tokens a pass
    constexpr int PASSES = 128 / ROWS;             // passes over the largest page
    __shared__ unsigned long long starts;
    __shared__ uint32_t match[kAppendThreads / 32];
    __shared__ uint32_t amax_sm[kAppendThreads / 32];
    __shared__ int sums[D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, kv = blockIdx.z;
    const int win = blockIdx.x / share, part = blockIdx.x % share;
    const int t0 = win * kWindow, page = 1 << p.page_log2;
    const long long limit = (long long)p.num_pages << p.page_log2;
    const __nv_bfloat16 *const x_of = static_cast<const __nv_bfloat16 *>(kv ? p.x[1] : p.x[0]);
    const long long stride = kv ? p.stride[1] : p.stride[0];
    float *const scale_of = kv ? p.scale[1] : p.scale[0];
    uint8_t *const pages_of = kv ? p.pages[1] : p.pages[0];

    // run starts of the window
    {
        bool start = false;
        const int t = t0 + tid;
        if (tid < kWindow && t < p.T) {
            const int s = p.slots[t];
            start = s >= 0 && s < limit && (t == 0 || p.slots[t - 1] != s - 1 || (s & (page - 1)) == 0);
            if (s >= limit) atomicExch(&g_status_kv_cache, (int)FA_ERR_BAD_PAGE);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, start);
        if (lane == 0 && warp < 2) reinterpret_cast<uint32_t *>(&starts)[warp] = m;
        __syncthreads();
    }
    unsigned long long todo = starts;
    for (int ordinal = 0; todo; ++ordinal) {
        const int t = t0 + __ffsll((long long)todo) - 1;
        todo &= todo - 1;
        if (ordinal % share != part) continue;
        const int slot = p.slots[t], off = slot & (page - 1), pg = slot >> p.page_log2;
        const bool same = tid < page - off && t + tid < p.T && p.slots[t + tid] == slot + tid;
        const uint32_t m = __ballot_sync(0xffffffffu, same);
        __syncthreads();  // the shared words of the run before are read
        if (lane == 0) match[warp] = m;
        if (tid < D) sums[tid] = 0;
        __syncthreads();
        int n = 0;  // tokens of the run
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) {
            if (n == 32 * w) n += match[w] == 0xffffffffu ? 32 : __ffs((int)~match[w]) - 1;
        }

        const int sub = tid % TPT, row0 = tid / TPT;
        const __nv_bfloat16 *x = x_of + h * D + sub * 8;
        uint4 w[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (row0 + i * ROWS < n)
                w[i] = __ldg(reinterpret_cast<const uint4 *>(x + (long long)(t + row0 + i * ROWS) * stride));
        }
        // magnitudes of bf16 compare as integers; those of exponent 255 do not count
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t lo = u[c] & 0x7fffu, hi = (u[c] >> 16) & 0x7fffu;
                am = max(am, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
        }
        am = __reduce_max_sync(0xffffffffu, am);
        if (lane == 0) amax_sm[warp] = am;
        const long long ph = (long long)pg * p.Hkv + h;
        const float was = scale_of[ph];
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kAppendThreads / 32; ++v) am = max(am, amax_sm[v]);
        float scale = pow2_scale(__uint_as_float(am << 16));
        if (off > 0) scale = fmaxf(scale, was);
        if (tid == 0) scale_of[ph] = scale;  // every thread has read it (the barrier above)

        uint8_t *codes = pages_of + ((ph << p.page_log2) * D) + sub * 8;
        const bool mean = kv == 0 && p.mean != nullptr;
        int sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        // x / scale is x * (1 / scale) exactly where the scale is a power of two
        // (always, unless the caller put another one there)
        const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
        const float inv_scale = 1.f / scale;
        // the rows before the run, rounded again where the scale has grown
        if (off > 0 && (mean || scale != was)) {
            const float f = was / scale;
            for (int r = row0; r < off; r += ROWS) {
                uint2 c = *reinterpret_cast<const uint2 *>(codes + (long long)r * D);
                float y[8];
                decode8(c, y);
                if (scale != was) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= f;
                    c = encode8(y);
                    *reinterpret_cast<uint2 *>(codes + (long long)r * D) = c;
                    decode8(c, y);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += y[i] == y[i] ? (int)(y[i] * 512.f) : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = row0 + i * ROWS;
            if (r < n) {
                float y[8];
                bf16x8(w[i], y);
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = pow2 ? y[c] * inv_scale : y[c] / scale;
                const uint2 c = encode8(y);
                *reinterpret_cast<uint2 *>(codes + (long long)(off + r) * D) = c;
                if (mean) {
                    decode8(c, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += y[j] == y[j] ? (int)(y[j] * 512.f) : 0;
                }
            }
        }
        if (mean) {  // integer sums: the same in any order
#pragma unroll
            for (int j = 0; j < 8; ++j) atomicAdd(&sums[sub * 8 + j], sum[j]);
            __syncthreads();
            int a = tid < D ? abs(sums[tid]) : 0;
            a = __reduce_max_sync(0xffffffffu, a);
            if (lane == 0) amax_sm[warp] = (uint32_t)a;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kAppendThreads / 32; ++v) a = max(a, (int)amax_sm[v]);
            const float af = (float)a, inv = a > 0 ? 127.f / af : 0.f;
            if (tid < D) p.mean[ph * D + tid] = (int8_t)__float2int_rn((float)sums[tid] * inv);
            if (tid == 0) p.mean_scale[ph] = (af * (scale * 0.001953125f)) / (float)(127 * (off + n));
        }
    }
}

cudaError_t launch_kv_append(int D, const AppendParams &p, int num_sms, cudaStream_t stream) {
    const int windows = (p.T + kWindow - 1) / kWindow;
    // CTAs that share a window's runs: as many as a decode step has (64 of one
    // token each) while there are few windows, one when a prompt fills the chip
    const long long per = (long long)windows * p.Hkv * 2;
    int share = (int)((32ll * num_sms + per - 1) / per);
    share = share < 1 ? 1 : (share > kWindow ? kWindow : share);
    const dim3 grid((unsigned)(windows * share), p.Hkv, 2);
    if (D == 64)
        fa_kv_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(p, share);
    else
        fa_kv_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(p, share);
    return cudaGetLastError();
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
