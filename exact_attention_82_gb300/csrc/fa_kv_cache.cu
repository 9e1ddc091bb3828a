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
#include "fa_kv_append.cuh"
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

// POSITIONS: whether the tokens' positions are written too.
template <bool POSITIONS>
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
        int slot = -1, position = -1;
        if (i < cu[p.B]) {
            const int b = count_le(cu + 1, p.B, i);
            const Request r = plan_request(p, b);
            if (POSITIONS) position = (int)((uint32_t)r.cached + (uint32_t)(i - cu[b]));
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
        if (POSITIONS) p.positions[i] = position;
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
    auto *const kernel = p.positions ? fa_kv_plan_kernel<true> : fa_kv_plan_kernel<false>;
    if (smem > 48 * 1024) {  // beyond what a kernel may have without asking
        // always the most: the limit is the function's, and another thread's call would lower one set to this call's size
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * (kMaxSequences + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, dim3((unsigned)grid), kPlanThreads, smem, stream, 1, p);
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
template <int D, int PAGE>
__global__ void __launch_bounds__(AppendCfg<D, PAGE>::THREADS, AppendCfg<D, PAGE>::BLOCKS) fa_kv_append_kernel(const __grid_constant__ AppendParams p, int share) {
    using C = AppendCfg<D, PAGE>;
    grid_wait();
    __shared__ AppendShared<D, PAGE, C> sm;
    int *const slot_of = sm.slot_of;
    uint32_t *const starts = sm.starts;
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
    const AppendTeam<D, PAGE, C> me{p, sm, lane, warp, team, first_warp, tt, t0};

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
        const int slot = slot_of[i0], off = slot % PAGE;
        int n = 0;  // tokens of the run
#pragma unroll
        for (int w = 0; w < (PAGE + 31) / 32; ++w) {
            const int i = w * 32 + lane;
            const uint32_t m = __ballot_sync(0xffffffffu, i < PAGE - off && slot_of[i0 + min(i, PAGE - 1)] == slot + i);
            if (n == 32 * w) n += m == 0xffffffffu ? 32 : __ffs((int)~m) - 1;
        }

        const AppendRun of{i0, slot, n};
        if (n == PAGE)
            me.template append<true, true>(of, h, kv == 0, x_of, stride, pages_of, scale_of);
        else
            me.template append<false, true>(of, h, kv == 0, x_of, stride, pages_of, scale_of);
        me.sync();  // the next run overwrites the shared words
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
    if (p.rot) return launch_kv_append_rope(D, p, num_sms, stream);
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
