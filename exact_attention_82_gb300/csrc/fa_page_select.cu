// fa_page_select.cu -- which pages of the paged 8-bit cache a sequence's
// queries attend to, on GB300 (sm_103a).
//
// For each (sequence, key/value head), with the query rows r of the head's
// group rounded to 8 bits (q8 = rint(q * (127 / max|q|))) and the pages' mean
// keys m (int8, one scale a page):
//   score(page) = max_r (sum_d q8_rd m_d) * (max|q_r| / 127) * mean_scale(page)
// The sum is exact in integers and the two products are rounded the same way
// whatever the order of the work, so equal inputs give equal choices.  The top
// k are found by their bits, eight at a time from the highest, without sorting.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"

namespace fa {

static __device__ int g_status_page_select = 0;

constexpr int kSelThreads = 256;
constexpr int kSelRows = 16;  // query rows scored at a time

// Unsigned numbers in the order of the floats; -0 counts as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) fa_page_select_kernel(const SelectParams p) {
    extern __shared__ uint32_t key[];  // [max_pages] the order of each page's score
    __shared__ __align__(16) int q8[kSelRows][D / 4];
    __shared__ float qs[kSelRows];
    __shared__ int hist[256];
    __shared__ int warp_sums[kSelThreads / 32];
    __shared__ uint32_t pick[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, b = blockIdx.y;
    const int q0 = max(0, min(p.cu_q[b], p.T)), q1 = max(q0, min(p.cu_q[b + 1], p.T));
    const int page = 1 << p.page_log2;
    const long long len = max(0ll, min((long long)p.seq_lens[b], (long long)p.max_pages << p.page_log2));
    const int n = (int)((len + page - 1) >> p.page_log2);
    const int take = q1 > q0 ? min(n, p.top_k) : 0;
    int *sel = p.sel + ((long long)b * p.Hkv + h) * p.top_k;
    if (tid == 0) p.sel_count[(long long)b * p.Hkv + h] = take;
    for (int i = take + tid; i < p.top_k; i += kSelThreads) sel[i] = -1;
    if (n <= p.top_k) {  // every page
        for (int i = tid; i < take; i += kSelThreads) sel[i] = i;
        return;
    }
    if (take == 0) return;

    const int *table = p.table + (long long)b * p.max_pages;
    const int rows = (q1 - q0) * p.G;
    for (int r0 = 0; r0 < rows; r0 += kSelRows) {
        __syncthreads();
        for (int r = warp; r < min(kSelRows, rows - r0); r += kSelThreads / 32) {
            const int t = q0 + (r0 + r) / p.G, g = (r0 + r) % p.G;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (long long)t * p.q_stride +
                                     (long long)(h * p.G + g) * D + lane * (D / 32);
            float x[D / 32], amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                x[i] = __bfloat162float(q[i]);
                if (!(fabsf(x[i]) < INFINITY)) x[i] = 0.f;
                amax = fmaxf(amax, fabsf(x[i]));
            }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            const float inv = amax > 0.f ? 127.f / amax : 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                reinterpret_cast<int8_t *>(q8[r])[lane * (D / 32) + i] = (int8_t)__float2int_rn(x[i] * inv);
            if (lane == 0) qs[r] = amax / 127.f;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kSelThreads) {
            const int pg = table[i];
            uint32_t k = 0;  // a page outside the cache: behind all others
            if (pg >= 0 && pg < p.num_pages) {
                const long long ph = (long long)pg * p.Hkv + h;
                const int4 *m = reinterpret_cast<const int4 *>(p.mean + ph * D);
                int4 w[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c) w[c] = __ldg(m + c);
                const float ms = p.mean_scale[ph];
                for (int r = 0; r < min(kSelRows, rows - r0); ++r) {
                    int dot = 0;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int4 q = *reinterpret_cast<const int4 *>(&q8[r][4 * c]);
                        dot = __dp4a(w[c].x, q.x, dot);
                        dot = __dp4a(w[c].y, q.y, dot);
                        dot = __dp4a(w[c].z, q.z, dot);
                        dot = __dp4a(w[c].w, q.w, dot);
                    }
                    const uint32_t o = order_of(((float)dot * qs[r]) * ms);
                    k = max(k, min(max(o, 1u), 0xfffffffeu));
                }
            } else if (r0 == 0) {
                atomicExch(&g_status_page_select, (int)FA_ERR_BAD_PAGE);
            }
            if (i < p.keep_first || i >= n - p.keep_last) k = 0xffffffffu;
            key[i] = r0 == 0 ? k : max(k, key[i]);
        }
    }
    __syncthreads();

    // the take-th largest key, eight bits at a time from the top
    uint32_t prefix = 0, known = 0;
    int left = take;  // how many of the keys that agree with the prefix are taken
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kSelThreads)
            if ((key[i] & known) == prefix) atomicAdd(&hist[(key[i] >> shift) & 255], 1);
        __syncthreads();
        // sums over the bins from the highest down: thread t has bin 255 - t
        int s = hist[255 - tid];
        const int mine = s;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        for (int w = 0; w < warp; ++w) s += warp_sums[w];
        if (s >= left && s - mine < left) {
            pick[0] = 255 - tid;
            pick[1] = left - (s - mine);
        }
        __syncthreads();
        prefix |= pick[0] << shift;
        known |= 255u << shift;
        left = (int)pick[1];
    }
    // positions in ascending order: all keys above, and the first `left` equal ones
    int above = 0, equal = 0;  // over the rounds before
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < n ? key[i] : 0u;
        const bool gt = i < n && k > prefix, eq = i < n && k == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = __popc(mg) | (__popc(me) << 16);
        __syncthreads();
        int g = above + __popc(mg & ((1u << lane) - 1)), e = equal + __popc(me & ((1u << lane) - 1));
        for (int w = 0; w < kSelThreads / 32; ++w) {
            const int c = warp_sums[w];
            if (w < warp) g += c & 0xffff, e += c >> 16;
            above += c & 0xffff, equal += c >> 16;
        }
        if (gt || (eq && e < left)) sel[g + min(e, left)] = i;
    }
}

cudaError_t launch_page_select(int D, const SelectParams &p, cudaStream_t stream) {
    const int smem = p.max_pages * (int)sizeof(uint32_t);
    const dim3 grid(p.Hkv, p.B);
    const void *f = D == 64 ? (const void *)fa_page_select_kernel<64> : (const void *)fa_page_select_kernel<128>;
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (D == 64)
        fa_page_select_kernel<64><<<grid, kSelThreads, smem, stream>>>(p);
    else
        fa_page_select_kernel<128><<<grid, kSelThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t page_select_status_read_and_clear(int *out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_page_select, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status_page_select, &zero, sizeof(int));
    *out = v;
    return e;
}

}  // namespace fa
