// fa_page_select.cu -- which pages of the paged 8-bit cache a sequence's
// queries attend to, on GB300 (sm_103a).
//
// For each (sequence, key/value head), with the query rows r of the head's
// group rounded to 8 bits (q8 = rint(q * (127 / max|q|))) and the pages' mean
// keys m (int8, one scale a page):
//   score(page) = max_r (sum_d q8_rd m_d) * (max|q_r| / 127) * mean_scale(page)
// The sum is exact in integers and the two products are rounded the same way
// whatever the order of the work, so equal inputs give equal choices.
//
// Bound by latency: a page's mean key is 68 or 132 bytes, so even 131072 tokens have
// some MB to read, and the answer is a few hundred numbers.  So it is one launch: a
// cluster of 1 to 8 blocks takes one (sequence, head), each block scores its share of
// the pages (a page a thread, its mean key in registers, the 8-bit queries read from
// shared memory by all threads at once, four products an instruction) and writes the
// scores' bits into the first block's shared memory, which finds the k-th largest by its
// bits, eight at a time from the highest, without sorting.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"

namespace fa {

static __device__ int g_status_page_select = 0;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelRows = 16;   // query rows scored at a time
constexpr int kSelShare = 256; // pages of the table that make another block of the cluster worth its while

// Unsigned numbers in the order of the floats; -0 counts as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of `p` in the cluster's first block
__device__ __forceinline__ uint32_t in_first_block(const void *p) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return a;
}
__device__ __forceinline__ void store_cluster(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) fa_page_select_kernel(const __grid_constant__ SelectParams p) {
    grid_wait();
    extern __shared__ uint32_t key[];  // [max_pages] the order of each page's score, in the first block
    __shared__ __align__(16) int q8[kSelRows][D / 4];
    __shared__ float qs[kSelRows];
    __shared__ int hist[256];
    __shared__ int warp_sums[kSelWarps];
    __shared__ uint32_t pick[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int h = blockIdx.y, b = blockIdx.z;
    const int q0 = max(0, min(p.cu_q[b], p.T)), q1 = max(q0, min(p.cu_q[b + 1], p.T));
    const int page = 1 << p.page_log2;
    const long long len = max(0ll, min((long long)p.seq_lens[b], (long long)p.max_pages << p.page_log2));
    const int n = (int)((len + page - 1) >> p.page_log2);
    const int take = q1 > q0 ? min(n, p.top_k) : 0;
    const long long bh = (long long)b * p.Hkv + h;
    int *const sel = p.sel + bh * p.top_k;
    if (rank == 0) {
        if (tid == 0) p.sel_count[bh] = take;
        for (int i = take + tid; i < p.top_k; i += kSelThreads) sel[i] = -1;
    }
    if (n <= p.top_k || take == 0) {  // every page, or none; the same in all blocks of the cluster
        if (rank == 0)
            for (int i = tid; i < take; i += kSelThreads) sel[i] = i;
        return;
    }
    if (size > 1) cluster_sync();  // the first block's shared memory is there

    const int *const table = p.table + (long long)b * p.max_pages;
    const int rows = (q1 - q0) * p.G;
    const int chunk = (n + (int)size - 1) / (int)size, begin = min(n, (int)rank * chunk), end = min(n, begin + chunk);
    for (int r0 = 0; r0 < rows; r0 += kSelRows) {
        if (r0 > 0) __syncthreads();
        const int some = min(kSelRows, rows - r0);
        for (int r = warp; r < some; r += kSelWarps) {
            const int t = q0 + (r0 + r) / p.G, g = (r0 + r) % p.G;
            const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(
                static_cast<const __nv_bfloat16 *>(p.q) + (long long)t * p.q_stride + (long long)(h * p.G + g) * D);
            float x[D / 32], amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float2 f = __bfloat1622float2(q[lane * (D / 64) + i]);
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
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
        for (int i = begin + tid; i < end; i += kSelThreads) {
            const int pg = table[i];
            uint32_t k = 0;  // a page outside the cache: behind all others
            if (pg >= 0 && pg < p.num_pages) {
                const long long ph = (long long)pg * p.Hkv + h;
                const int4 *m = reinterpret_cast<const int4 *>(p.mean + ph * D);
                int4 w[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c) w[c] = __ldg(m + c);
                const float ms = p.mean_scale[ph];
#pragma unroll 2
                for (int r = 0; r < some; ++r) {
                    int dot[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int4 q = *reinterpret_cast<const int4 *>(&q8[r][4 * c]);
                        dot[0] = __dp4a(w[c].x, q.x, dot[0]);
                        dot[1] = __dp4a(w[c].y, q.y, dot[1]);
                        dot[2] = __dp4a(w[c].z, q.z, dot[2]);
                        dot[3] = __dp4a(w[c].w, q.w, dot[3]);
                    }
                    const uint32_t o = order_of(((float)(dot[0] + dot[1] + dot[2] + dot[3]) * qs[r]) * ms);
                    k = max(k, min(max(o, 1u), 0xfffffffeu));
                }
            } else if (r0 == 0) {
                atomicExch(&g_status_page_select, (int)FA_ERR_BAD_PAGE);
            }
            if (i < p.keep_first || i >= n - p.keep_last) k = 0xffffffffu;
            if (size == 1) {
                key[i] = r0 == 0 ? k : max(k, key[i]);
            } else {  // this block's own copy holds the maximum over the rows so far
                if (r0 > 0) k = max(k, key[i - begin]);
                if (r0 + kSelRows < rows)
                    key[i - begin] = k;
                else if (rank == 0)
                    key[i] = k;
                else
                    store_cluster(in_first_block(key + i), k);
            }
        }
    }
    if (size > 1)
        cluster_sync();
    else
        __syncthreads();
    if (rank != 0) return;

    // the take-th largest key, eight bits at a time from the top
    uint32_t prefix = 0, known = 0;
    int left = take;  // how many of the keys that agree with the prefix are taken
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += kSelThreads) {
            const int i = i0 + tid;
            const bool in = i < n && (key[min(i, n - 1)] & known) == prefix;
            const uint32_t bin = in ? (key[i] >> shift) & 255u : 256u;
            // scores are alike in their highest bits: equal bins of a warp are counted at once
            const uint32_t same = __match_any_sync(0xffffffffu, bin);
            if (in && lane == __ffs((int)same) - 1) atomicAdd(&hist[bin], __popc(same));
        }
        __syncthreads();
        // sums over the bins from the highest down: thread t has bin 255 - t
        int s = tid < 256 ? hist[255 - tid] : 0;
        const int mine = s;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        for (int w = 0; w < warp; ++w) s += warp_sums[w];
        if (tid < 256 && s >= left && s - mine < left) {
            pick[0] = 255 - tid;
            pick[1] = left - (s - mine);
        }
        __syncthreads();
        prefix |= pick[0] << shift;
        known |= 255u << shift;
        left = (int)pick[1];
    }
    // Positions in ascending order: all keys above, and the first `left` equal ones.
    // A thread has a run of keys; one scan over the threads' counts.
    const int per = (n + kSelThreads - 1) / kSelThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int g = 0, e = 0;
    for (int i = i0; i < i1; ++i) g += key[i] > prefix, e += key[i] == prefix;
    unsigned long long x = (unsigned long long)e << 32 | (uint32_t)g;
    const unsigned long long own = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __shared__ unsigned long long warp_counts[kSelWarps];
    if (lane == 31) warp_counts[warp] = x;
    __syncthreads();
    x -= own;
    for (int w = 0; w < warp; ++w) x += warp_counts[w];
    g = (int)(uint32_t)x, e = (int)(x >> 32);
    for (int i = i0; i < i1; ++i) {
        if (key[i] > prefix)
            sel[g++ + min(e, left)] = i;
        else if (key[i] == prefix) {
            if (e < left) sel[g + e] = i;
            ++e;
        }
    }
}

cudaError_t launch_page_select(int D, const SelectParams &p, cudaStream_t stream) {
    int size = 1;
    while (size < 8 && size * kSelShare < p.max_pages) size *= 2;
    void (*const f)(SelectParams) = D == 64 ? fa_page_select_kernel<64> : fa_page_select_kernel<128>;
    const size_t smem = p.max_pages * sizeof(uint32_t);
    if (smem > 40 * 1024) {  // beyond what a kernel may have, beside its own arrays, without asking
        const cudaError_t e = cudaFuncSetAttribute((const void *)f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_early(f, dim3(size, p.Hkv, p.B), kSelThreads, smem, stream, size, p);
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
