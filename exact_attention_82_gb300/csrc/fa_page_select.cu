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
// cluster of 1 to 8 blocks takes one (sequence, head), and each block scores its share
// of the pages.  The products run on the tensor cores in integers (16 pages by 8 rows by
// 32 elements an instruction; four products a lane and instruction took twice as long,
// most of it to read the queries from shared memory; fp16 products, exact with the bytes as
// subnormal numbers and quicker by themselves, take longer with what prepares them: 6.1 and
// 9.8 us for 5.8 and 9.7).  The scores' bits are
// written into the first block's shared memory, which finds the k-th largest without
// sorting: counted in 2048 equal steps from the least score to the largest, it is among
// the few of one step, and is the one that has the right number of those above it.  Where
// that does not tell them apart (ties, infinities) it is found by its bits, eleven at a time.
// (By bits alone, whose highest are alike, so that counts collide: 6.2 and 10.3 us for 5.8 and
// 9.7.)  8 sequences of 16384 tokens, 8 of 32 heads, pages of 64: 5.8 us; one of 131072, 8 of
// 64 heads, pages of 32: 9.7 us, a chain of latencies: lengths 0.9, queries 1.4, table and
// means twice 2.9, barrier 0.6, the k-th largest 2.7, the list 1.4.
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
constexpr int kSelBins = 2048;
constexpr int kSelShare = 256; // pages of the table that make another block of the cluster worth its while

// Unsigned numbers in the order of the floats; -0 counts as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t order) {
    return __uint_as_float((order & 0x80000000u) ? order & 0x7fffffffu : ~order);
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// c (16 x 8, int32) += a (16 x 32, int8) b (32 x 8, int8)
__device__ __forceinline__ void mma_s8(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

__device__ __forceinline__ void min_cluster(uint32_t a, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void max_cluster(uint32_t a, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) fa_page_select_kernel(const __grid_constant__ SelectParams p) {
    grid_wait();
    extern __shared__ uint32_t key[];  // [max_pages] the order of each page's score, in the first block
    __shared__ __align__(16) int q8[kSelRows][D / 4];
    __shared__ float qs[kSelRows];
    __shared__ __align__(16) int hist[kSelBins];
    __shared__ int warp_sums[kSelWarps];
    __shared__ uint32_t pick[3], key_min, key_max;  // of the keys that are scores
    __shared__ int listed;
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
        if (tid == 0) {
            p.sel_count[bh] = take;
            key_min = 0xffffffffu, key_max = 0, listed = 0;
        }
        for (int i = take + tid; i < p.top_k; i += kSelThreads) sel[i] = -1;
    }
    if (size > 1) cluster_arrive();      // this block's shared memory is there
    if (n <= p.top_k || take == 0) {  // every page, or none; the same in all blocks of the cluster
        if (rank == 0)
            for (int i = tid; i < take; i += kSelThreads) sel[i] = i;
        if (size > 1) cluster_wait();
        return;
    }

    // ---- scores: 16 pages at a time a warp
    const int *const table = p.table + (long long)b * p.max_pages;
    const int rows = (q1 - q0) * p.G, g = lane >> 2, t = lane & 3;
    const int chunk = (((n + (int)size - 1) / (int)size) + 15) & ~15, begin = min(n, (int)rank * chunk), end = min(n, begin + chunk);
    constexpr int KS = D / 32;  // instructions along a row
    bool waited = size == 1;
    uint32_t k_min = 0xffffffffu, k_max = 0;
    for (int r0 = 0; r0 < rows; r0 += kSelRows) {
        // The first pages are asked for before the queries are rounded.  Lane t takes
        // 16-byte pieces t (and t + 4) of the mean keys of pages g and g + 8.
        int4 w[2][D / 64];
        float ms[2];
        int pg[2];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = i0 + g + 8 * j;
                pg[j] = i < end ? table[i] : 0;
                const bool good = pg[j] >= 0 && pg[j] < p.num_pages;
                if (!good) {
                    if (r0 == 0) atomicExch(&g_status_page_select, (int)FA_ERR_BAD_PAGE);
                    pg[j] = -1;
                }
                const long long ph = (long long)max(pg[j], 0) * p.Hkv + h;
                const int4 *const m = reinterpret_cast<const int4 *>(p.mean + ph * D) + t;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) w[j][c] = __ldg(m + 4 * c);
                ms[j] = p.mean_scale[ph];
            }
        };
        int i0 = begin + warp * 16;
        if (i0 < end) fetch(i0);
        if (r0 > 0) __syncthreads();
        const int some = min(kSelRows, rows - r0);
        for (int r = warp; r < kSelRows; r += kSelWarps) {
            float x[D / 32], amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) x[i] = 0.f;
            if (r < some) {
                const int tok = q0 + (r0 + r) / p.G, gq = (r0 + r) % p.G;
                const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(
                    static_cast<const __nv_bfloat16 *>(p.q) + (long long)tok * p.q_stride + (long long)(h * p.G + gq) * D);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const float2 f = __bfloat1622float2(q[lane * (D / 64) + i]);
                    x[2 * i] = f.x, x[2 * i + 1] = f.y;
                }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                if (!(fabsf(x[i]) < INFINITY)) x[i] = 0.f;
                amax = fmaxf(amax, fabsf(x[i]));
            }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            // 127 / amax is past the largest float below 2^-121: such rows are scaled, exactly
            const float up = amax < 0x1p-100f ? 0x1p100f : 1.f, inv = amax > 0.f ? 127.f / (amax * up) : 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                reinterpret_cast<int8_t *>(q8[r])[lane * (D / 32) + i] = (int8_t)__float2int_rn(x[i] * up * inv);
            if (lane == 0) qs[r] = amax / 127.f;
        }
        __syncthreads();
        // the order of a row's elements is free as long as both operands have the same
        int qf[kSelRows / 8][KS][2];
        float qscale[kSelRows / 8][2];
#pragma unroll
        for (int nt = 0; nt < kSelRows / 8; ++nt) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) qf[nt][k][c] = q8[nt * 8 + g][D == 128 ? 4 * (t + 4 * c) + k : 4 * t + 2 * k + c];
            qscale[nt][0] = qs[nt * 8 + 2 * t], qscale[nt][1] = qs[nt * 8 + 2 * t + 1];
        }
        k_min = 0xffffffffu, k_max = 0;  // (the last rows' stay)
        for (; i0 < end; i0 += 16 * kSelWarps) {
            uint32_t best[2] = {0, 0};
#pragma unroll
            for (int nt = 0; nt < kSelRows / 8; ++nt) {
                if (nt * 8 >= some) continue;
                int dot[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    int a[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            a[j][c] = reinterpret_cast<const int *>(&w[j][D == 128 ? c : 0])[D == 128 ? k : 2 * k + c];
                    mma_s8(dot, a[0][0], a[1][0], a[0][1], a[1][1], qf[nt][k][0], qf[nt][k][1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (nt * 8 + 2 * t + (j & 1) < some) {
                        const uint32_t o = order_of(((float)dot[j] * qscale[nt][j & 1]) * ms[j >> 1]);
                        best[j >> 1] = max(best[j >> 1], min(max(o, 1u), 0xfffffffeu));
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                best[j] = max(best[j], __shfl_xor_sync(0xffffffffu, best[j], 1));
                best[j] = max(best[j], __shfl_xor_sync(0xffffffffu, best[j], 2));
                if (pg[j] < 0) best[j] = 0;  // a page outside the cache: behind all others
            }
            if (!waited) {
                cluster_wait();
                waited = true;
            }
            const int i = i0 + g + 8 * t;  // lanes t = 0 and 1 write pages g and g + 8
            uint32_t k = t == 0 ? best[0] : best[1];
            if (t < 2 && i < end) {
                if (i < p.keep_first || i >= n - p.keep_last) k = 0xffffffffu;
                if (r0 > 0) k = max(k, key[i - begin]);  // this block's own copy: the maximum over the rows so far
                if (k != 0xffffffffu && k != 0) k_min = min(k_min, k), k_max = max(k_max, k);
                if (rank == 0 || r0 + kSelRows < rows)
                    key[i - begin] = k;
                else
                    store_cluster(in_first_block(key + i), k);
            }
            if (i0 + 16 * kSelWarps < end) fetch(i0 + 16 * kSelWarps);
        }
    }
    k_min = __reduce_min_sync(0xffffffffu, k_min), k_max = __reduce_max_sync(0xffffffffu, k_max);
    if (lane == 0 && k_max > 0) {
        min_cluster(in_first_block(&key_min), k_min);
        max_cluster(in_first_block(&key_max), k_max);
    }
    if (size > 1) {
        if (!waited) cluster_wait();
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;

    // Finds in which bin of `hist`, counted from the highest down, the left-th member is:
    // pick = {the bin, how many of its members are taken, how many it has}.
    auto find_bin = [&](int left) {
        // thread t has bin 2047 - 4 t and the three below
        const int4 c4 = *reinterpret_cast<const int4 *>(&hist[kSelBins - 4 - 4 * tid]);
        const int c[4] = {c4.w, c4.z, c4.y, c4.x}, mine = c[0] + c[1] + c[2] + c[3];
        int s = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w)
            if (w < warp) s += warp_sums[w];
        int before = s - mine;
        if (before < left && s >= left) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before < left && before + c[j] >= left) {
                    pick[0] = kSelBins - 1 - 4 * tid - j;
                    pick[1] = left - before;
                    pick[2] = c[j];
                }
                before += c[j];
            }
        }
        __syncthreads();
    };
    static_assert(kSelBins == 4 * kSelThreads, "");

    // The take-th largest key, `prefix`, and how many of those equal to it are taken, `left`.
    uint32_t prefix = 0;
    int left = take;
    const float low = float_of(key_min), range = float_of(key_max) - low;  // NaN where there is no score
    const float per_bin = (kSelBins - 1) / range;
    bool found = false;
    const int scored_left = take - p.keep_first - p.keep_last;  // the kept pages' keys are above all others
    if (scored_left == 0) {
        prefix = 0xfffffffeu, left = 0;
        found = true;
    } else if (range > 0.f && per_bin < INFINITY && range < INFINITY) {
        // no less for larger scores; pages outside the cache are in bin 0
        auto bin_of = [&](uint32_t k) { return k ? min(kSelBins - 1, (int)((float_of(k) - low) * per_bin)) : 0; };
        *reinterpret_cast<int4 *>(&hist[4 * tid]) = make_int4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < n; i += kSelThreads) {
            const uint32_t k = key[i];
            if (k != 0xffffffffu) atomicAdd(&hist[bin_of(k)], 1);
        }
        __syncthreads();
        find_bin(scored_left);
        const int bin = (int)pick[0], in_bin = (int)pick[2];
        left = (int)pick[1];
        if (in_bin <= kSelThreads) {
            uint32_t *const list = reinterpret_cast<uint32_t *>(hist);  // the bin's members, over the counts
#pragma unroll 4
            for (int i = tid; i < n; i += kSelThreads) {
                const uint32_t k = key[i];
                if (k != 0xffffffffu && bin_of(k) == bin) list[atomicAdd(&listed, 1)] = k;
            }
            __syncthreads();
            if (tid < in_bin) {
                const uint32_t mine = list[tid];
                int above = 0, equal = 0;
#pragma unroll 4
                for (int i = 0; i < in_bin; ++i) above += list[i] > mine, equal += list[i] == mine;
                if (above < left && left <= above + equal) pick[0] = mine, pick[1] = left - above;
            }
            __syncthreads();
            prefix = pick[0], left = (int)pick[1];
            found = true;
        } else {
            left = take;
        }
    }
    // by its bits, eleven at a time from the top
    uint32_t known = 0;
    bool all = found;  // whether all that agree with the prefix are taken
    for (int shift = 21; shift > -11 && !all; shift -= shift == 10 ? 10 : 11) {
        const uint32_t digit = shift == 0 ? 1023u : 2047u;
        *reinterpret_cast<int4 *>(&hist[4 * tid]) = make_int4(0, 0, 0, 0);
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += 4 * kSelThreads) {
            uint32_t k[4];
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * kSelThreads + tid;
                k[j] = i < n ? key[i] : 0u;
                in[j] = i < n && (k[j] & known) == prefix;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t members = __ballot_sync(0xffffffffu, in[j]);
                if (!members) continue;
                // scores are alike in their highest bits: those in one bin with the first are counted at once
                const uint32_t bin = (k[j] >> shift) & digit, first = __shfl_sync(0xffffffffu, bin, __ffs((int)members) - 1);
                const uint32_t same = __ballot_sync(0xffffffffu, in[j] && bin == first);
                if (lane == 0) atomicAdd(&hist[first], __popc(same));
                if (in[j] && bin != first) atomicAdd(&hist[bin], 1);
            }
        }
        __syncthreads();
        find_bin(left);
        prefix |= pick[0] << shift;
        known |= digit << shift;
        left = (int)pick[1];
        all = left == (int)pick[2];
        __syncthreads();
        if (shift == 0) break;
    }
    if (all && !found) {  // every key from the prefix on, whatever its other bits
        prefix -= 1;
        left = 0;
    }
    // Positions in ascending order: all keys above, and the first `left` equal ones.
    // A thread has a run of keys; one scan over the threads' counts.
    const int per = (n + kSelThreads - 1) / kSelThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int gt = 0, eq = 0;
    uint32_t marks = 0;  // of the first 32 keys: those that are not below
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key[i];
        gt += k > prefix, eq += k == prefix;
        if (k >= prefix && i - i0 < 32) marks |= 1u << (i - i0);
    }
    unsigned long long x = (unsigned long long)eq << 32 | (uint32_t)gt;
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
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) x += warp_counts[w];
    gt = (int)(uint32_t)x, eq = (int)(x >> 32);
    auto put = [&](int i) {
        if (key[i] > prefix)
            sel[gt++ + min(eq, left)] = i;
        else if (key[i] == prefix) {
            if (eq < left) sel[gt + eq] = i;
            ++eq;
        }
    };
    for (; marks; marks &= marks - 1) put(i0 + __ffs((int)marks) - 1);
    for (int i = i0 + 32; i < i1; ++i) put(i);
}

cudaError_t launch_page_select(int D, const SelectParams &p, cudaStream_t stream) {
    int size = 1;
    while (size < 8 && size * kSelShare < p.max_pages) size *= 2;
    void (*const f)(SelectParams) = D == 64 ? fa_page_select_kernel<64> : fa_page_select_kernel<128>;
    const size_t smem = p.max_pages * sizeof(uint32_t);
    if (smem > 32 * 1024) {  // beyond what a kernel may have, beside its own arrays, without asking
        // always the most: the limit is the function's, and another thread's call would lower one set to this call's size
        const cudaError_t e = cudaFuncSetAttribute((const void *)f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectMaxPages * (int)sizeof(uint32_t));
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
