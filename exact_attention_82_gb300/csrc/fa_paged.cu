// fa_paged.cu -- attention of a few query tokens over the paged 8-bit cache
// on GB300 (sm_103a): O = softmax(scale q K^T) V and the row log-sum-exp, K and
// V read as e4m3 codes with one scale for each page and head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_paged = 0;

__device__ __forceinline__ float2 codes2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// One CTA of four warps for each query row; each warp takes every fourth key
// with its own running maximum and sum, and the four are joined at the end.
template <int D>
__global__ void __launch_bounds__(128) fa_fwd_paged_simple(const PagedParams p) {
    constexpr int E = D / 32;
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int t = blockIdx.x, qh = blockIdx.y, h = qh / p.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b = 0;
    while (b < p.B && p.cu_q[b + 1] <= t) ++b;
    if (b == p.B) return;
    const int q0 = max(0, min(p.cu_q[b], p.T)), q1 = max(q0, min(p.cu_q[b + 1], p.T));
    const int page = 1 << p.page_log2;
    const long long len = max(0ll, min((long long)p.seq_lens[b], (long long)p.max_pages << p.page_log2));
    const long long limit = len - (q1 - q0) + (t - q0) + 1;
    const int n_pages = (int)((len + page - 1) >> p.page_log2);
    const long long bh = (long long)b * p.Hkv + h;
    const int n = p.sel ? max(0, min(p.sel_count[bh], p.sel_width)) : n_pages;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (long long)t * p.q_stride + (long long)qh * D + lane * E;
    float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < E; ++i) x[i] = __bfloat162float(q[i]);
    for (int s = 0; s < n; ++s) {
        const int pos = p.sel ? p.sel[bh * p.sel_width + s] : s;
        const int pg = pos >= 0 && pos < n_pages ? p.table[(long long)b * p.max_pages + pos] : -1;
        if ((long long)pos * page >= limit && pos >= 0 && pos < n_pages) continue;
        if (pg < 0 || pg >= p.num_pages) {
            m = l = __int_as_float(0x7fc00000);
            atomicExch(&g_status_paged, (int)FA_ERR_BAD_PAGE);
            continue;
        }
        const long long ph = (long long)pg * p.Hkv + h;
        const float ks = p.k_scale[ph], vs = p.v_scale[ph];
        for (int r = warp; r < page && (long long)pos * page + r < limit; r += 4) {
            const long long at = ((ph << p.page_log2) + r) * D + lane * E;
            float d = 0.f, v[E];
            for (int i = 0; i < E; i += 2) {
                const float2 k2 = codes2(*reinterpret_cast<const uint16_t *>(p.k_pages + at + i));
                const float2 v2 = codes2(*reinterpret_cast<const uint16_t *>(p.v_pages + at + i));
                d += k2.x * x[i] + k2.y * x[i + 1];
                v[i] = v2.x * vs, v[i + 1] = v2.y * vs;
            }
            for (int k = 16; k; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
            const float y = d * ks * p.scale_log2, m1 = fmaxf(m, y), f = exp2f(m - m1), e = exp2f(y - m1);
            m = m1 == m1 ? m1 : y;
            l = l * f + e;
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + e * v[i];
        }
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
    for (int i = 0; i < E; ++i) sm_o[warp][lane * E + i] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    bool bad = false;
    for (int w = 0; w < 4; ++w) bad |= !(sm_l[w] == sm_l[w]), M = fmaxf(M, sm_m[w]);
    for (int w = 0; w < 4; ++w) L += sm_m[w] == -INFINITY ? 0.f : sm_l[w] * exp2f(sm_m[w] - M);
    if (bad) L = M = __int_as_float(0x7fc00000);
    for (int d = threadIdx.x; d < D; d += 128) {
        float y = 0.f;
        for (int w = 0; w < 4; ++w) y += sm_m[w] == -INFINITY ? 0.f : sm_o[w][d] * exp2f(sm_m[w] - M);
        if (bad) y = L;
        static_cast<__nv_bfloat16 *>(p.o)[((long long)t * p.Hkv * p.G + qh) * D + d] =
            __float2bfloat16_rn(M == -INFINITY ? 0.f : y / L);
    }
    if (threadIdx.x == 0)
        p.lse[(long long)t * p.Hkv * p.G + qh] = M == -INFINITY ? M : (M + log2f(L)) * 0.69314718055994531f;
}

size_t paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int num_sms) {
    return (size_t)num_sms * 4 * 16 * (D + 2) * sizeof(float);
}

cudaError_t launch_fwd_paged(int D, const PagedParams &p, int num_sms, cudaStream_t stream) {
    const dim3 grid(p.T, p.Hkv * p.G);
    if (D == 64)
        fa_fwd_paged_simple<64><<<grid, 128, 0, stream>>>(p);
    else
        fa_fwd_paged_simple<128><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t paged_status_read_and_clear(int *out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_paged, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status_paged, &zero, sizeof(int));
    *out = v;
    return e;
}

}  // namespace fa
