// fa_rope.cu -- rotary positions of queries and keys on GB300 (sm_103a), and their
// gradient (the transposed rotation).
//
// For pair i of a token at position p, with the angle t = p * phase_i (fa_rope.cuh) and
// amplitude a:  (y1, y2) = a (x1 cos t - x2 sin t, x1 sin t + x2 cos t); the gradient has
// -sin t.  One rounding, of the result to bf16.
//
// Bound by HBM: 2 bytes read and 2 written an element.  What must not cost more is the
// angles: sine and cosine of a (token, pair) are the same for every head, so a thread
// keeps eight pairs of one token (16 elements of a head, two 16-byte pieces) and goes
// through the heads of its group, queries and keys alike, with the loads of several
// heads in flight.  A head's elements behind the rotated part are copied by the threads
// that have no pairs.  Strides are free, so the call that rotates also takes heads out of
// a fused projection and lays them out for attention.
//
// Measured: 4 x 4096 tokens, 16 and 16 heads, D = 128 42.3 us, 6,350 GB/s (93% of the copy rate); 16384 packed tokens, 32
// and 8 heads, positions past 10^5, 52.4 us (94%); 16 x 1000 tokens, 32 and 32 heads, D = 64, half of each rotated in neighbouring
// pairs, as views [B, H, S, D], 43 us (90%); 64 tokens 2.8 us, a launch and two latencies.  Two or six heads in flight instead of
// four: 45.0 and 44.6 for 43.8 us in the third case; blocks of 128 or 512 threads 47.0 and 44.9.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "fa_rope.cuh"

namespace fa {

constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 4;  // heads whose loads are in flight

template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const __grid_constant__ RopeParams p, int tpt_log2, int group) {
    grid_wait();
    const int sub = threadIdx.x & ((1 << tpt_log2) - 1);
    const long long at = (long long)blockIdx.x * (kRopeThreads >> tpt_log2) + (threadIdx.x >> tpt_log2);
    if (at >= (long long)p.B * p.S) return;
    const int b = (int)(at / p.S), s = (int)(at - (long long)b * p.S);
    const bool turned = sub < p.rot / 16;
    const int2 piece = rope_pieces(sub, p.rot, INTER);
    float2 f[8];
    if (turned) {
        const int position = p.positions ? __ldg(p.positions + (long long)b * p.positions_stride + s) : s;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = rope_factor(__ldg(p.phases + 8 * sub + j), position, p.amplitude);
            if (p.inverse) f[j].y = -f[j].y;
        }
    }
    const int h0 = blockIdx.y * group, h1 = min(h0 + group, p.H[0] + p.H[1]);
    auto row = [&](const long long (&stride)[3], int h) { return b * stride[0] + s * stride[1] + h * stride[2]; };
#pragma unroll 1
    for (int h = h0; h < h1; h += kRopeAhead) {
        uint4 w[kRopeAhead][2];
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            if (h + i >= h1) break;
            const int t = h + i >= p.H[0] ? 1 : 0;
            const __nv_bfloat16 *const x = static_cast<const __nv_bfloat16 *>(p.x[t]) + row(p.x_stride[t], h + i - (t ? p.H[0] : 0));
            w[i][0] = *reinterpret_cast<const uint4 *>(x + 8 * piece.x);
            w[i][1] = *reinterpret_cast<const uint4 *>(x + 8 * piece.y);
        }
#pragma unroll
        for (int i = 0; i < kRopeAhead; ++i) {
            if (h + i >= h1) break;
            const int t = h + i >= p.H[0] ? 1 : 0;
            if (turned) {
                float x[16];
                bf16x8_to_float(w[i][0], x);
                bf16x8_to_float(w[i][1], x + 8);
                rope_turn16<INTER>(x, f);
                w[i][0] = float_to_bf16x8(x);
                w[i][1] = float_to_bf16x8(x + 8);
            }
            __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(p.y[t]) + row(p.y_stride[t], h + i - (t ? p.H[0] : 0));
            *reinterpret_cast<uint4 *>(y + 8 * piece.x) = w[i][0];
            *reinterpret_cast<uint4 *>(y + 8 * piece.y) = w[i][1];
        }
    }
}

cudaError_t launch_rope(const RopeParams &p, int num_sms, cudaStream_t stream) {
    const int tpt_log2 = p.D == 64 ? 2 : 3;  // D / 16 threads a token
    const int tokens = kRopeThreads >> tpt_log2, H = p.H[0] + p.H[1];
    const long long blocks = ((long long)p.B * p.S + tokens - 1) / tokens;
    // Heads a block goes through: all where the tokens fill the chip, fewer where they
    // do not (each group computes the angles anew).  With 4, 8, 16 and 32 blocks for each SM the three larger cases above take
    // 44.8 43.8 43.0 43.0, 55.2 53.6 53.3 52.6 and 53.9 47.1 43.8 43.1 us.
    long long groups = (32ll * num_sms + blocks - 1) / blocks;
    if (groups > H) groups = H;
    const int group = (int)((H + groups - 1) / groups);
    const dim3 grid((unsigned)blocks, (unsigned)((H + group - 1) / group));
    return p.interleaved ? launch_early(fa_rope_kernel<true>, grid, kRopeThreads, 0, stream, 1, p, tpt_log2, group)
                         : launch_early(fa_rope_kernel<false>, grid, kRopeThreads, 0, stream, 1, p, tpt_log2, group);
}

}  // namespace fa
