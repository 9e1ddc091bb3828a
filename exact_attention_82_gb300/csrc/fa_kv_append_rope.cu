// fa_kv_append_rope.cu -- fa_kv_append with the keys rotated on the way, and the step's
// queries rotated beside, on GB300 (sm_103a).
//
// The page's scale comes from the rotated keys, so a run's rows are rotated, their largest
// magnitude taken, and only then rounded; in between they are kept in fp32, so that a key is
// rounded once.  Values go the way of fa_kv_append, by the same function (fa_kv_append.cuh); its
// kernel (fa_kv_cache.cu) stays apart: with the rotation's instantiations beside it in one kernel it lost a sixth to registers.
//
// Bound by HBM: 4 bytes read and 2 written for a key and a value element, 2 and 2 for a
// query's.  A prompt of 16384 tokens, 8 heads of keys, 32 of queries, D = 128: 62.3 us, 5,920
// GB/s (87% of the copy rate), with means 63.6; without queries 28.8, where fa_kv_append takes 17.4: a team waits
// for memory, for the largest magnitude of the page and to be written, head after head, and a quarter
// of the keys' time is sines and cosines.  (A head's rows asked for while the one before is written: no gain.)
// 64 single tokens 5.5 us (with means 7.6), 256 14.4 us.  16 ragged prompts of 30 to 1000 tokens, 32 heads, D = 64, pages of 16: 21.2 us
// (with means 28.6), where fa_kv_append takes 12.8 on the same runs: the values' path has the registers of the rotation's kernel here, and so fewer
// threads, and every instantiation spills 208 to 424 bytes.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_kv_append.cuh"
#include "fa_paged.h"
#include "fa_rope.cuh"

namespace fa {

static __device__ int g_status_kv_append_rope = 0;

constexpr int kRopeThreadsAnSm = 1024;  // that the kernel's registers are held to (768: 89 us for the prompt, 1536: 96, when it took 78)
constexpr int kAppendFill = 1024;       // threads an SM, of each kind, that the windows' blocks are to make up

enum class Turn { none, halves, pairs };  // whether rows are rotated, and which elements make a pair

// One of `share` blocks' part of the runs of a window, of heads h0 .. h0 + heads - 1 of K (kv = 0) or V; `turns`: shared memory for the
// angles of a team's run, which all its heads take.  Its teams take run after run, or (EVEN) as many (run, head) each, one run's heads in a
// row, so that single tokens (many runs) and prompts (few) keep the same blocks busy.
template <int D, int PAGE, class C, Turn TURN, bool EVEN>
__device__ __forceinline__ void append_runs(const AppendParams &p, const int share, const int h0, const int heads, const int kv, AppendShared<D, PAGE, C> &sm,
                                            const int win, const int part, float4 *const turns = nullptr) {
    int *const slot_of = sm.slot_of;
    uint32_t *const starts = sm.starts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = C::TEAMS == 1 ? 0 : warp / C::TEAM, first_warp = team * C::TEAM, tt = tid - first_warp * 32;
    const int t0 = win * kWindow;
    const int limit = p.num_pages * PAGE;  // fewer than 2^31
    const __nv_bfloat16 *const x_first = static_cast<const __nv_bfloat16 *>(kv ? p.x[1] : p.x[0]) + h0 * D;
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
        if (s >= limit) atomicExch(&g_status_kv_append_rope, (int)FA_ERR_BAD_PAGE);
        const uint32_t m = __ballot_sync(0xffffffffu, start);
        if (lane == 0) starts[i / 32] = m;
    }
    __syncthreads();
    // this lane's two tokens, and how many runs begin before each
    const uint32_t s0 = starts[0], s1 = starts[1], lt = (1u << lane) - 1;
    const int rank0 = (s0 >> lane) & 1u ? __popc(s0 & lt) : -1, rank1 = (s1 >> lane) & 1u ? __popc(s0) + __popc(s1 & lt) : -1;
    const int runs = __popc(s0) + __popc(s1);
    const int each = (runs * heads + share * C::TEAMS - 1) / (share * C::TEAMS);
    int item = (part * C::TEAMS + team) * (EVEN ? each : 1);
    const int last = EVEN ? min(item + each, runs * heads) : runs;
    while (item < last) {
        int run = item, h = h0, h1 = h0 + heads;
        if constexpr (EVEN) {
            run = item / heads;
            h += item - run * heads;
            h1 = min(h1, h + last - item);
            item += h1 - h;
        } else {
            item += share * C::TEAMS;
        }
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

        const AppendRun of{i0, slot, n};
        // Rotated rows: a thread has two pieces of each of its rows, whose elements are one
        // another's partners, and keeps them in fp32 between the pass that takes the largest
        // magnitude and the one that writes codes, so that they are rounded once.
        auto append_turned = [&](auto whole) {
            constexpr bool W = decltype(whole)::value;
            const __nv_bfloat16 *const x_of = x_first + (h - h0) * D;
            constexpr int TPT = D / 16, ROWS = 32 * C::TEAM / TPT, PASSES = PAGE / ROWS;
            static_assert(PASSES * 8 <= 32, "sums of codes are exact in fp32");
            const int sub = tt % TPT, r0 = tt / TPT;
            const long long ph = (long long)pg * p.Hkv + h;
            const float was = W ? 0.f : scale_of[ph];
            const int2 piece = rope_pieces(sub, p.rot, TURN == Turn::pairs);
            uint8_t *const codes = pages_of + ph * PAGE * D;
            const bool mean = p.mean != nullptr, turned = sub < p.rot / 16;
            // ---- what is read, at once: the run's rows, and codes before it for the mean
            uint4 w[PASSES][2];
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r0 + i * ROWS;
                w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
                if (W || (r >= off && r < off + n)) {
                    const long long token = (long long)(t0 + i0 - off) + r;
                    w[i][0] = __ldg(reinterpret_cast<const uint4 *>(x_of + token * stride + 8 * piece.x));
                    w[i][1] = __ldg(reinterpret_cast<const uint4 *>(x_of + token * stride + 8 * piece.y));
                } else if (mean && r < off) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(codes + r * D + 8 * piece.x);
                    const uint2 b = *reinterpret_cast<const uint2 *>(codes + r * D + 8 * piece.y);
                    w[i][0] = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
            float y[PASSES][16];
            uint32_t am = 0;  // magnitudes of fp32 compare as integers; infinities and NaN do not count
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r0 + i * ROWS;
                if (!W && (r < off || r >= off + n)) continue;
                bf16x8_to_float(w[i][0], y[i]);
                bf16x8_to_float(w[i][1], y[i] + 8);
                if (turned) {
                    float2 f[8];
                    const float4 *const from = turns + (r - off) * (p.rot / 4) + sub;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 two = from[j * (p.rot / 16)];
                        f[2 * j] = make_float2(two.x, two.y), f[2 * j + 1] = make_float2(two.z, two.w);
                    }
                    rope_turn16<TURN == Turn::pairs>(y[i], f);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t u = __float_as_uint(y[i][j]) & 0x7fffffffu;
                    am = max(am, u < 0x7f800000u ? u : 0u);
                }
            }
            float scale = pow2_scale(__uint_as_float(me.join_max(am)));
            if (!W && off > 0) scale = fmaxf(scale, was);
            if (tt == 0) scale_of[ph] = scale;  // every thread has read it (the barrier above)
            const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
            const float inv_scale = 1.f / scale, shrink = was / scale;
            const bool grown = !W && off > 0 && scale != was;  // the rows before the run are rounded again
            float sum[2][8] = {};
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r0 + i * ROWS;
                if (!W && (r < off || r >= off + n)) continue;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x = y[i][j];
                    y[i][j] = x * inv_scale;  // exact for powers of two; the remainder corrects it otherwise
                    if (!W && !pow2 && fabsf(x) < INFINITY) y[i][j] = fmaf(fmaf(-y[i][j], scale, x), inv_scale, y[i][j]);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float *const v = y[i] + 8 * c;
                    const uint2 code = make_uint2(pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7]));
                    *reinterpret_cast<uint2 *>(codes + r * D + 8 * (c ? piece.y : piece.x)) = code;
                    if (mean) add8(without_nan(code), sum[c]);
                }
            }
            if (!W && off > 0 && (mean || grown)) {
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int r = r0 + i * ROWS;
                    if (r >= off) continue;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint2 *const at = reinterpret_cast<uint2 *>(codes + r * D + 8 * (c ? piece.y : piece.x));
                        uint2 code = mean ? (c ? make_uint2(w[i][0].z, w[i][0].w) : make_uint2(w[i][0].x, w[i][0].y)) : *at;
                        float v[8];
                        if (grown) {
                            decode8(code, v);
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] *= shrink;
                            code = encode8(v);
                            *at = code;
                        }
                        decode8(without_nan(code), v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[c][j] += v[j];
                    }
                }
            }
            if (mean) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        int x = (int)(sum[c][j] * 512.f);
#pragma unroll
                        for (int d = TPT; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                        if (lane < TPT) sm.sums[warp][8 * (c ? piece.y : piece.x) + j] = x;
                    }
                me.write_mean(ph, scale, W ? PAGE : off + n);
            }
        };
        if constexpr (TURN != Turn::none) {
            // The run's angles: pair 8 s + 2 j + e of row r is half e of word (r, j, s), so that the threads of a row read
            // neighbouring words.
            const int pairs = p.rot / 2;
            for (int e = tt; e < n * pairs; e += 32 * C::TEAM) {
                const int r = e / pairs, pair = e - r * pairs;
                const float2 f = rope_factor(__ldg(p.phases + pair), __ldg(p.positions + t0 + i0 + r), p.amplitude);
                reinterpret_cast<float2 *>(turns)[2 * (r * (p.rot / 4) + (pair >> 1 & 3) * (p.rot / 16) + (pair >> 3)) + (pair & 1)] = f;
            }
            me.sync();
        }
#pragma unroll 1
        do {
            if constexpr (TURN != Turn::none) {
                if (n == PAGE)
                    append_turned(std::true_type());
                else
                    append_turned(std::false_type());
            } else {
                const __nv_bfloat16 *const x_of = x_first + (h - h0) * D;
                if (n == PAGE)
                    me.template append<true, false>(of, h, false, x_of, stride, pages_of, scale_of);
                else
                    me.template append<false, false>(of, h, false, x_of, stride, pages_of, scale_of);
            }
            me.sync();  // the next run overwrites the shared words
        } while (++h < h1);
    }
}

// Keys rotated on the way.  Blocks of a third kind rotate queries, of the key/value heads' groups, so that a step has
// one launch for keys, values and queries.  The keys' blocks, which wait for most, are the first to begin (neighbouring
// blocks of different kinds instead: three prompts of 5000 tokens 64 for 60 us, 16384 tokens in pages of 128 73 for 70).  A sine and cosine
// is some 50 instructions, and the same for all heads: a block takes `per` heads, and their angles once
// (a prompt of 16384 tokens, 8 heads of keys, 32 of queries: 109 us with an angle for every head).
template <int D, int PAGE, bool INTER, bool EVEN>
__global__ void __launch_bounds__(AppendCfg<D, PAGE, 32>::THREADS, kRopeThreadsAnSm / AppendCfg<D, PAGE, 32>::THREADS) fa_kv_append_rope_kernel(const __grid_constant__ AppendParams p, int share, int per, int q_tokens, int q_groups) {
    using C = AppendCfg<D, PAGE, 32>;
    grid_wait();
    extern __shared__ __align__(16) float4 turns_sm[];
    __shared__ AppendShared<D, PAGE, C> sm;
    const int windows = (p.T + kWindow - 1) / kWindow, each = windows * share, kind = min((int)blockIdx.x / each, 2);
    const int block = (int)blockIdx.x - kind * each, n = kind < 2 ? share : q_tokens * q_groups, win = block / n, part = block % n;
    const int h0 = EVEN ? 0 : blockIdx.y * per, heads = EVEN ? p.Hkv : min(per, p.Hkv - h0);
    if (kind == 0) {
        append_runs<D, PAGE, C, INTER ? Turn::pairs : Turn::halves, EVEN>(p, share, h0, heads, 0, sm, win, part,
                                                                          turns_sm + threadIdx.x / (32 * C::TEAM) * PAGE * (p.rot / 4));
    } else if (kind == 1) {
        append_runs<D, PAGE, C, Turn::none, EVEN>(p, share, h0, heads, 1, sm, win, part);
    } else {
        constexpr int TPT = D / 16, TOKENS = C::THREADS / TPT;
        const int sub = threadIdx.x % TPT, group = part / q_tokens;
        const int all = heads * p.G, a_group = (all + q_groups - 1) / q_groups, q0 = h0 * p.G + min(group * a_group, all), q_heads = min(a_group, h0 * p.G + all - q0);
        const bool turned = sub < p.rot / 16;
        const int2 piece = rope_pieces(sub, p.rot, INTER);
        for (int i = part % q_tokens * TOKENS + threadIdx.x / TPT; i < kWindow; i += q_tokens * TOKENS) {
            const int t = win * kWindow + i;
            if (t >= p.T) break;
            float2 f[8];
            if (turned) {
                const int position = __ldg(p.positions + t);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = rope_factor(__ldg(p.phases + 8 * sub + j), position, p.amplitude);
            }
            const __nv_bfloat16 *const x = static_cast<const __nv_bfloat16 *>(p.q) + t * p.q_stride + (long long)q0 * D;
            __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(p.q_out) + t * p.q_out_stride + (long long)q0 * D;
            constexpr int AHEAD = 4;  // heads whose loads are in flight (a store may not pass a load that is written below it)
#pragma unroll 1
            for (int g = 0, n = q_heads; g < n; g += AHEAD) {
                uint4 w[AHEAD][2];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (g + k >= n) break;
                    w[k][0] = *reinterpret_cast<const uint4 *>(x + (g + k) * D + 8 * piece.x);
                    w[k][1] = *reinterpret_cast<const uint4 *>(x + (g + k) * D + 8 * piece.y);
                }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (g + k >= n) break;
                    if (turned) {
                        float v[16];
                        bf16x8_to_float(w[k][0], v);
                        bf16x8_to_float(w[k][1], v + 8);
                        rope_turn16<INTER>(v, f);
                        w[k][0] = float_to_bf16x8(v);
                        w[k][1] = float_to_bf16x8(v + 8);
                    }
                    *reinterpret_cast<uint4 *>(y + (g + k) * D + 8 * piece.x) = w[k][0];
                    *reinterpret_cast<uint4 *>(y + (g + k) * D + 8 * piece.y) = w[k][1];
                }
            }
        }
    }
}

template <int D, int PAGE>
static cudaError_t launch_append_rope(const AppendParams &p, int num_sms, cudaStream_t stream) {
    using C = AppendCfg<D, PAGE, 32>;
    const int windows = (p.T + kWindow - 1) / kWindow;
    int share, groups = 1, per = 0, q_tokens = 0, q_groups = 0;  // blocks of each kind for a window (and group of heads)
    const bool even = windows < num_sms;
    if (!even) {
        // With a window for each SM the tokens are prompts': groups of heads, as many as fill the chip, and no more blocks than a prompt's
        // window has runs for (others would find none: 16384 tokens, 8 and 32 heads, D = 128, pages of 64 70.6 -> 64.9 us, of 128 83.9 -> 73.2).
        // Many short runs instead are a block's one after another: 4,096 sequences of three tokens 245 us, shared out as below 235; the
        // prompt of 16384 62.4 and 67.7.
        constexpr int prompt = std::max(1, (kWindow / PAGE + (C::TEAMS > 1 ? C::TEAMS : 0)) / C::TEAMS);
        groups = std::min((kAppendFill / C::THREADS * num_sms + windows - 1) / windows, p.Hkv);
        per = (p.Hkv + groups - 1) / groups;
        groups = (p.Hkv + per - 1) / per;
        share = prompt;
        if (p.q) q_tokens = prompt, q_groups = 1;
    } else {
        // Fewer may be of single tokens, each a run, or of prompts: shared out evenly.  (With groups of heads, as above, of whose
        // blocks many have no run, 256 single tokens of 8 heads, queries of 32, took 23.3 us for 15.6, a prompt of 700 18.6 for 9.5; now 14.4 and 8.1.)  Teams that are a whole
        // block do better with half of the threads (64 single tokens 7.9 -> 6.5), those of a warp with all (the ragged prompts 24.2 -> 21.4).
        const int tokens = std::min(p.T, kWindow), fill = ((C::TEAMS > 1 ? kAppendFill : kAppendFill / 2) / C::THREADS * num_sms + windows - 1) / windows;
        constexpr int at_once = C::THREADS / (D / 16);
        share = std::min(fill, (tokens * p.Hkv + C::TEAMS - 1) / C::TEAMS);
        if (p.q) q_tokens = std::min(fill, (tokens + at_once - 1) / at_once), q_groups = std::max(1, std::min(fill / q_tokens, p.Hkv * p.G));
    }
    const dim3 grid((unsigned)(windows * (2 * share + q_tokens * q_groups)), groups);
    const size_t smem = (size_t)C::TEAMS * PAGE * p.rot * 4;
    auto *const kernel = even ? (p.interleaved ? fa_kv_append_rope_kernel<D, PAGE, true, true> : fa_kv_append_rope_kernel<D, PAGE, false, true>)
                              : (p.interleaved ? fa_kv_append_rope_kernel<D, PAGE, true, false> : fa_kv_append_rope_kernel<D, PAGE, false, false>);
    if (smem + sizeof(AppendShared<D, PAGE, C>) > 48 * 1024) {  // beyond what a kernel may have without asking: always the most, as other threads' calls set it too
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::TEAMS * PAGE * D * 4);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, grid, C::THREADS, smem, stream, 1, p, share, per, q_tokens, q_groups);
}

template <int D>
static cudaError_t launch_append_rope_page(const AppendParams &p, int num_sms, cudaStream_t stream) {
    switch (p.page_log2) {
        case 4: return launch_append_rope<D, 16>(p, num_sms, stream);
        case 5: return launch_append_rope<D, 32>(p, num_sms, stream);
        case 6: return launch_append_rope<D, 64>(p, num_sms, stream);
        default: return launch_append_rope<D, 128>(p, num_sms, stream);
    }
}

cudaError_t launch_kv_append_rope(int D, const AppendParams &p, int num_sms, cudaStream_t stream) {
    return D == 64 ? launch_append_rope_page<64>(p, num_sms, stream) : launch_append_rope_page<128>(p, num_sms, stream);
}

cudaError_t kv_append_rope_status_read_and_clear(int *out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_kv_append_rope, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status_kv_append_rope, &zero, sizeof(int));
    *out = v;
    return e;
}

}  // namespace fa
