// fa_paged_chunk.cu -- attention of many new tokens a sequence (prompts, chunks of them)
// over the paged 8-bit cache on GB300 (sm_103a): O = softmax(scale q K^T) V and the row
// log-sum-exp, K and V read as e4m3 codes with one scale for each page and head.
//
// Mathematics.  The online softmax in base 2 (c = scale log2 e), over tiles of 128 keys from
// the last to the first:
//   p_rj = 2^(c q_r . k_j - m_r + 4),  O_r = sum_j p_rj v_j / l_r,  l_r = sum_j p_rj,
//   LSE_r = ln2 (m_r - 4 + log2 l_r),
// for any m_r.  m_r is the largest score of the row's first tile, and is taken again where a
// half tile's sum of p passes 2^15, so that p fits fp16 (no larger than 2^15, and rounded by half a step, 2^-11
// of itself, down to 2^-14; steps of 2^-24 below, 2^-28 of a weight at the maximum in use).
// k_j = code * scale in bf16, exactly where the scale is a power of two, beside q as it is.
// v_j = code * 2^(e_j - e) in fp16, e the largest exponent of the value scales in the first
// tile and e_j the page's, exact while |e_j - e| <= 5 (codes are 2^-9 to 448); O's sums are in
// units of 2^e.  A tile with a page further off, or with a scale that is no power of two, has both P
// and V in bf16, which has the range of fp32 (and rounds weights to 2^-8).
//
// What bounds it: 4 D operations for a row and a key on the tensor cores, with enough rows
// (256 rows share a tile of 128 keys: 2 D bytes a key for 1024 D operations); the conversion
// of the codes, which the tensor cores cannot read beside 16-bit queries, is 2 D elements a key
// and 256 rows.
//
// Roles of a block (one an SM, persistent):
//   warps 0-3, 4-7   softmax of row sub-tile 0 and 1 (128 rows each): S from tensor memory, P back
//                    over it, O out of it at the end;
//   warps 8-11       codes: read from global memory a tile ahead (in registers), converted, and
//                    written to shared memory in the layout that the MMAs read (128-byte swizzle);
//   warp 12          issues the MMAs, in the order S0_j, O1 += P1 V_{j+1}, S1_j, O0 += P0 V_j, so
//                    that one sub-tile's products run while the other's softmax does;
//   warp 13          the block's work, segment by segment, a ring of four ahead of the others;
//   warps 14-15      queries into shared memory.
//
// Split.  Items (sequence, key/value head, 256 rows) are laid end to end, each as long as its
// keys and a fixed cost, and the line is cut into equal shares, one a block.  What a block has of
// an item is a segment of its tiles.  An item that is cut leaves its parts (normalised sums, m, l)
// in the workspace, and a second kernel joins them in order.  Lengths are read on the device.
//
// Every wait is bounded in time; one that gives up records a status code and the block winds down.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_chunk = 0;

constexpr int kCkThreads = 512;
constexpr int kCkRows = 256;        // rows of an item, two sub-tiles of 128
constexpr int kCkTile = 128;        // keys a tile
constexpr int kCkFixed = 256;       // keys that an item's fixed cost stands for
constexpr int kCkMinShare = 768;    // of a block, in keys
constexpr int kCkSegs = 4;          // segments in the ring
constexpr float kCkShift = 4.f;     // exponent of a weight at the maximum in use
constexpr float kCkMost = 32768.f;  // of a half tile's sum
constexpr int kCkApart = 5;         // of value scales' exponents, beyond which a tile takes bf16
constexpr unsigned long long kCkDrainNs = 20ull * 1000 * 1000;
// Registers: 512 x 128 at launch; what the last four warps give goes to the others.
constexpr uint32_t kCkRegsSoftmax = 152, kCkRegsCodes = 136, kCkRegsOther = 72;
static_assert(256 * kCkRegsSoftmax + 128 * kCkRegsCodes + 128 * kCkRegsOther <= 512 * 128, "register split");

template <int D>
struct CkCfg {
    static constexpr int ST = D == 128 ? 2 : 3;               // stages of K and of V
    static constexpr uint32_t QT_BYTES = 128 * D * 2;         // a sub-tile's queries
    static constexpr uint32_t KV_BYTES = kCkTile * D * 2;
    static constexpr uint32_t CHUNK = 128 * 128;              // 128 rows x 128 bytes
    static constexpr uint32_t OFF_K = 2 * QT_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + ST * KV_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_V + ST * KV_BYTES;
    static constexpr uint32_t SMEM = OFF_BAR + 1024 + 1024;   // barriers and segments; alignment
    static constexpr uint32_t TM_O = 256;
    static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kCkTile, false);
    static constexpr uint32_t IDESC_PV_BF16 = idesc_bf16_f32(128, D, true);
    static constexpr uint32_t IDESC_PV = IDESC_PV_BF16 & ~((7u << 7) | (7u << 10));  // fp16 operands: format 0
    static constexpr int GROUP_LOADS = D / 32;                // 16-byte loads a lane for 16 keys
    static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_BAR % 1024 == 0, "atoms");
    static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one block an SM");
};

// barriers (8 bytes each) in the block's last kilobyte of shared memory
enum : uint32_t {
    C_Q_FULL = 0,    // + sub-tile
    C_Q_FREE = 2,
    C_K_FULL = 4,    // + stage (up to 3)
    C_K_EMPTY = 7,
    C_V_FULL = 10,
    C_V_EMPTY = 13,
    C_S_FULL = 16,   // + sub-tile
    C_P_HALF = 18,
    C_P_FULL = 20,
    C_PH_DONE = 22,
    C_O_DONE = 24,
    C_O_FREE = 26,
    C_SEG_FULL = 28,  // + ring place
    C_SEG_FREE = 32,
    C_DRAIN = 36,
    C_COUNT = 37
};
constexpr uint32_t kSlotTmem = 304, kSlotAbort = 308;
constexpr uint32_t kSlotWide = 320;   // 8 words: a tile's P and V are bf16 (by the tile's number)
constexpr uint32_t kSlotExp = 352;    // 4 words: e of a segment
constexpr uint32_t kSlotNan = 368;    // 4 words: number + 1 of a segment with NaN among masked tiles' values
constexpr uint32_t kSlotSegs = 384;   // 4 segments of 64 bytes
static_assert(C_COUNT * 8 <= kSlotTmem, "");

// What a block does of one item.
struct __align__(16) Seg {
    int q0, rows, row0, c;     // first token; rows of the (sequence, head); the item's first; keys before the step's tokens
    int b, h, len, t0;         // sequence, head, its keys; tiles [t0, t1)
    int t1, first[2], act1;    // load order (from t1 - 1 down) in which each sub-tile begins; whether there is a second one
    int slot, end, pad[2];     // partial result: -1 none (the item is whole), 0 begun before, 1 left off; no more work
};
static_assert(sizeof(Seg) == 64, "");

// ---------------------------------------------------------------- the line
struct CkSeq {
    int q0, nq, len;
};

__device__ __forceinline__ CkSeq ck_sequence(const ChunkParams &p, int b) {
    CkSeq s;
    s.q0 = max(0, min(p.cu_q[b], p.T));
    s.nq = max(s.q0, min(p.cu_q[b + 1], p.T)) - s.q0;
    s.len = max(0, min(p.seq_lens[b], p.max_len));
    return s;
}

// Where item i of a (sequence, head) begins in it, in keys: an item costs its fixed part, the
// keys before the step's tokens and those up to its last row's token (256 (i + 1) / G).
__device__ __forceinline__ long long ck_begin(const ChunkParams &p, long long i, int c) {
    return i * (kCkFixed + max(c, 0)) + 128 * i * (i + 1) / p.G;
}
__device__ __forceinline__ int ck_items(const ChunkParams &p, int nq) {
    return (int)(((long long)nq * p.G + kCkRows - 1) / kCkRows);
}
__device__ __forceinline__ long long ck_weight(const ChunkParams &p, int b) {
    const CkSeq s = ck_sequence(p, b);
    return ck_begin(p, ck_items(p, s.nq), s.len - s.nq) * p.Hkv;
}
// Tiles that the rows up to `last` see some of.
__device__ __forceinline__ int ck_tiles(const ChunkParams &p, int c, int last) {
    return max(0, c + last / p.G + 1 + kCkTile - 1) / kCkTile;
}

// An item and how many of its tiles lie before a cut.
struct Cut {
    int b, h, i, done;
    long long begin;   // where the item begins in the line; LLONG_MAX: behind the last one
};

// Moves a cut at the end of item i to the next item.
__device__ __forceinline__ void ck_next(const ChunkParams &p, Cut &u) {
    CkSeq s = ck_sequence(p, u.b);
    const int n = ck_items(p, s.nq), c = s.len - s.nq;
    u.begin += ck_begin(p, u.i + 1, c) - ck_begin(p, u.i, c);
    u.done = 0;
    if (++u.i < n) return;
    u.i = 0;
    if (++u.h < p.Hkv) return;
    u.h = 0;
    do {
        if (++u.b >= p.B) {
            u.begin = LLONG_MAX;
            return;
        }
        s = ck_sequence(p, u.b);
    } while (s.nq == 0);
}

// Tiles of the item (of `tiles`, at begin .. begin + w) that lie before place pos of the line.
__device__ __forceinline__ int ck_done(long long pos, long long begin, long long w, int tiles, long long share) {
    const long long in = pos - begin;
    if (in <= kCkFixed) return 0;
    // items of a small part of a share are not cut, nor those a little longer than one
    const bool whole = w <= share / 4 || tiles <= 3 || (w > share && w <= share + share / 3);
    if (whole) return 2 * in < w ? 0 : tiles;
    const int done = (int)((double)(in - kCkFixed) * tiles / (double)(w - kCkFixed) + 0.5);
    return done < 2 ? 0 : (done > tiles - 2 ? tiles : done);
}

// The cut at place pos, which lies in sequence b that begins at `base`.
__device__ Cut ck_cut(const ChunkParams &p, int b, long long base, long long pos, long long share) {
    const CkSeq s = ck_sequence(p, b);
    const int n = ck_items(p, s.nq), c = s.len - s.nq, rows = s.nq * p.G;
    const long long head = max(ck_begin(p, n, c), 1ll);
    Cut u;
    u.b = b;
    u.h = (int)min((pos - base) / head, (long long)p.Hkv - 1);
    const long long in = pos - base - u.h * head;
    int lo = 0, hi = max(n - 1, 0);  // the last item that begins at or before `in`
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ck_begin(p, mid, c) <= in)
            lo = mid;
        else
            hi = mid - 1;
    }
    u.i = lo;
    u.begin = base + u.h * head + ck_begin(p, lo, c);
    const long long w = ck_begin(p, lo + 1, c) - ck_begin(p, lo, c);
    const int tiles = ck_tiles(p, c, min(rows, (lo + 1) * kCkRows) - 1);
    u.done = ck_done(pos, u.begin, w, tiles, share);
    if (u.done >= tiles && pos > u.begin) ck_next(p, u);
    return u;
}

// ---------------------------------------------------------------- workspace
// For each block what the item that it leaves off needs to be joined, then two slots of
// partial results a block: [256][D] normalised sums, [256] m, [256] l.
struct __align__(16) CkTail {
    int parts, q0, rows, row0;   // parts 0: none.  Part 0 is slot 1 of this block, part j slot 0 of the j-th behind
    int h, pad[3];
};
__device__ __forceinline__ CkTail *ck_tail(float *ws, int block) { return reinterpret_cast<CkTail *>(ws) + block; }
__device__ __forceinline__ float *ck_slot(float *ws, int blocks, int block, int slot, int D) {
    return ws + (size_t)blocks * (sizeof(CkTail) / 4) + ((size_t)block * 2 + slot) * kCkRows * (D + 2);
}

// ------------------------------------------------------------- conversions
__device__ __forceinline__ uint32_t ck_codes_f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
// 16 codes times `scale`, in bf16
__device__ __forceinline__ void ck_bf16(const uint4 w, float scale, uint32_t (&y)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = ck_codes_f16x2(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        y[i] = pack_bf16x2(f.x * scale, f.y * scale);
    }
}
// 16 codes times a power of two (twice, in halves of a word), in fp16
__device__ __forceinline__ void ck_f16(const uint4 w, uint32_t scale2, uint32_t (&y)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = ck_codes_f16x2(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&scale2));
        y[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
}
__device__ __forceinline__ uint32_t ck_nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// NaN codes as 0; whether there were any
__device__ __forceinline__ bool ck_without_nan(uint4 &w) {
    uint32_t *const u[4] = {&w.x, &w.y, &w.z, &w.w};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t nan = ck_nan_codes(*u[i]);
        any |= nan;
        if (nan) *u[i] &= ~((nan >> 7) * 0xffu);
    }
    return any != 0;
}
__device__ __forceinline__ uint32_t ck_pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float ck_two_to(int e) { return __uint_as_float((uint32_t)(max(-126, min(127, e)) + 127) << 23); }

// Which columns of a row are NaN because a key that it sees in a masked tile has a NaN value there
// (the MMA had zeros in their place: another row may not see the key).  Rare.
template <int D>
__device__ __noinline__ void ck_nan_columns(const ChunkParams &p, const Seg *g, int limit, uint32_t *mask) {
    const int from = max(g->t0, max(0, g->c + g->row0 / p.G + 1) / kCkTile) * kCkTile, to = min(min(limit, g->len), g->t1 * kCkTile);
    for (int j = from; j < to; ++j) {
        const int pg = p.table[(long long)g->b * p.max_pages + (j >> p.page_log2)];
        if (pg < 0 || pg >= p.num_pages) continue;
        const unsigned long long row = ((unsigned long long)((uint32_t)pg * p.Hkv + g->h) << p.page_log2) + (j & ((1 << p.page_log2) - 1));
        const uint32_t *const v = reinterpret_cast<const uint32_t *>(p.v_pages + row * D);
#pragma unroll 1
        for (int i = 0; i < D / 4; ++i) {
            const uint32_t nan = ck_nan_codes(v[i]) >> 7;  // a bit a byte
            const uint32_t four = (nan & 1u) | (nan >> 7 & 2u) | (nan >> 14 & 4u) | (nan >> 21 & 8u);
            mask[i / 8] |= four << (i % 8 * 4);
        }
    }
}

__device__ __forceinline__ void ck_cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// --------------------------------------------------------------- the kernel
template <int D>
__global__ void __launch_bounds__(kCkThreads, 1) fa_fwd_paged_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using C = CkCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long scan_sm[kCkThreads / 32];
    __shared__ long long share_sm;
    __shared__ Cut cut_sm[2];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = sbase + C::OFF_BAR;
    auto bar = [&](uint32_t i) { return bars + 8u * i; };
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(gbase + C::OFF_BAR);
    volatile uint32_t *const abort_flag = words + kSlotAbort / 4;
    volatile uint32_t *const wide_of = words + kSlotWide / 4;
    volatile uint32_t *const exp_of = words + kSlotExp / 4;
    volatile uint32_t *const nan_of = words + kSlotNan / 4;
    Seg *const segs = reinterpret_cast<Seg *>(gbase + C::OFF_BAR + kSlotSegs);

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(C_Q_FULL + t), 2);     // a lane of each of two warps
            mbar_init(bar(C_Q_FREE + t), 1);
            mbar_init(bar(C_S_FULL + t), 1);
            mbar_init(bar(C_P_HALF + t), 128);
            mbar_init(bar(C_P_FULL + t), 128);
            mbar_init(bar(C_PH_DONE + t), 1);
            mbar_init(bar(C_O_DONE + t), 1);
            mbar_init(bar(C_O_FREE + t), 128);
        }
        for (int s = 0; s < C::ST; ++s) {
            mbar_init(bar(C_K_FULL + s), 4);     // a lane of each of four warps
            mbar_init(bar(C_K_EMPTY + s), 1);
            mbar_init(bar(C_V_FULL + s), 4);
            mbar_init(bar(C_V_EMPTY + s), 1);
        }
        for (int s = 0; s < kCkSegs; ++s) {
            mbar_init(bar(C_SEG_FULL + s), 1);
            mbar_init(bar(C_SEG_FREE + s), 15);  // 8 softmax, 4 codes, 1 MMA, 2 query warps
            nan_of[s] = 0;
        }
        mbar_init(bar(C_DRAIN), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(bars + kSlotTmem, 512);
        tmem_relinquish();
    }
    grid_wait();

    // ---- the line: a scan of the sequences' weights, and this block's two cuts
    {
        const int per = (p.B + kCkThreads - 1) / kCkThreads;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += ck_weight(p, b);
        long long x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) scan_sm[warp] = x;
        if (tid < 2) cut_sm[tid].begin = LLONG_MAX;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kCkThreads / 32; ++w) {
            if (w < warp) before += scan_sm[w];
            total += scan_sm[w];
        }
        const long long share = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)kCkMinShare);
        if (tid == 0) {
            share_sm = share;
            ck_tail(p.ws, blockIdx.x)->parts = 0;
        }
        const long long end = before + x, begin = end - mine;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const long long pos = ((long long)blockIdx.x + e) * share;
            if (pos < begin || pos >= end) continue;  // some other thread's, or behind the line
            long long base = begin;
            int b = b0;
            for (; b < b1 - 1; ++b) {
                const long long w = ck_weight(p, b);
                if (pos < base + w) break;
                base += w;
            }
            cut_sm[e] = ck_cut(p, b, base, pos, share);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = words[kSlotTmem / 4];
    const unsigned long long tlim = p.timeout_ns;
    auto wait = [&](uint32_t b, uint32_t parity) {
        return mbar_wait(bar(b), parity, abort_flag, tlim, &g_status_chunk, FA_ERR_TIMEOUT);
    };
    auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
    // segment n of the block, once it is there
    auto segment = [&](int n) { return wait_all(C_SEG_FULL + n % kCkSegs, (uint32_t)(n / kCkSegs) & 1u); };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C_SEG_FREE + n % kCkSegs));
    };

    if (warp >= 12) {
        regs_decrease<kCkRegsOther>();
        if (warp == 13) {
            // ================================================= segments
            Cut at = cut_sm[0];
            const Cut end = cut_sm[1];
            const long long share = share_sm;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int place = n % kCkSegs;
                if (n >= kCkSegs) ok = wait_all(C_SEG_FREE + place, (uint32_t)(n / kCkSegs - 1) & 1u);
                if (!ok) break;
                const bool more = at.begin < end.begin || (at.begin == end.begin && at.begin != LLONG_MAX && at.done < end.done);
                Seg g{};
                g.end = !more;
                if (more) {
                    const CkSeq s = ck_sequence(p, at.b);
                    g.q0 = s.q0;
                    g.rows = s.nq * p.G;
                    g.row0 = at.i * kCkRows;
                    g.c = s.len - s.nq;
                    g.b = at.b;
                    g.h = at.h;
                    g.len = s.len;
                    const int last = min(g.rows, g.row0 + kCkRows) - 1;
                    const int tiles = ck_tiles(p, g.c, last);
                    const int done1 = at.begin == end.begin ? min(end.done, tiles) : tiles;
                    g.t1 = tiles - at.done;
                    g.t0 = tiles - done1;
                    g.act1 = g.rows > g.row0 + 128;
                    const int see0 = ck_tiles(p, g.c, min(g.rows, g.row0 + 128) - 1);
                    g.first[0] = g.t1 - min(g.t1, see0);
                    g.first[1] = g.act1 ? 0 : g.t1 - g.t0;
                    g.slot = at.done > 0 ? 0 : (done1 < tiles ? 1 : -1);
                    if (g.slot == 1) {  // how many blocks have a part of it
                        const long long w = ck_begin(p, at.i + 1, g.c) - ck_begin(p, at.i, g.c);
                        int parts = 0;
                        for (int j0 = 1; parts == 0; j0 += 32) {
                            const int j = j0 + lane;  // the j-th block behind has its last part, if its end is not in it
                            const long long pos = ((long long)blockIdx.x + j + 1) * share;
                            const bool last_one = pos >= at.begin + w || (int)blockIdx.x + j + 1 >= (int)gridDim.x ||
                                                  ck_done(pos, at.begin, w, tiles, share) >= tiles;
                            const uint32_t some = __ballot_sync(0xffffffffu, last_one);
                            if (some) parts = j0 + __ffs((int)some);
                        }
                        if (lane == 0) {
                            CkTail tail{};
                            tail.parts = parts;
                            tail.q0 = g.q0;
                            tail.rows = g.rows;
                            tail.row0 = g.row0;
                            tail.h = g.h;
                            *ck_tail(p.ws, blockIdx.x) = tail;
                        }
                    }
                    if (at.begin == end.begin)
                        at = end;
                    else
                        ck_next(p, at);
                }
                if (lane == 0) {
                    segs[place] = g;
                    mbar_arrive(bar(C_SEG_FULL + place));
                }
                __syncwarp();
                if (!more) break;
            }
        } else if (warp >= 14) {
            // ================================================= queries
            int use[2] = {0, 0};
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = segment(n);
                if (!ok) break;
                const Seg *const g = segs + n % kCkSegs;
                const int q0 = g->q0, rows = g->rows, row0 = g->row0, h = g->h, N = g->t1 - g->t0, end = g->end;
                const int first[2] = {g->first[0], g->first[1]};
                release(n);
                if (end) break;
                for (int t = 0; t < 2; ++t) {
                    if (first[t] >= N) continue;  // the sub-tile sees none of the tiles
                    const int k = use[t]++;
                    if (k > 0) ok = wait_all(C_Q_FREE + t, (uint32_t)(k - 1) & 1u);
                    if (!ok) break;
                    constexpr int PIECES = D / 8;  // of 16 bytes, a row
#pragma unroll 4
                    for (int i = tid - 14 * 32; i < 128 * PIECES; i += 64) {
                        const int r = i / PIECES, piece = i % PIECES, R = row0 + t * 128 + r;
                        const int row = min(R, rows - 1), tok = row / p.G;
                        const __nv_bfloat16 *const src = static_cast<const __nv_bfloat16 *>(p.q) + (long long)(q0 + tok) * p.q_stride +
                                                         (long long)(h * p.G + row - tok * p.G) * D + piece * 8;
                        const uint32_t dst = sbase + t * C::QT_BYTES + (piece >> 3) * C::CHUNK + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                        ck_cp_async16(dst, src, R < rows ? 16 : 0);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C_Q_FULL + t));
                }
            }
        } else if (warp == 12) {
            // ================================================= MMA issuer
            const uint64_t dq = sw128_desc(sbase, 16, 1024);
            const uint64_t dk = sw128_desc(sbase + C::OFF_K, 16, 1024);
            const uint64_t dv = sw128_desc(sbase + C::OFF_V, C::CHUNK, 1024);
            int sk = 0, sv = 0;
            uint32_t kph = 0, vph = 0;
            int qn[2] = {0, 0}, npv[2] = {0, 0};
            int tile = 0;  // tiles so far, over all segments
            bool ok = true;
            auto issue_s = [&](int t, int stage) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4;
                    tc_mma_ss(tmem + t * 128, dq + ((t * C::QT_BYTES) >> 4) + off, dk + ((stage * C::KV_BYTES) >> 4) + off, C::IDESC_S,
                              kk > 0 ? 1u : 0u);
                }
            };
            auto issue_half = [&](int t, bool accumulate, int stage, uint32_t idesc, int k0) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_ts(tmem + C::TM_O + t * D, tmem + t * 128 + (k0 + kk) * 8,
                              dv + ((stage * C::KV_BYTES + (k0 + kk) * 16 * 128) >> 4), idesc, (accumulate || kk > 0) ? 1u : 0u);
            };
            for (int n = 0; ok; ++n) {
                ok = segment(n);
                if (!ok) break;
                const Seg *const g = segs + n % kCkSegs;
                const int N = g->t1 - g->t0, end = g->end, act1 = g->act1, first0 = g->first[0];
                release(n);
                if (end) break;
                bool begun0 = false, begun1 = false;
                // P_t V in two halves of 64 keys, the first as soon as the softmax has written it
                auto issue_pv = [&](int t, bool begun, int stage, uint32_t phase, int number) -> bool {
                    const uint32_t idesc = wide_of[number & 7] ? C::IDESC_PV_BF16 : C::IDESC_PV;
                    if (!wait_all(C_P_HALF + t, (uint32_t)npv[t] & 1u)) return false;
                    if (!wait_all(C_V_FULL + stage, phase)) return false;
                    if (!begun && qn[t] > 0 && !wait_all(C_O_FREE + t, (uint32_t)(qn[t] - 1) & 1u)) return false;
                    tc_fence_after();
                    issue_half(t, begun, stage, idesc, 0);
                    tc_commit(bar(C_PH_DONE + t));
                    if (!wait_all(C_P_FULL + t, (uint32_t)npv[t] & 1u)) return false;
                    tc_fence_after();
                    issue_half(t, true, stage, idesc, 4);
                    ++npv[t];
                    return true;
                };
                int svp = 0;
                uint32_t vpph = 0;
                for (int it = 0; it < N; ++it, ++tile) {
                    ok = wait_all(C_K_FULL + sk, kph);
                    if (!ok) break;
                    const bool p0 = it >= first0, p1 = act1 != 0;
                    if (p0) {
                        if (it == first0) {
                            ok = wait_all(C_Q_FULL + 0, (uint32_t)qn[0] & 1u);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        issue_s(0, sk);
                        tc_commit(bar(C_S_FULL + 0));
                        if (it == N - 1) tc_commit(bar(C_Q_FREE + 0));
                    }
                    if (p1 && it > 0) {
                        ok = issue_pv(1, begun1, svp, vpph, tile - 1);
                        begun1 = true;
                        if (!ok) break;
                        tc_commit(bar(C_V_EMPTY + svp));
                    }
                    if (p1) {
                        if (it == 0) {
                            ok = wait_all(C_Q_FULL + 1, (uint32_t)qn[1] & 1u);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        issue_s(1, sk);
                        tc_commit(bar(C_S_FULL + 1));
                        if (it == N - 1) tc_commit(bar(C_Q_FREE + 1));
                    }
                    tc_commit(bar(C_K_EMPTY + sk));
                    if (p0) {
                        ok = issue_pv(0, begun0, sv, vph, tile);
                        begun0 = true;
                        if (!ok) break;
                        if (it == N - 1) tc_commit(bar(C_O_DONE + 0));
                        if (!p1) tc_commit(bar(C_V_EMPTY + sv));
                    }
                    if (++sk == C::ST) sk = 0, kph ^= 1u;
                    svp = sv;
                    vpph = vph;
                    if (++sv == C::ST) sv = 0, vph ^= 1u;
                }
                if (!ok) break;
                if (act1 && N > 0) {
                    ok = issue_pv(1, begun1, svp, vpph, tile - 1);
                    if (!ok) break;
                    tc_commit(bar(C_O_DONE + 1));
                    tc_commit(bar(C_V_EMPTY + svp));
                }
                if (first0 < N) ++qn[0];
                if (act1 && N > 0) ++qn[1];
            }
            tc_commit(bar(C_DRAIN));
            mbar_wait_drain(bar(C_DRAIN), 0, kCkDrainNs);
        }
    } else if (warp >= 8) {
        // ===================================================== codes
        regs_increase<kCkRegsCodes>();
        const int cw = warp - 8;  // takes the tile's keys 32 cw .. 32 cw + 31: two groups of 16, each in one page
        // A load's lanes: pairs of rows in which eight lanes cover the same 64 columns (four
        // pieces of 16 codes), so that what they write falls into different banks.
        const int ld_row = 2 * (D == 128 ? lane >> 4 : lane >> 3) + ((lane >> 2) & 1);
        const int ld_piece = (lane & 3) + (D == 128 ? (lane >> 3 & 1) * 4 : 0);
        constexpr int LD_ROWS = D == 128 ? 4 : 8;
        struct Tile {   // of the sequence of tiles over all segments
            int seg, key0, len, edge, first;  // edge: keys that the item's first row sees; first tile of a segment
        };
        int seg_next = 0, it_next = 0;
        Tile cur{}, nxt{};
        bool ok = true;
        int seg_n = 0, seg_t1 = 0, seg_len = 0, seg_edge = 0, seg_b = 0, seg_h = 0;
        // The next tile, and this lane's group of it (lanes 0-7): its entry of the block table.  Where the
        // tile's segment is not there yet: to be asked again, or waited for.  (Only once all tiles
        // before it are handed over: a segment's place in the ring is free when the softmax is
        // through with the one four before it, and segments without tiles lie between.)
        int pg_look = -2;  // -2: no keys there
        Tile look{};
        int h_look = 0;
        bool looked = false, end = false;
        auto look_up = [&](bool may_wait) {
            if (looked || end) return;
            while (it_next == seg_n) {
                if (may_wait)
                    ok = segment(seg_next);
                else if (!__all_sync(0xffffffffu, mbar_try_wait(bar(C_SEG_FULL + seg_next % kCkSegs), (uint32_t)(seg_next / kCkSegs) & 1u)))
                    return;
                if (!ok) return;
                const Seg *const g = segs + seg_next % kCkSegs;
                if (g->end) {
                    release(seg_next);
                    end = true;
                    return;
                }
                seg_n = g->t1 - g->t0;
                seg_t1 = g->t1;
                seg_len = g->len;
                seg_edge = g->c + g->row0 / p.G + 1;
                seg_b = g->b;
                seg_h = g->h;
                release(seg_next);
                ++seg_next;
                it_next = 0;
            }
            look.seg = seg_next - 1;
            look.key0 = (seg_t1 - 1 - it_next) * kCkTile;
            look.len = seg_len;
            look.edge = seg_edge;
            look.first = it_next == 0;
            h_look = seg_h;
            ++it_next;
            const int key = look.key0 + 16 * (lane & 7);
            pg_look = -2;
            if (key < look.len) pg_look = p.table[(long long)seg_b * p.max_pages + (key >> p.page_log2)];
            looked = true;
        };
        // what is known of a tile whose codes are being read: per lane (0-7) its group's page
        struct Meta {
            int ph;          // page * Hkv + head; -1: outside the cache, -2: no keys
            float ks, vs;
        };
        auto resolve = [&]() {
            Meta m{-2, 1.f, 1.f};
            if (pg_look != -2) {
                const bool good = pg_look >= 0 && pg_look < p.num_pages;
                m.ph = good ? pg_look * p.Hkv + h_look : -1;
                if (good) {
                    m.ks = __ldg(p.k_scale + m.ph);
                    m.vs = __ldg(p.v_scale + m.ph);
                } else {
                    atomicExch(&g_status_chunk, (int)FA_ERR_BAD_PAGE);
                }
            }
            return m;
        };
        uint4 kr[2 * C::GROUP_LOADS], vr[2 * C::GROUP_LOADS];
        const int page_mask = (1 << p.page_log2) - 1;
        auto load = [&](const uint8_t *pages, const Tile &x, const Meta &m, uint4 (&r)[2 * C::GROUP_LOADS]) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int key = x.key0 + 16 * (2 * cw + g);
                const int ph = __shfl_sync(0xffffffffu, m.ph, 2 * cw + g);
                const unsigned long long row = ((unsigned long long)(uint32_t)max(ph, 0) << p.page_log2) + (key & page_mask);
                const uint8_t *const src = pages + (row + ld_row) * D + ld_piece * 16;
#pragma unroll
                for (int i = 0; i < C::GROUP_LOADS; ++i) {
                    r[g * C::GROUP_LOADS + i] = make_uint4(0, 0, 0, 0);
                    if (ph >= 0 && key + i * LD_ROWS + ld_row < x.len)
                        r[g * C::GROUP_LOADS + i] = __ldg(reinterpret_cast<const uint4 *>(src + i * LD_ROWS * D));
                }
            }
        };
        auto store = [&](uint32_t base, int g, int i, const uint32_t (&y)[8]) {
            const int r = 16 * (2 * cw + g) + i * LD_ROWS + ld_row;
            const uint32_t at = base + (ld_piece >> 2) * C::CHUNK + r * 128, piece = 2 * (ld_piece & 3), sw = r & 7;
            st_shared_v4(at + ((piece ^ sw) << 4), y[0], y[1], y[2], y[3]);
            st_shared_v4(at + (((piece + 1) ^ sw) << 4), y[4], y[5], y[6], y[7]);
        };
        Meta m_cur{-2, 1.f, 1.f}, m_nxt{-2, 1.f, 1.f};
        look_up(true);
        bool have = looked;
        if (have) {
            looked = false;
            cur = look;
            m_cur = resolve();
            load(p.k_pages, cur, m_cur, kr);
            look_up(false);
        }
        int e_ref = 0;
        for (int n = 0; ok && have; ++n) {
            // ---- which operands the tile's second product takes (all four warps find the same)
            const uint32_t vu = __float_as_uint(m_cur.vs);
            const int e = (int)(vu >> 23 & 0xffu) - 127;
            const bool there = lane < 8 && m_cur.ph >= 0;
            if (cur.first) {
                const int top = __reduce_max_sync(0xffffffffu, there ? e : -1000);
                e_ref = top == -1000 ? 0 : top;
            }
            const bool wide = __any_sync(0xffffffffu, there && ((vu & 0x7fffffu) != 0 || e - e_ref > kCkApart || e_ref - e > kCkApart));
            if (cw == 0 && lane == 0) {
                wide_of[n & 7] = wide;
                if (cur.first) exp_of[cur.seg % kCkSegs] = (uint32_t)e_ref;
            }
            // ---- K of the tile
            const int st = n % C::ST;
            const uint32_t use = (uint32_t)(n / C::ST) & 1u;
            if (n >= C::ST) ok = wait_all(C_K_EMPTY + st, use ^ 1u);
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float ks = __shfl_sync(0xffffffffu, m_cur.ks, 2 * cw + g);
                const bool bad = __shfl_sync(0xffffffffu, m_cur.ph, 2 * cw + g) == -1;
#pragma unroll
                for (int i = 0; i < C::GROUP_LOADS; ++i) {
                    uint32_t y[8];
                    ck_bf16(kr[g * C::GROUP_LOADS + i], bad ? __uint_as_float(0x7fc00000u) : ks, y);
                    store(sbase + C::OFF_K + st * C::KV_BYTES, g, i, y);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_K_FULL + st));
            // ---- what comes next is asked for: this tile's V, the next one's K, and pages behind it
            load(p.v_pages, cur, m_cur, vr);
            auto go_on = [&]() {
                if (!looked) return false;
                looked = false;
                nxt = look;
                m_nxt = resolve();
                load(p.k_pages, nxt, m_nxt, kr);
                look_up(false);
                return true;
            };
            bool more = go_on();
            // ---- V of the tile
            if (n >= C::ST) ok = wait_all(C_V_EMPTY + st, use ^ 1u);
            if (!ok) break;
            const bool masked = cur.key0 + kCkTile > cur.edge;  // a row does not see some of its keys: their NaN must not reach it
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float vs = __shfl_sync(0xffffffffu, m_cur.vs, 2 * cw + g);
                const int de = (int)(__float_as_uint(vs) >> 23 & 0xffu) - 127 - e_ref;
                const uint32_t f16 = (uint32_t)(max(-14, min(15, de)) + 15) << 10, two = f16 | f16 << 16;  // 2^de
                const float f32 = vs * ck_two_to(-e_ref);
#pragma unroll
                for (int i = 0; i < C::GROUP_LOADS; ++i) {
                    uint4 w = vr[g * C::GROUP_LOADS + i];
                    if (masked && ck_without_nan(w)) nan_of[cur.seg % kCkSegs] = (uint32_t)cur.seg + 1u;
                    uint32_t y[8];
                    if (wide)
                        ck_bf16(w, f32, y);
                    else
                        ck_f16(w, two, y);
                    store(sbase + C::OFF_V + st * C::KV_BYTES, g, i, y);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_V_FULL + st));
            if (!more) {
                look_up(true);
                if (!ok) break;
                more = go_on();
            }
            cur = nxt;
            m_cur = m_nxt;
            have = more;
        }
    } else {
        // ============================================ softmax warpgroups
        regs_increase<kCkRegsSoftmax>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lane_off + t * 128;
        const uint32_t o_tm = tmem + lane_off + C::TM_O + t * D;
        const float sl2 = p.scale_log2;
        const uint64_t c2 = f2_pack(sl2, sl2);
        int ns = 0, od = 0, tile = 0;  // S tiles and items of this sub-tile, tiles of the block so far
        bool ok = true;
        for (int n = 0; ok; ++n) {
            ok = segment(n);
            if (!ok) break;
            const Seg *const g = segs + n % kCkSegs;  // (released behind the epilogue, which reads it again)
            if (g->end) {
                release(n);
                break;
            }
            const int N = g->t1 - g->t0, first = t ? g->first[1] : g->first[0];
            if (t == 1 && !g->act1) {
                tile += N;
                release(n);
                continue;
            }
            const int limit = g->c + min(g->row0 + t * 128 + row, g->rows - 1) / p.G + 1;  // keys that this row sees
            const int edge = g->c + (g->row0 + t * 128) / p.G + 1;                         // and the sub-tile's first row
            const int key1 = g->t1 * kCkTile;
            tile += min(first, N);
            float m_used = -INFINITY, l_run = 0.f;
            for (int it = first; it < N; ++it, ++tile) {
                ok = wait_all(C_S_FULL + t, (uint32_t)ns & 1u);
                if (!ok) break;
                ++ns;
                tc_fence_after();
                const bool wide = wide_of[tile & 7] != 0;
                const int col0 = key1 - (it + 1) * kCkTile;
                const bool masked = col0 + kCkTile > edge;
                const int lim = limit - col0;
                // S goes through the registers 32 keys at a time, the next 32 on their way
                uint32_t s[2][32];
                auto mask32 = [&](uint32_t (&x)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= lim) x[e] = __float_as_uint(-INFINITY);
                };
                auto scale_o = [&](float f) {
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(o_tm + c * 16, o);
                        tmem_ld_wait16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(o_tm + c * 16, o);
                        tmem_st_wait16(o);
                    }
                };
                // the largest of m_used and the scores of chunks [cb, 4)
                auto max_from = [&](int cb) {
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = cb; c < 4; ++c) {
                        tmem_ld32(s_tm + c * 32, s[0]);
                        tmem_ld_wait(s[0]);
                        if (masked) mask32(s[0], c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mq[q] = max3f(mq[q], __uint_as_float(s[0][e + 2 * q]), __uint_as_float(s[0][e + 2 * q + 1]));
                    }
                    return fmaxf(m_used, max3f(mq[0], mq[1], fmaxf(mq[2], mq[3])) * sl2);
                };
                // the factor of what was summed so far when the maximum becomes m_new
                auto raise = [&](float m_new) {
                    const float f = m_new == -INFINITY ? 1.f : ex2_approx(m_used - m_new);  // 0 on a row's first keys
                    m_used = m_new;
                    return f;
                };
                uint32_t pk[32];
                // p of chunks cb and cb + 1, of which the first is already being loaded; returns their sum
                auto exp_half = [&](int cb) -> float {
                    const float nm = m_used == -INFINITY ? 0.f : kCkShift - m_used;  // no key yet: p = 0
                    const uint64_t nm2 = f2_pack(nm, nm);
                    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld_wait(s[c]);
                        if (cb + c < 3) tmem_ld32(s_tm + (cb + c + 1) * 32, s[c ^ 1]);
                        if (masked) mask32(s[c], cb + c);
                        if (wide) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), c2, nm2), x0, x1);
                                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                                acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
                                pk[c * 16 + e] = pack_bf16x2(p0, p1);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), c2, nm2), x0, x1);
                                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                                acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
                                pk[c * 16 + e] = ck_pack_f16(p0, p1);
                            }
                        }
                    }
                    float a0, a1, b0, b1;
                    f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
                    f2_unpack(f2_add(acc[2], acc[3]), b0, b1);
                    return (a0 + a1) + (b0 + b1);
                };
                auto store_half = [&](int half) {
                    tmem_st16(s_tm + half * 32, pk);
                    tmem_st16(s_tm + half * 32 + 16, pk + 16);
                    tmem_st_wait(pk);
                    tc_fence_before();
                };
                const bool took_max = __any_sync(0xffffffffu, m_used == -INFINITY);
                float alpha = 1.f, beta = 1.f;
                if (took_max) alpha = raise(max_from(0));
                tmem_ld32(s_tm, s[0]);
                float sa = exp_half(0);
                const bool redo = !took_max && __any_sync(0xffffffffu, !(sa <= kCkMost));
                if (redo) {  // nothing of this tile is handed over yet: its true maximum
                    tmem_ld_wait(s[0]);
                    alpha = raise(max_from(0));
                    tmem_ld32(s_tm, s[0]);
                    sa = exp_half(0);
                }
                if (it > first && (redo || took_max)) scale_o(alpha);  // O holds earlier tiles at the old maximum
                tmem_ld_wait(s[0]);  // (S of chunk 2: P may overwrite chunks 0 and 1, which are read)
                store_half(0);
                mbar_arrive(bar(C_P_HALF + t));
                float sb = exp_half(2);
                if (!took_max && !redo && __any_sync(0xffffffffu, !(sb <= kCkMost))) {
                    // the first half's product must be in O before O is rescaled
                    ok = wait_all(C_PH_DONE + t, (uint32_t)(ns - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    beta = raise(max_from(2));  // chunks 2 and 3 are still there: P is in columns 0-31
                    scale_o(beta);
                    tmem_ld32(s_tm + 64, s[0]);
                    sb = exp_half(2);
                }
                store_half(1);
                l_run = (l_run * alpha + sa) * beta + sb;
                mbar_arrive(bar(C_P_FULL + t));
            }
            if (!ok) break;
            // ---- the rows' results, 32 columns at a time
            const bool some = first < N;  // the sub-tile has tiles here
            float unit = 1.f;
            uint32_t nan_mask[4] = {0, 0, 0, 0};
            bool nan_there = false;
            if (some) {
                ok = wait_all(C_O_DONE + t, (uint32_t)od & 1u);
                if (!ok) break;
                ++od;
                tc_fence_after();
                unit = ck_two_to((int)exp_of[n % kCkSegs]);
                nan_there = nan_of[n % kCkSegs] == (uint32_t)n + 1u;
                if (nan_there) ck_nan_columns<D>(p, g, limit, nan_mask);
            }
            const int R = g->row0 + t * 128 + row, slot = g->slot;
            const bool there = R < g->rows, empty = l_run == 0.f;  // empty: no key
            const float inv = empty ? 0.f : 1.f / l_run;
            const int tok = min(R, g->rows - 1) / p.G;
            const long long at = (long long)(g->q0 + tok) * (p.Hkv * p.G) + g->h * p.G + (R - tok * p.G);
            float *const part = ck_slot(p.ws, gridDim.x, blockIdx.x, max(slot, 0), D);
            const int r = t * 128 + row;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (some) {
                    tmem_ld32(o_tm + c * 32, o);
                    tmem_ld_wait(o);
                }
                const uint32_t nan = nan_there ? (c == 0 ? nan_mask[0] : c == 1 ? nan_mask[1] : c == 2 ? nan_mask[2] : nan_mask[3]) : 0u;
                if (!there) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float x = __uint_as_float(o[e]) * inv * unit;
                    o[e] = empty ? 0u : (nan >> e & 1u) ? 0x7fc00000u : __float_as_uint(x);
                }
                if (slot < 0) {
                    uint4 *const dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + at * D + c * 32);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(o[u * 8 + 2 * e]), __uint_as_float(o[u * 8 + 2 * e + 1]));
                        dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *const dst = reinterpret_cast<uint4 *>(part + (size_t)r * D + c * 32);
#pragma unroll
                    for (int u = 0; u < 8; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                }
            }
            if (some) {
                tc_fence_before();
                mbar_arrive(bar(C_O_FREE + t));
            }
            if (there) {
                if (slot < 0) {
                    p.lse[at] = empty ? -INFINITY : ((m_used - kCkShift) + log2f(l_run)) * 0.69314718055994531f;
                } else {
                    part[(size_t)kCkRows * D + r] = m_used;
                    part[(size_t)kCkRows * (D + 1) + r] = l_run;
                }
            }
            release(n);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- the join
// O = sum_s w_s o_s / sum_s w_s with w_s = l_s 2^(m_s - max m), LSE = ln2 (max m - 4 + log2 sum_s w_s), the
// parts in order: a warp a row, D / 32 columns a lane.
constexpr int kCkJoinRows = 8;
template <int D>
__global__ void __launch_bounds__(32 * kCkJoinRows) fa_fwd_paged_chunk_join(const __grid_constant__ ChunkParams p) {
    grid_wait();
    const CkTail tail = *ck_tail(p.ws, blockIdx.x);
    const int r = blockIdx.y * kCkJoinRows + (threadIdx.x >> 5), lane = threadIdx.x & 31, row = tail.row0 + r;
    if (tail.parts == 0 || row >= tail.rows) return;
    auto part = [&](int j) { return ck_slot(p.ws, gridDim.x, (int)blockIdx.x + j, j == 0 ? 1 : 0, D); };
    float top = -INFINITY;
    for (int j = lane; j < tail.parts; j += 32) {
        const float *const s = part(j);
        if (s[(size_t)kCkRows * (D + 1) + r] != 0.f) top = fmaxf(top, s[(size_t)kCkRows * D + r]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    constexpr int PER = D / 32;
    float acc[PER] = {}, sum = 0.f;
#pragma unroll 2
    for (int j = 0; j < tail.parts; ++j) {
        const float *const s = part(j);
        const float l = s[(size_t)kCkRows * (D + 1) + r], m = s[(size_t)kCkRows * D + r];
        if (l == 0.f) continue;
        const float w = l * exp2f(m == top ? 0.f : m - top);
        sum += w;
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] = fmaf(w, s[(size_t)r * D + lane * PER + c], acc[c]);
    }
    const int tok = row / p.G;
    const long long at = (long long)(tail.q0 + tok) * (p.Hkv * p.G) + tail.h * p.G + (row - tok * p.G);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t *const dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + at * D) + lane * (PER / 2);
#pragma unroll
    for (int c = 0; c < PER / 2; ++c) dst[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    if (lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : ((top - kCkShift) + log2f(sum)) * 0.69314718055994531f;
}

size_t paged_chunk_workspace_bytes(int D, int num_sms) {
    return (size_t)num_sms * (sizeof(CkTail) + 2 * (size_t)kCkRows * (D + 2) * sizeof(float));
}

template <int D>
static cudaError_t launch_chunk(const ChunkParams &p, int num_sms, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(fa_fwd_paged_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CkCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_early(fa_fwd_paged_chunk_kernel<D>, dim3((unsigned)num_sms), kCkThreads, CkCfg<D>::SMEM, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_early(fa_fwd_paged_chunk_join<D>, dim3((unsigned)num_sms, kCkRows / kCkJoinRows), 32 * kCkJoinRows, 0, stream, 1, p);
}

cudaError_t launch_fwd_paged_chunk(int D, ChunkParams p, int num_sms, cudaStream_t stream) {
    p.max_len = p.max_pages << p.page_log2;
    return D == 64 ? launch_chunk<64>(p, num_sms, stream) : launch_chunk<128>(p, num_sms, stream);
}

cudaError_t paged_chunk_status_read_and_clear(int *out) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_chunk, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_status_chunk, &zero, sizeof(int));
    *out = v;
    return e;
}

}  // namespace fa
