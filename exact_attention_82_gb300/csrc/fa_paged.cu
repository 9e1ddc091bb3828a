// fa_paged.cu -- attention of a few query tokens over the paged 8-bit cache
// on GB300 (sm_103a): O = softmax(scale q K^T) V and the row log-sum-exp, K and
// V read as e4m3 codes with one scale for each page and head.
//
// Mathematics.  For a query row r and key j with codes k_j, v_j and their pages'
// scales ks_j, vs_j, in base 2 (c = scale log2 e):
//   x_rj = c ks_j (q_r . k_j) + log2 vs_j,
//   w_rj = 2^(x_rj - m_r + 8)                    (the weight of the CODES v_j)
//   O_r  = sum_j w_rj v_j / l_r,   l_r = sum_j w_rj / vs_j  (kept as 2^-12 of it),
//   LSE_r = ln2 (m_r - 8 + log2 l_r),
// for any m_r.  m_r is the largest x_rj so far when it was last taken, rounded down to a
// whole number (sums are then scaled exactly, and x - m loses nothing to a value scale's large
// logarithm), and is taken again when some x_rj exceeds it by more than 7, so w is at most 2^15 however
// unevenly the pages are scaled and can be rounded to fp16 (to 2^-11 of each; bf16 would
// keep three bits less).  fp16's subnormal numbers end at 2^-24, which is 2^-32 of the largest
// 2^x so far.  That may be a key's whose values are 0, for a page of zeros has scale 1, so
// where a page's value scale is below 2^-4 of the largest before it (or beside it), its
// 16 keys are a block of their own: weights rounded against their own maximum, and the sums scaled
// to m_r in fp32.  So no softmax weight is off by more than 2^-11 of itself and 2^-29 of the
// row's largest.  l sums the unrounded weights in fp32.  e4m3 codes are exact
// in fp16, and a query row is scaled by a power of two to a largest element in
// [1, 2), so that its bf16 values are exact too: both products run on fp16 operands
// with fp32 accumulators, and nothing but w and O is rounded.
//
// What bounds it: 2 D bytes read for a key and key/value head and 2 FLOP a byte
// for each query row, so for a few rows (grouped heads, drafts) the HBM stream.
// The products are computed transposed, S^T = K Q^T and O^T = V^T W^T, so that
// the long side of the MMA tile (16) lies along the keys or the head dimension
// and the short one (8) along the few query rows.  Each warp streams its own
// tiles of 32 keys through a private ring of asynchronous copies and keeps its own
// running maximum and sums: nothing waits for another warp before the end of an
// item.  tcgen05's tiles would lie the same way, 128 keys or D by 8 or more rows, but
// take their operands from shared memory: codes converted to fp16 would be written
// back there (its 8-bit kinds take them as they are, and would need queries and weights
// as several 8-bit terms), and scores and weights would pass through TMEM and shared memory
// between the products.  Up to 8 rows there is nothing to gain, the stream runs at the copy
// rate; beyond, where this kernel is bound by its own instructions, it is not built.
//
// Split.  The tiles of all items (sequence, key/value head, 8 to 32 query rows)
// are laid end to end, each item behind a few places that stand for its fixed
// cost, and the line is cut into equal shares, one a block (an SM), and each of
// them again into equal ones, one a warp, whatever the lengths: a long sequence is
// cut over many warps, short ones follow one another in one (small items are not cut
// at all).  Lengths are read on the device (a scan of a few hundred integers).  A
// warp's ring runs on across its items, so that the next one's keys arrive while it
// writes out the last one's rows.  What a block's warps have of an item is joined
// within the block, in shared memory; an item that crosses blocks leaves one partial
// result a block in the workspace, which a second kernel joins.
//
// Measured (back to back, other inputs in turn, of 6,705 GB/s that a copy reaches): 8 sequences
// of 65536 keys, 8 of 32 heads, D = 128, 162 us, 6,600 GB/s; of 16384 keys 49.5 us, 81% of the copy rate;
// with 16 query rows 59 us; at D = 64 87 us for 65536; 64 ragged sequences of 50 to 8000 keys 42.8 us.
// What a call takes without the stream: 8.3 us for one sequence of 32 keys (two launches, lengths and
// shares 2.5, one tile, the stores), 9.6 for one tile on every SM, 13.4 for one of 1000 keys and 32
// heads, whose items are joined.  Beyond 8 rows it is bound by its own instructions: 16 sequences with
// 16 to 40 rows each 75 us, 30.7 at the copy rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_paged = 0;

constexpr int kPgTile = 32;         // keys a tile; two halves of 16, each in one page
constexpr int kPgFixed = 2;         // places of the line that an item's fixed cost takes
constexpr int kPgMinShare = 36;     // places of a block: three tiles a warp
// An item of an eighth of a share is not cut (16 sequences of 2000 to 16000 keys with 2 to 5
// tokens: 84 us with half a share, whose blocks have up to one and a half of it, 73 with a quarter,
// 74.5 with an eighth; 64 ragged sequences 44.2, 43.6 and 42.6), nor is one of 8 places (256 sequences
// of 100 keys: 24.4 us without this, 21.2 with it).  What is not cut between warps must not be between blocks: else a warp's end
// could be moved past its block's.
constexpr int kPgSmall = 8;
constexpr int kPgWhole = 8;
constexpr int kPgMaxLen = 0x7fffff00;
constexpr float kPgShift = 8.f;    // exponent of a weight at x = m
constexpr float kPgMost = 15.f;    // and the largest one
constexpr float kPgNone = -3e38f;  // m before any key
// What l is kept scaled by, 2^-12: beside the smallest value scale of 2^-100 a weight of 2^15 adds 2^115 to
// it, and 8192 keys would pass the largest float; now 2^25 (2^32 of a weight of 2^8).  At the other end, 2^120, l is
// still 2^-124 or more.
constexpr float kPgDown = 12.f;
// log2 of how far value scales may lie apart before weights are rounded apart (see above).  Scales of pages
// that hold like values differ by 1 or 2.  Where one page in 64 is zeros beside small values, 8 sequences of 16384
// keys take 50.4 us for 49.6, drafts of 16 to 40 rows 92 for 75; every second page 51.1 and 85.
constexpr float kPgApart = 4.f;

template <int D, int NT>
struct PgCfg {
    static constexpr int CHUNKS = D / 16;                    // 16-byte pieces of a row
    static constexpr int HALF_BYTES = 16 * D;                // 16 rows of K or of V
    static constexpr int STAGE_BYTES = 4 * HALF_BYTES;       // K and V of a tile
    static constexpr int WARPS = NT == 1 ? 12 : 8;           // one block an SM
    static constexpr int THREADS = 32 * WARPS;
    // Beside 32 rows the registers are full of sums, and the query fragments lie in shared
    // memory, each lane's apart (D / 2 KB of about 200; the ring has the rest).
    static constexpr bool Q_SHARED = NT > 2;
    static constexpr int ST = D == 128 ? (NT == 2 ? 3 : 2) : (NT == 1 ? 4 : NT == 2 ? 6 : 5);  // stages a warp
    static constexpr int OFF_META = WARPS * ST * STAGE_BYTES;  // 2 float4 a stage
    static constexpr int OFF_WORK = OFF_META + WARPS * ST * 2 * 16;
    static constexpr int WORKS = 8;                          // items looked up ahead: ST + 1 at most
    static constexpr int OFF_SUMS = OFF_WORK + WARPS * WORKS * 48;
    static constexpr int OFF_Q = (OFF_SUMS + THREADS * 4 + 127) / 128 * 128;
    static constexpr int SMEM = OFF_Q + (Q_SHARED ? WARPS * 8 * NT * D * 2 : 0);
    // Where a 16-byte piece of a row lies: pieces are swapped within 128 bytes so that
    // eight rows' same piece (ldmatrix) falls into different banks, and so do pieces 0 to 3
    // of two neighbouring rows (16-byte loads).
    static __device__ __forceinline__ int swap(int row) {
        return D == 128 ? (row & 2) | ((row & 1) << 2) | ((row >> 2) & 1) : (row >> 1) & 3;
    }
    // The key of MMA row g of a half; row g + 8 has the key 2 further.  In this order the
    // weights that the transposition leaves a lane are those of the four keys 4t .. 4t+3,
    // whose values ldmatrix leaves it in one register.
    static __device__ __forceinline__ int key_of(int g) { return 4 * (g >> 1) + (g & 1); }
};

// A place in the line of tiles (32 bits: the caller has checked that they do).
struct Place {
    int entry;   // sequence, or sequence * Hkv + head where pages are selected
    int base;    // first place of the entry
    int pos;
};

struct Seq {
    int q0, nq, len;
};

// What of the parameters says how the work is laid out, for shared memory: an out of line
// function that is given the parameters themselves reads them as if from global memory
// (work_at before the first copy took 1930 cycles so, and takes 1200).
struct Layout {
    const int *cu_q, *seq_lens, *sel, *sel_count;
    int B, T, G, Hkv, sel_width, page_log2, max_len;
};

template <class P>
__device__ __forceinline__ Seq sequence(const P &p, int b) {
    Seq s;
    s.q0 = max(0, min(p.cu_q[b], p.T));
    s.nq = max(s.q0, min(p.cu_q[b + 1], p.T)) - s.q0;
    s.len = max(0, min(p.seq_lens[b], p.max_len));
    return s;
}

// Tiles of one item of (b, h), at least one: an item without keys still writes its rows.
template <class P>
__device__ __forceinline__ int item_tiles(const P &p, int b, int h, int len) {
    int keys = len;
    if (p.sel) keys = max(0, min(p.sel_count[(long long)b * p.Hkv + h], p.sel_width)) << p.page_log2;
    return max(1, (int)((uint32_t)(keys + kPgTile - 1) / kPgTile));
}

template <int NR, class P>
__device__ __forceinline__ int entry_weight(const P &p, int e) {
    const int b = p.sel ? e / p.Hkv : e, h = p.sel ? e % p.Hkv : 0;
    const Seq s = sequence(p, b);
    const int rt = (uint32_t)(s.nq * p.G + NR - 1) / NR;
    return rt * (p.sel ? 1 : p.Hkv) * (kPgFixed + item_tiles(p, b, h, s.len));
}

// The place of `pos`, which thread `at`'s entries contain (`base`: the places before
// them).  Where it falls into an item's fixed places, or into an item of at most `small`
// places, it is moved to the item's beginning or its nearer end.
template <int NR>
__device__ __forceinline__ Place place_of(const PagedParams &p, int at, int base, int per, int n, int pos, int small) {
    Place f{min(at * per, n - 1), base, pos};
#pragma unroll 1
    for (const int e1 = min(n, f.entry + per); f.entry < e1 - 1; ++f.entry) {
        const int w = entry_weight<NR>(p, f.entry);
        if (pos < f.base + w) break;
        f.base += w;
    }
    const int b = p.sel ? f.entry / p.Hkv : f.entry, h = p.sel ? f.entry % p.Hkv : 0;
    const int size = kPgFixed + item_tiles(p, b, h, sequence(p, b).len), in = (uint32_t)(pos - f.base) % (uint32_t)size;
    if (in <= kPgFixed || (size <= small && 2 * in < size))
        f.pos -= in;
    else if (size <= small)
        f.pos += size - in;
    return f;
}

// What a warp does for one item.
struct Work {
    int q0, nq, len;
    int b, h, row0, rows;     // its first query row, and how many the sequence has for this head
    int tiles, t0, t1;        // tiles of the item, and this warp's of them
    int last;                 // whether the warp's share ends with it
    int end;                  // the place behind its last tile
};
static_assert(sizeof(Work) == 48, "");

// Where a warp is: behind the last item that it has looked up.
struct Start {
    Place ahead;   // entry -1: no work
    int end;       // of the warp's share
};

// The next item of a warp, into `it`; `at` moves behind the warp's tiles of it.  Called
// by one lane or by a whole warp (whose lanes then write the same), with both in shared
// memory.  (Rare work like this is kept out of line, so that the loop over tiles stays
// within the instruction cache: with all of it inlined, in 64 bits, the kernel was 192 KB
// long and spent 25 us on fetching itself.)
template <int NR>
__device__ __noinline__ void work_at(const Layout &p, Start *at, Work *it) {
    // The scan's lengths and these are the same unless the caller changes them during
    // the call; the bounds on entry, head and block keep every access inside even then.
    const int n = p.sel ? p.B * p.Hkv : p.B, pos = at->ahead.pos, end = at->end;
    int entry = at->ahead.entry, base = at->ahead.base;
#pragma unroll 1
    for (; entry < n - 1; ++entry) {
        const int w = entry_weight<NR>(p, entry);
        if (pos < base + w) break;
        base += w;
    }
    const int b = p.sel ? entry / p.Hkv : entry;
    int h = p.sel ? entry % p.Hkv : 0;
    const Seq s = sequence(p, b);
    const int tiles = item_tiles(p, b, h, s.len), w = kPgFixed + tiles, rows = s.nq * p.G;
    int rt = (int)((uint32_t)(pos - base) / (uint32_t)w);
    const int first = base + rt * w;
    if (!p.sel) {
        const int rts = (uint32_t)(rows + NR - 1) / NR;
        h = rt;
        if (rts > 1)
            h = rt / rts, rt %= rts;
        else
            rt = 0;
        h = min(h, p.Hkv - 1);
    }
    const int t0 = max(0, pos - first - kPgFixed), t1 = max(t0 + 1, min(tiles, end - first - kPgFixed));
    it->q0 = s.q0, it->nq = s.nq, it->len = s.len;
    it->b = b, it->h = h, it->row0 = rt * NR, it->rows = rows;
    it->tiles = tiles, it->t0 = t0, it->t1 = t1;
    it->last = first + kPgFixed + t1 >= end;
    it->end = first + w;
    at->ahead = Place{entry, base, first + kPgFixed + t1};
}

// Scans the line and starts every warp of the block.  Returns the share of a block.
template <int WARPS, int NR>
__device__ __forceinline__ int scan_line(const PagedParams &p, Layout *layout, int *sums, Start *start, Work *work_of, int works) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int THREADS = 32 * WARPS;
    __shared__ int share_sm;
    const int n = p.sel ? p.B * p.Hkv : p.B;
    const int per = (n + THREADS - 1) / THREADS;
    long long x = 0;
#pragma unroll 4
    for (int e = min(n, tid * per); e < min(n, tid * per + per); ++e) x += entry_weight<NR>(p, e);
    sums[tid] = (int)min(x, 0x7fffffffll);
    __syncthreads();
    if (warp == 0) {  // a lane takes WARPS threads' sums, then a boundary between warps, then a warp's first item
        int sum[WARPS];
        long long all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            all += sums[lane * WARPS + w];
            sum[w] = (int)all;
        }
        x = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        const long long all_places = __shfl_sync(0xffffffffu, x, 31);
        int total = (int)all_places;
        if (all_places >= 0x7ff00000ll) {  // cu_q does not ascend: more tokens than T
            total = 0;
            if (lane == 0) atomicExch(&g_status_paged, (int)FA_ERR_BAD_SHAPE);
        }
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sums[lane * WARPS + w] = sum[w] + (int)(x - all);
        __syncwarp();
        int share = (int)((uint32_t)(total + gridDim.x - 1) / gridDim.x);
        // With less work than the chip has room for, items of up to two least shares stay whole.
        const int small = share <= kPgMinShare ? 2 * kPgMinShare : max(share / kPgSmall, kPgWhole);
        share = max(share, kPgMinShare);
        // The block's ends.  Which thread's entries hold them: a lane's twelve or eight sums,
        // then one of those.
        const int x32 = (int)min(x, 0x7fffffffll);
        auto holder = [&](int pos) {
            const int in = max(0, __ffs((int)__ballot_sync(0xffffffffu, x32 > pos)) - 1);
            const uint32_t above = __ballot_sync(0xffffffffu, lane < WARPS && sums[in * WARPS + min(lane, WARPS - 1)] > pos);
            return in * WARPS + max(0, __ffs((int)above) - 1);
        };
        const long long cut0 = (long long)blockIdx.x * share, cut1 = cut0 + share;
        const int at0 = holder((int)min(cut0, total - 1ll)), at1 = holder((int)min(cut1, total - 1ll));
        Place f{0, 0, total};
        {
            const long long cut = lane == WARPS ? cut1 : cut0;
            const int at = lane == WARPS ? at1 : at0;
            if (cut < total) f = place_of<NR>(p, at, at ? sums[at - 1] : 0, per, n, (int)cut, small);
        }
        // the warps' ends, between them
        const int begin = __shfl_sync(0xffffffffu, f.pos, 0), end = __shfl_sync(0xffffffffu, f.pos, WARPS);
        const int part = (end - begin + WARPS - 1) / WARPS, pos = begin + lane * part;
        if (lane > 0 && lane < WARPS) {
            f.pos = end;
            if (pos < end) {
                int lo = at0, hi = at1;  // the first thread whose sum is above pos
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sums[mid] > pos)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                f = place_of<NR>(p, lo, lo ? sums[lo - 1] : 0, per, n, pos, max(part / kPgSmall, kPgWhole));
            }
        }
        const int mine = __shfl_down_sync(0xffffffffu, f.pos, 1);
        if (lane < WARPS) {
            start[lane] = Start{f, mine};
            if (f.pos < mine)
                work_at<NR>(*layout, start + lane, work_of + lane * works);
            else
                start[lane].ahead.entry = -1;
        }
        if (lane == 0) share_sm = share;
    }
    __syncthreads();
    return share_sm;
}

// ------------------------------------------------------------- instructions
// 16 bytes, or zeros for bytes = 0; read once, so the first to leave the L2
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// two 16x16 tiles of bytes, transposed: lane l's address is row l of the 32.  Of each tile
// the lane gets bytes 4t .. 4t+3 of (transposed) rows g and g + 8.
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// one such tile: lane l's address is row l of the 16
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x1.trans.shared.b8 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
// two e4m3 codes -> two fp16
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
// c (16 x 8, fp32) += a (16 x 16, fp16) b (16 x 8, fp16)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// The workspace: for each block what the item that it leaves off needs to be
// joined, then two slots of partial results for each warp: 0 for an item that was begun
// before the warp, 1 (the first warp's) for the one that the block leaves off.  A slot is
// [rows][D] sums, [rows] m, [rows] l.
struct __align__(16) Tail {
    int parts;               // 0: no item is left off.  Part 0 is slot 1 of this block's first
    int q0, nq, h;           // warp, part j slot 0 of that of the j-th block behind
    int row0, pad[3];
};
__device__ __forceinline__ Tail *tail_of(float *ws, int block) { return reinterpret_cast<Tail *>(ws) + block; }
__device__ __forceinline__ float *slot_of(float *ws, int blocks, int worker, int slot, int nr, int D) {
    return ws + (long long)blocks * (sizeof(Tail) / 4) + (2ll * worker + slot) * nr * (D + 2);
}

// m - 8 + 12 + log2 l in base e.  l's exponent is added to m before its mantissa's
// logarithm: both are near what LSE is not, and would cost it their rounding.
__device__ __forceinline__ float lse_of(float m, float l) {
    const uint32_t u = __float_as_uint(l);
    const float whole = (float)((int)(u >> 23) - 127) + (kPgDown - kPgShift);
    const float frac = log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
    if (l == 0.f) return -INFINITY;
    if (!(l < INFINITY)) return m + l;
    return ((m + whole) + frac) * 0.69314718055994531f;
}

// What O's sums are multiplied with.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : 0x1p-12f / l; }
static_assert(kPgDown == 12.f, "");

// The token of a sequence that a row belongs to.
__device__ __forceinline__ int token_of(const PagedParams &p, int nq, int row) { return nq > 1 ? row / p.G : 0; }

// The place of a row of (sequence, head) among the T * Hq rows of O and LSE.
__device__ __forceinline__ long long out_row(const PagedParams &p, int q0, int nq, int h, int row) {
    const int tok = token_of(p, nq, row);
    return (long long)(q0 + tok) * (p.Hkv * p.G) + h * p.G + (row - tok * p.G);
}

__device__ __noinline__ void write_tail(float *ws, const Work *it, int share) {
    const int parts = min((it->end - 1) / share, (int)gridDim.x - 1) - (int)blockIdx.x + 1;
    *tail_of(ws, blockIdx.x) = Tail{parts, it->q0, it->nq, it->h, it->row0, {0, 0, 0}};
}

// --------------------------------------------------------------- the kernel
template <int D, int NT>
__global__ void __launch_bounds__(PgCfg<D, NT>::THREADS, 1) fa_fwd_paged_kernel(const __grid_constant__ PagedParams p) {
    using C = PgCfg<D, NT>;
    constexpr int NR = 8 * NT;
    constexpr int KG = D / 64;  // groups of four 16-byte pieces of a row
    // Halves of a tile at a time: one where the registers are full of sums.
    constexpr int HB = D == 128 && NT == 4 ? 1 : 2;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ Start start[C::WARPS];
    __shared__ Layout layout;
    __shared__ int flag_of[C::WARPS];
    __shared__ float join_m[C::WARPS][NR], join_l[C::WARPS][NR], join_f[C::WARPS][NR];
    __shared__ float close_f[C::WARPS][NR], inv_of[C::WARPS][NR];
    // (the parameters are there before the kernel before this one has ended)
    if (threadIdx.x == 0) layout = Layout{p.cu_q, p.seq_lens, p.sel, p.sel_count, p.B, p.T, p.G, p.Hkv, p.sel_width, p.page_log2, p.max_len};
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int page = 1 << p.page_log2;
    const uint32_t ring = smem_u32(sm) + warp * C::ST * C::STAGE_BYTES;
    float4 *const meta_of = reinterpret_cast<float4 *>(sm + C::OFF_META) + warp * C::ST * 2;
    Work *const work_of = reinterpret_cast<Work *>(sm + C::OFF_WORK) + warp * C::WORKS;
    const uint64_t policy = l2_policy_evict_first();

    const int share = scan_line<C::WARPS, NR>(p, &layout, reinterpret_cast<int *>(sm + C::OFF_SUMS), start,
                                              reinterpret_cast<Work *>(sm + C::OFF_WORK), C::WORKS);
    const bool busy = start[warp].ahead.entry >= 0;
    if (lane == 0) {
        if (warp == 0) tail_of(p.ws, blockIdx.x)->parts = 0;
        flag_of[warp] = 0;
    }

    // ---- pages: up to 16 tiles (32 halves) of one item looked up at a time, a half a
    // lane, one such batch ahead of the copies; the items go into a ring for the loop below
    // (What is used once an item stays in shared memory: the loop needs the registers.)
    const Work *next = work_of;  // the item being looked up
    int t_next = busy ? next->t0 : 0, works = 1;
    int ph_next, key_next, nv_next, n_next;  // page * Hkv + head (-1: outside the cache), first key, keys there
    auto look_up = [&]() {
        n_next = 0;
        ph_next = 0, key_next = kPgMaxLen, nv_next = 0;
        if (!busy) return;
        if (t_next == next->t1) {
            if (next->last) return;
            next = work_of + (works & (C::WORKS - 1));
            ++works;
            __syncwarp();
            if (lane == 0) work_at<NR>(layout, start + warp, const_cast<Work *>(next));
            __syncwarp();
            t_next = next->t0;
        }
        n_next = min(16, next->t1 - t_next);
        const int at = (t_next + (lane >> 1)) * kPgTile + (lane & 1) * 16;
        t_next += n_next;
        if ((lane >> 1) >= n_next) return;
        int of = at >> p.page_log2;  // position in the block table
        if (p.sel) {
            const long long bh = (long long)next->b * p.Hkv + next->h;
            if ((uint32_t)of >= (uint32_t)max(0, min(p.sel_count[bh], p.sel_width))) return;
            of = p.sel[bh * p.sel_width + of];
            if (of < 0 || of >= (next->len + page - 1) >> p.page_log2) {
                ph_next = -1, key_next = 0;
                return;
            }
            const int k = (of << p.page_log2) + (at & (page - 1));
            if (k >= next->len) return;
            key_next = k;
        } else {
            if ((uint32_t)at >= (uint32_t)next->len) return;
            key_next = at;
        }
        const int pg = p.table[(long long)next->b * p.max_pages + of];
        const bool good = pg >= 0 && pg < p.num_pages;
        ph_next = good ? pg * p.Hkv + next->h : -1;
        nv_next = good ? min(16, next->len - key_next) : 0;
    };
    look_up();
    // The batch being copied: each lane's half as a row of the cache.
    uint32_t row_now = 0, full_now = 0;
    int ph_now = 0, key_now = 0, nv_now = 0, n_now = 0, at_now = 0, stage_in = 0;
    const uint8_t *const k_lane = p.k_pages + lane * 16, *const v_lane = p.v_pages + lane * 16;
    const int r_lane = lane / C::CHUNKS;  // row of this lane's piece among those of one copy
    const uint32_t dst_lane = ring + r_lane * D + ((lane % C::CHUNKS) ^ C::swap(r_lane)) * 16;
    constexpr int PER = C::HALF_BYTES / 512;           // copies a half
    constexpr uint32_t ODD = D == 128 ? 16u : 0u;      // every other copy's rows are 4 further
    auto issue = [&]() {
        if (at_now == n_now) {
            at_now = 0;
            n_now = n_next;
            if (n_now > 0) {
                ph_now = ph_next, key_now = key_next;
                row_now = ((uint32_t)max(ph_now, 0) << p.page_log2) + (key_next & (page - 1));
                nv_now = nv_next;
                full_now = __ballot_sync(0xffffffffu, nv_now == 16);
            }
        }
        if (at_now < n_now) {
            const uint32_t st = dst_lane + stage_in * C::STAGE_BYTES;
            const bool full = ((full_now >> (2 * at_now)) & 3u) == 3u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t row = __shfl_sync(0xffffffffu, row_now, 2 * at_now + half);
                const uint8_t *const ks = k_lane + (unsigned long long)row * D, *const vs = v_lane + (unsigned long long)row * D;
                if (full) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const uint32_t dst = ((j & 1) ? st ^ ODD : st) + half * C::HALF_BYTES + j * 512;
                        cp_async16(dst, ks + j * 512, policy);
                        cp_async16(dst + 2 * C::HALF_BYTES, vs + j * 512, policy);
                    }
                } else {  // rows behind the sequence read as 0
                    const int nv = __shfl_sync(0xffffffffu, nv_now, 2 * at_now + half);
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const uint32_t dst = ((j & 1) ? st ^ ODD : st) + half * C::HALF_BYTES + j * 512;
                        const int n = j * (16 / PER) + r_lane < nv ? 16 : 0;
                        cp_async16(dst, ks + j * 512, n, policy);
                        cp_async16(dst + 2 * C::HALF_BYTES, vs + j * 512, n, policy);
                    }
                }
            }
            if ((lane >> 1) == at_now) {  // what the tile's consumer needs: the first key and the page's scales
                float *const meta = reinterpret_cast<float *>(meta_of + stage_in * 2 + (lane & 1));
                meta[0] = __int_as_float(key_now);
                if (ph_now >= 0) {
                    cp_async4(smem_u32(meta + 1), p.k_scale + ph_now);
                    cp_async4(smem_u32(meta + 2), p.v_scale + ph_now);
                } else {
                    meta[1] = __int_as_float(0x7fc00000), meta[2] = 1.f;
                    atomicExch(&g_status_paged, (int)FA_ERR_BAD_PAGE);
                }
            }
            if (at_now == 0) look_up();  // the next batch's pages, while the copies run
            ++at_now;
            stage_in = stage_in + 1 == C::ST ? 0 : stage_in + 1;
        }
        cp_commit();
    };
    // where this lane reads: K rows by 16-byte loads, V rows by ldmatrix
    const int gk = C::key_of(g);
    const uint32_t k_read = ring + gk * D + (t ^ C::swap(gk)) * 16;
    constexpr uint32_t TWO = D == 128 ? 32u : 16u;  // what two rows further changes of where a piece lies
    const int v_row = HB == 2 ? lane : lane & 15;
    const uint32_t v_read = ring + 2 * C::HALF_BYTES + v_row * D + C::swap(v_row) * 16;
    int stage_out = 0;

    // ---- the warp's tiles, item after item
    const Work *it = work_of;
    int i = 0, done = 0, fill = C::ST - 1;
    int t1 = 0;  // where the item's tiles end
    uint32_t qf[C::Q_SHARED ? 1 : NT][KG][4][2];  // fragments of Q^T (lane: row g of each tile of 8)
    uint2 *const q_sm = reinterpret_cast<uint2 *>(sm + C::OFF_Q) + warp * (KG * 4 * NT * 32) + lane;  // or here, [kg][w][nt]
    float fac[NT][2];           // c 2^e of the rows 2t, 2t+1, which this lane holds in accumulators
    int lim_min = 0;              // the first key that some row of the item does not see
    float z_top = kPgNone;        // the largest value scale of the item so far, as a logarithm
    float m[NT][2], l[NT][2], acc[C::CHUNKS][NT][4];
    if (busy) {
#pragma unroll 1
        for (;;) {
            if (fill == 0) {
                cp_wait<C::ST - 2>();
                __syncwarp();
            }
            issue();  // into the stage that the tile before was read from
            if (i == t1) {  // the next item
                __syncwarp();
                it = work_of + (done & (C::WORKS - 1));
                ++done;
                i = it->t0, t1 = it->t1;
                z_top = kPgNone;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = it->row0 + nt * 8 + g, tok = token_of(p, it->nq, row);
                const __nv_bfloat16 *const q = static_cast<const __nv_bfloat16 *>(p.q) + (long long)(it->q0 + tok) * p.q_stride +
                                               (long long)(it->h * p.G + row - tok * p.G) * D + 16 * t;
                uint4 w[KG][2];
                uint32_t am = 0;
#pragma unroll
                for (int i = 0; i < KG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        w[i][j] = make_uint4(0, 0, 0, 0);
                        if (row < it->rows) {
                            w[i][j] = __ldg(reinterpret_cast<const uint4 *>(q + 64 * i + 8 * j));
                        }
                        const uint32_t u[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) am = max(am, max(u[c] & 0x7fffu, (u[c] >> 16) & 0x7fffu));
                    }
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                const int e = am ? max(-126, min(126, (int)(am >> 7) - 127)) : 0;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int i = 0; i < KG; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t u[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
                        uint32_t f[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            f[c] = pack_f16x2(__uint_as_float(u[c] << 16) * down, __uint_as_float(u[c] & 0xffff0000u) * down);
                        if (C::Q_SHARED) {
                            q_sm[((i * 4 + 2 * j) * NT + nt) * 32] = make_uint2(f[0], f[1]);
                            q_sm[((i * 4 + 2 * j + 1) * NT + nt) * 32] = make_uint2(f[2], f[3]);
                        } else {
                            qf[C::Q_SHARED ? 0 : nt][i][2 * j][0] = f[0], qf[C::Q_SHARED ? 0 : nt][i][2 * j][1] = f[1];
                            qf[C::Q_SHARED ? 0 : nt][i][2 * j + 1][0] = f[2], qf[C::Q_SHARED ? 0 : nt][i][2 * j + 1][1] = f[3];
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fac[nt][j] = p.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
                }
            }
            lim_min = it->len - it->nq + token_of(p, it->nq, it->row0) + 1;

#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    m[nt][0] = m[nt][1] = kPgNone;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[c][nt][j] = 0.f;
                }
            }
            if (fill > 0) {
                --fill;
                continue;
            }
            const uint32_t st = stage_out * C::STAGE_BYTES;
            const float4 *const stage_meta = meta_of + stage_out * 2;
            stage_out = stage_out + 1 == C::ST ? 0 : stage_out + 1;
#pragma unroll 1
            for (int h0 = 0; h0 < 2; h0 += HB) {
                float4 meta[HB];  // first key, scales
                int key[HB], key_max = 0;
#pragma unroll
                for (int half = 0; half < HB; ++half) {
                    meta[half] = stage_meta[h0 + half];
                    key[half] = __float_as_int(meta[half].x);
                    key_max = max(key_max, key[half]);
                }
#pragma unroll
                for (int half = 0; half < HB; ++half) {  // the value scale's logarithm, exact for powers of two, and its inverse
                    const int u = __float_as_int(meta[half].z);
                    meta[half].z = fmaxf((float)((u >> 23) - 127) + lg2_approx(__int_as_float((u & 0x7fffff) | 0x3f800000)), -100.f);
                    meta[half].w = ex2_approx(-meta[half].z) * 0x1p-12f;
                    if (key[half] != kPgMaxLen) z_top = fmaxf(z_top, meta[half].z);
                }
                bool apart = false;  // whether some keys' value scale is far below one before
#pragma unroll
                for (int half = 0; half < HB; ++half) apart |= key[half] != kPgMaxLen && meta[half].z < z_top - kPgApart;

                // ---- S^T = K Q^T: a half of 16 keys an MMA tile.  The order of d within the
                // contraction is free as long as Q's is the same: lane t takes whole 16-byte
                // pieces t and t + 4 of its keys' rows, four MMAs' worth each.
                float sc[HB][NT][4];
#pragma unroll
                for (int half = 0; half < HB; ++half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sc[half][nt][j] = 0.f;
                // Both halves' MMAs take turns: one that adds to the sums of another waits for it.
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
                    uint32_t a[HB][4], b8[HB][4];
#pragma unroll
                    for (int half = 0; half < HB; ++half) {
                        const uint32_t at = ((k_read + st) ^ (kg * 64)) + (h0 + half) * C::HALF_BYTES;
                        ld_shared_v4(at, a[half][0], a[half][1], a[half][2], a[half][3]);
                        ld_shared_v4((at ^ TWO) + 2 * D, b8[half][0], b8[half][1], b8[half][2], b8[half][3]);
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint2 q[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            q[nt] = C::Q_SHARED ? q_sm[((kg * 4 + w) * NT + nt) * 32]
                                                : make_uint2(qf[C::Q_SHARED ? 0 : nt][kg][w][0], qf[C::Q_SHARED ? 0 : nt][kg][w][1]);
#pragma unroll
                        for (int half = 0; half < HB; ++half) {
                            const uint32_t a0 = codes_f16x2(a[half][w]), a1 = codes_f16x2(b8[half][w]);
                            const uint32_t a2 = codes_f16x2(a[half][w] >> 16), a3 = codes_f16x2(b8[half][w] >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(sc[half][nt], a0, a1, a2, a3, q[nt].x, q[nt].y);
                        }
                    }
                }
                // ---- exponents of the weights, against the maximum in use
                const bool edge = key_max + 16 > lim_min;  // some row does not see some key
                float y[HB][NT][4], top = kPgNone;
                auto exponents = [&](int half, int nt, int j, float off, int limit) {
                    const float x = fmaf(sc[half][nt][j], fac[nt][j & 1] * meta[half].y, meta[half].z + off);
                    return key[half] + gk + (j >> 1) * 2 < limit ? x : -INFINITY;
                };
                if (!edge) {
#pragma unroll
                    for (int half = 0; half < HB; ++half)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                y[half][nt][j] = fmaf(sc[half][nt][j], fac[nt][j & 1] * meta[half].y,
                                                      meta[half].z + (kPgShift - m[nt][j & 1]));
                                top = fmaxf(top, y[half][nt][j]);
                            }
                }
                if (__any_sync(0xffffffffu, edge || top > kPgMost)) {
                    // a new maximum: the sums so far are scaled to it
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int row = it->row0 + nt * 8 + 2 * t + j;
                            const int limit = !edge ? INT_MAX : row < it->rows ? it->len - it->nq + token_of(p, it->nq, row) + 1 : it->len;
                            float x = kPgNone;
#pragma unroll
                            for (int half = 0; half < HB; ++half)
                                x = fmaxf(x, fmaxf(exponents(half, nt, j, 0.f, limit), exponents(half, nt, j + 2, 0.f, limit)));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            x = fmaxf(floorf(x), m[nt][j]);
                            const float f = ex2_approx(m[nt][j] - x);
                            m[nt][j] = x;
                            l[nt][j] *= f;
#pragma unroll
                            for (int c = 0; c < C::CHUNKS; ++c) acc[c][nt][j] *= f, acc[c][nt][j + 2] *= f;
#pragma unroll
                            for (int half = 0; half < HB; ++half) {
                                y[half][nt][j] = exponents(half, nt, j, kPgShift - x, limit);
                                y[half][nt][j + 2] = exponents(half, nt, j + 2, kPgShift - x, limit);
                            }
                        }
                }
                // ---- weights, and their transpose as the B operand (keys x rows); then
                // O^T += V^T W^T: a lane has the rows (of V^T) g and g + 8 of each tile of 16,
                // four keys in a register.
                uint32_t wf[HB][NT][2];
                if (!apart && (!edge || lim_min >= it->len)) {
#pragma unroll
                    for (int half = 0; half < HB; ++half)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                w[j] = ex2_approx(y[half][nt][j]);
                                l[nt][j & 1] = fmaf(w[j], meta[half].w, l[nt][j & 1]);
                            }
                            wf[half][nt][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                            wf[half][nt][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
                        }
                    constexpr int CG = NT == 1 ? 4 : NT == 2 ? 2 : 1;  // tiles whose MMAs take turns
#pragma unroll
                    for (int c0 = 0; c0 < C::CHUNKS; c0 += CG) {
                        uint32_t r[CG][2 * HB];
#pragma unroll
                        for (int c = 0; c < CG; ++c) ldmatrix_b8_trans(((v_read + st) ^ ((c0 + c) * 16)) + h0 * C::HALF_BYTES, r[c]);
#pragma unroll
                        for (int half = 0; half < HB; ++half)
#pragma unroll
                            for (int c = 0; c < CG; ++c) {
                                const uint32_t lo = r[c][2 * half], hi = r[c][2 * half + 1];
                                const uint32_t a0 = codes_f16x2(lo), a1 = codes_f16x2(hi);
                                const uint32_t a2 = codes_f16x2(lo >> 16), a3 = codes_f16x2(hi >> 16);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_f16(acc[c0 + c][nt], a0, a1, a2, a3, wf[half][nt][0], wf[half][nt][1]);
                            }
                    }
                } else {
                    // Rare tiles: value scales far apart, or keys that some rows do not see.  Each half's
                    // weights are rounded against their own maximum, and its sums scaled back in fp32.
                    // A weight of 0 would still turn a NaN among the values into NaN, so the values that
                    // a token does not see are cleared, a token at a time, and only that token's rows
                    // take the result.
                    const bool cut = edge && lim_min < it->len;
                    const int tok0 = cut ? it->row0 / p.G : 0, tok1 = cut ? min(it->nq - 1, (it->row0 + NR - 1) / p.G) : 0;
                    float back[HB][NT][2];
#pragma unroll
                    for (int half = 0; half < HB; ++half)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float(&yh)[4] = y[half][nt];
                            float w[4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float x = fmaxf(yh[j], yh[j + 2]);
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                x = x == -INFINITY ? 0.f : x - kPgShift;
                                back[half][nt][j] = ex2_approx(x);
#pragma unroll
                                for (int e = j; e < 4; e += 2) {
                                    w[e] = ex2_approx(yh[e] - x);
                                    l[nt][j] = fmaf(w[e] * back[half][nt][j], meta[half].w, l[nt][j]);
                                }
                            }
                            wf[half][nt][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                            wf[half][nt][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
                        }
#pragma unroll 1
                    for (int tok = tok0; tok <= tok1; ++tok) {
                        const int limit = cut ? it->len - it->nq + tok + 1 : INT_MAX, first = tok * p.G - it->row0;
                        bool my[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) my[nt][j] = !cut || (uint32_t)(nt * 8 + 2 * t + j - first) < (uint32_t)p.G;
                        uint32_t seen[HB];
#pragma unroll
                        for (int half = 0; half < HB; ++half) {
                            const int k = key[half] + 4 * t;  // the first of the lane's four keys
                            seen[half] = k + 4 <= limit ? 0xffffffffu : k >= limit ? 0u : (1u << 8 * (limit - k)) - 1;
                        }
#pragma unroll
                        for (int c = 0; c < C::CHUNKS; ++c) {
                            uint32_t r[2 * HB];
                            ldmatrix_b8_trans(((v_read + st) ^ (c * 16)) + h0 * C::HALF_BYTES, r);
#pragma unroll
                            for (int half = 0; half < HB; ++half) {
                                const uint32_t lo = r[2 * half] & seen[half], hi = r[2 * half + 1] & seen[half];
                                const uint32_t a0 = codes_f16x2(lo), a1 = codes_f16x2(hi);
                                const uint32_t a2 = codes_f16x2(lo >> 16), a3 = codes_f16x2(hi >> 16);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float o[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_f16(o, a0, a1, a2, a3, wf[half][nt][0], wf[half][nt][1]);
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        if (my[nt][j & 1]) acc[c][nt][j] = fmaf(o[j], back[half][nt][j & 1], acc[c][nt][j]);
                                }
                            }
                        }
                    }
                }
            }

            if (++i < t1) continue;

            // ---- an item ends here, or the warp's share of it.  Neighbouring lanes exchange
            // halves, so that each has two neighbouring elements: pair `pg` of a tile's 8.
            const int pg = (g >> 1) + 4 * (g & 1);
#pragma unroll
            for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float got = __shfl_xor_sync(0xffffffffu, (g & 1) ? acc[c][nt][j] : acc[c][nt][j + 2], 4);
                        if (g & 1)
                            acc[c][nt][j] = got;
                        else
                            acc[c][nt][j + 2] = got;
                    }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
                }
            bool whole = it->t0 == 0;
            float *part = slot_of(p.ws, gridDim.x, blockIdx.x * C::WARPS + warp, 0, NR, D);
            if (it->last) {
                // Warps that had nothing else than more of the item of the warp before them
                // form a group with it, and so does, if the item still goes on, what the next
                // warp left of its first item in its slot 0.  (That warp had other items
                // behind it, so the item ended there.)
                float2 *const sums_of = reinterpret_cast<float2 *>(sm + warp * C::ST * C::STAGE_BYTES) + lane;  // over the ring
                cp_wait<0>();
                __syncwarp();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (g == 0) {
                            join_m[warp][nt * 8 + 2 * t + j] = m[nt][j];
                            join_l[warp][nt * 8 + 2 * t + j] = l[nt][j];
                        }
#pragma unroll
                        for (int c = 0; c < C::CHUNKS; ++c)
                            sums_of[((c * NT + nt) * 2 + j) * 32] = make_float2(acc[c][nt][j], acc[c][nt][j + 2]);
                    }
                if (lane == 0)
                    flag_of[warp] = (warp > 0 && done == 1 && it->t0 > 0 ? 1 : 0) | (it->t1 < it->tiles ? 2 : 0) | (it->t0 == 0 ? 4 : 0) | 8;
                named_bar_sync(1, C::THREADS);
                int lead = warp, last = warp;
                while (lead > 0 && (flag_of[lead] & 1)) --lead;
                while (last + 1 < C::WARPS && (flag_of[last + 1] & 1)) ++last;
                bool open = flag_of[last] & 2;
                const bool begins = flag_of[lead] & 4;
                const bool closes = open && last + 1 < C::WARPS && (flag_of[last + 1] & 8);
                const float *const closing = slot_of(p.ws, gridDim.x, blockIdx.x * C::WARPS + min(last + 1, C::WARPS - 1), 0, NR, D);
                if (closes) open = false;
                whole = begins && !open;
                part = slot_of(p.ws, gridDim.x, blockIdx.x * C::WARPS, begins, NR, D);  // (begun before the block: by its first warp)
                if (begins && open && warp == lead && lane == 0)
                    write_tail(p.ws, it, share);
                if (lead != last || closes) {
                    if (lane < NR) {  // a row's maximum over the group, and the factors of its parts to it
                        float M = closes ? closing[NR * D + lane] : kPgNone, L = 0.f, f = 0.f;
#pragma unroll 4
                        for (int w = lead; w <= last; ++w) M = fmaxf(M, join_m[w][lane]);
                        if (closes) {
                            f = ex2_approx(closing[NR * D + lane] - M);
                            L = closing[NR * D + NR + lane] * f;
                        }
                        close_f[warp][lane] = f;
#pragma unroll 4
                        for (int w = lead; w <= last; ++w) L = fmaf(join_l[w][lane], ex2_approx(join_m[w][lane] - M), L);
                        join_f[warp][lane] = ex2_approx(join_m[warp][lane] - M);
                        inv_of[warp][lane] = whole ? inverse_of(L) : 1.f;
                        if (warp == lead) {
                            if (!whole)
                                part[NR * D + lane] = M, part[NR * D + NR + lane] = L;
                            else if (it->row0 + lane < it->rows)
                                p.lse[out_row(p, it->q0, it->nq, it->h, it->row0 + lane)] = lse_of(M, L);
                        }
                    }
                    named_bar_sync(1, C::THREADS);
#pragma unroll 1
                    for (int u = warp - lead; u < C::CHUNKS * NT * 2; u += last - lead + 1) {  // the group's warps share the sums
                        const int c = u / (2 * NT), r = (u / 2 % NT) * 8 + 2 * t + (u & 1);
                        float2 o = make_float2(0.f, 0.f);
                        if (closes) {
                            o = reinterpret_cast<const float2 *>(closing + r * D)[8 * c + pg];
                            o.x *= close_f[warp][r], o.y *= close_f[warp][r];
                        }
#pragma unroll 4
                        for (int w = lead; w <= last; ++w) {
                            const float2 x = reinterpret_cast<const float2 *>(sm + w * C::ST * C::STAGE_BYTES)[u * 32 + lane];
                            o.x = fmaf(x.x, join_f[w][r], o.x), o.y = fmaf(x.y, join_f[w][r], o.y);
                        }
                        const float inv = inv_of[warp][r];
                        if (!whole)
                            reinterpret_cast<float2 *>(part + r * D)[8 * c + pg] = o;
                        else if (it->row0 + r < it->rows)
                            reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.o) + out_row(p, it->q0, it->nq, it->h, it->row0 + r) * D)[8 * c + pg] =
                                pack_bf16x2(o.x * inv, o.y * inv);
                    }
                    return;
                }
                named_bar_sync(1, C::THREADS);
            }
            // ---- written out, or what is known of it
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = nt * 8 + 2 * t + j;
                    if (!whole) {
                        float2 *const o = reinterpret_cast<float2 *>(part + r * D) + pg;
#pragma unroll
                        for (int c = 0; c < C::CHUNKS; ++c) o[8 * c] = make_float2(acc[c][nt][j], acc[c][nt][j + 2]);
                        if (g == 0) part[NR * D + r] = m[nt][j], part[NR * D + NR + r] = l[nt][j];
                    } else if (it->row0 + r < it->rows) {
                        const float inv = inverse_of(l[nt][j]);
                        const long long at = out_row(p, it->q0, it->nq, it->h, it->row0 + r);
                        uint32_t *const o = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.o) + at * D) + pg;
#pragma unroll
                        for (int c = 0; c < C::CHUNKS; ++c) o[8 * c] = pack_bf16x2(acc[c][nt][j] * inv, acc[c][nt][j + 2] * inv);
                        if (g == 0) p.lse[at] = lse_of(m[nt][j], l[nt][j]);
                    }
                }
            if (it->last) return;
        }
    }
    // a warp without tiles: the others wait for it
    named_bar_sync(1, C::THREADS);
    named_bar_sync(1, C::THREADS);
}

// Joins the partial results of the items that cross blocks: each block of this kernel
// takes every fourth row of the item that one of them left off, a warp a row, or the
// whole block where there are many parts.  Bound by latency: 1 to 2 us behind the kernel
// above (8 x 16384 keys at an earlier step: 51.4 us without it, 54.0 with it; reading the first parts before it
// is known how many there are took off a third: ragged sequences 45.2 -> 44.1 us).
constexpr int kJoinWarps = 4;
constexpr int kJoinMany = 8;  // parts

template <int D, int NR>
struct JoinRow {
    static constexpr int E = D / 32;
    static constexpr int UN = 4;  // parts in flight
    float M, L, O[E];
    float m[UN], l[UN], o[UN][E];

    __device__ __forceinline__ void begin() {
        M = -INFINITY, L = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] = 0.f;
    }
    // parts j0, j0 + step, .. of those below `limit`
    __device__ __forceinline__ void fetch(const PagedParams &p, int blocks, int warps, int block, int r, int j0, int step, int limit) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int j = j0 + u * step;
            if (j >= limit) continue;
            const float *part = slot_of(p.ws, blocks, (block + j) * warps, j == 0, NR, D);
            m[u] = part[NR * D + r];
            l[u] = part[NR * D + NR + r];
            if (E == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(part + r * D + 4 * lane);
                o[u][0] = x.x, o[u][1] = x.y, o[u][E - 2] = x.z, o[u][E - 1] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(part + r * D + 2 * lane);
                o[u][0] = x.x, o[u][1] = x.y;
            }
        }
    }
    // what was fetched, as far as it is below `parts`
    __device__ __forceinline__ void take(int j0, int step, int parts) {
        float now = M;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const bool is = j0 + u * step < parts;
            if (!is || l[u] == 0.f) m[u] = -INFINITY;  // a part without keys does not count
            if (!is) l[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!is) o[u][e] = 0.f;
            now = fmaxf(now, m[u]);
        }
        const float base = now == -INFINITY ? 0.f : now, f0 = ex2_approx(M - base);
        M = now;
        L *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] *= f0;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const float f = ex2_approx(m[u] - base);
            L = fmaf(l[u], f, L);
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] = fmaf(o[u][e], f, O[e]);
        }
    }
    __device__ __forceinline__ void add(float m, float l, const float *o) {
        const float now = fmaxf(M, m), base = now == -INFINITY ? 0.f : now;
        const float f0 = ex2_approx(M - base), f = ex2_approx(m - base);
        M = now, L = fmaf(L, f0, l * f);
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] = fmaf(O[e], f0, o[e] * f);
    }
    __device__ __forceinline__ void write(const PagedParams &p, long long at) {
        const int lane = threadIdx.x & 31;
        const float inv = inverse_of(L);
        uint32_t *const o = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.o) + at * D) + lane * (E / 2);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) o[e] = pack_bf16x2(O[2 * e] * inv, O[2 * e + 1] * inv);
        if (lane == 0) p.lse[at] = lse_of(M == -INFINITY ? 0.f : M, L);
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) fa_paged_join_kernel(const __grid_constant__ PagedParams p) {
    constexpr int NR = 8 * NT, E = D / 32, WARPS = PgCfg<D, NT>::WARPS;
    __shared__ float red_m[kJoinWarps], red_l[kJoinWarps], red_o[kJoinWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.x, blocks = gridDim.x;
    JoinRow<D, NR> row_of;
    grid_wait();
    // The first parts that there may be are read with what says how many there are.
    const int r0 = blockIdx.y * kJoinWarps + warp;
    row_of.fetch(p, blocks, WARPS, block, r0, 0, 1, blocks - block);
    const Tail tail = *tail_of(p.ws, block);
    if (tail.parts == 0) return;
    const int rows = min(NR, tail.nq * p.G - tail.row0);
    row_of.begin();
    if (tail.parts <= kJoinMany) {
        if (r0 >= rows) return;
        row_of.take(0, 1, tail.parts);
#pragma unroll 1
        for (int j0 = row_of.UN; j0 < tail.parts; j0 += row_of.UN) {
            row_of.fetch(p, blocks, WARPS, block, r0, j0, 1, tail.parts);
            row_of.take(j0, 1, tail.parts);
        }
        row_of.write(p, out_row(p, tail.q0, tail.nq, tail.h, tail.row0 + r0));
        return;
    }
#pragma unroll 1
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        row_of.begin();
#pragma unroll 1
        for (int j0 = warp; j0 < tail.parts; j0 += row_of.UN * kJoinWarps) {
            row_of.fetch(p, blocks, WARPS, block, r, j0, kJoinWarps, tail.parts);
            row_of.take(j0, kJoinWarps, tail.parts);
        }
        __syncthreads();  // the row before is read
        if (lane == 0) red_m[warp] = row_of.M, red_l[warp] = row_of.L;
#pragma unroll
        for (int e = 0; e < E; ++e) red_o[warp][lane * E + e] = row_of.O[e];
        __syncthreads();
        if (warp != 0) continue;
#pragma unroll
        for (int v = 1; v < kJoinWarps; ++v) row_of.add(red_m[v], red_l[v], &red_o[v][lane * E]);
        row_of.write(p, out_row(p, tail.q0, tail.nq, tail.h, tail.row0 + r));
    }
}

template <int D, int NT>
static size_t workspace_of(int num_sms) {
    return num_sms * (sizeof(Tail) + (size_t)PgCfg<D, NT>::WARPS * 2 * 8 * NT * (D + 2) * sizeof(float));
}

size_t paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int num_sms) {
    (void)B, (void)T, (void)Hq, (void)Hkv;  // the same for all: what of the forms needs most
    if (D == 64)
        return std::max(workspace_of<64, 1>(num_sms), std::max(workspace_of<64, 2>(num_sms), workspace_of<64, 4>(num_sms)));
    return std::max(workspace_of<128, 1>(num_sms), std::max(workspace_of<128, 2>(num_sms), workspace_of<128, 4>(num_sms)));
}

template <int D, int NT>
static cudaError_t launch_paged(const PagedParams &p, int num_sms, cudaStream_t stream) {
    using C = PgCfg<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(fa_fwd_paged_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_early(fa_fwd_paged_kernel<D, NT>, dim3(num_sms), C::THREADS, C::SMEM, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_early(fa_paged_join_kernel<D, NT>, dim3(num_sms, 8 * NT / kJoinWarps), 32 * kJoinWarps, 0, stream, 1, p);
}

// Rows of an item: 8 or 16 while a sequence's query rows are no more (by the mean
// number of its tokens, padding rounded off).  Beyond, 32 at D = 64 (16 sequences of 16384
// keys, 32 rows: 100 us, 119 us in two items of 16).  At D = 128 the sums of 32 rows leave
// few registers, and items of 32 pay from more than 32 rows on: 8 sequences of 16384 keys with
// 64 rows take 156 us, 172 us in items of 16; with 32 rows 97 and 98 us; but 16 ragged ones
// with 16 to 40 rows 90 and 75 us.  The mean is all that the host knows, and batches of mixed
// kinds pay for it: 63 sequences with one token beside one with 512 take 706 us, 96 and 443 in
// two calls; 64 with one token each and T = 512 take 167 us, 98 with T = 64.
static int item_rows(int D, const PagedParams &p) {
    const long long tokens = (2ll * p.T + p.B) / (2ll * p.B), rows = (tokens > 1 ? tokens : 1) * p.G;
    return rows <= 8 ? 8 : rows <= (D == 128 ? 32 : 16) ? 16 : 32;
}

bool paged_fits(int D, const PagedParams &p) {
    const long long keys = (long long)(p.sel_width > p.max_pages ? p.sel_width : p.max_pages) << p.page_log2;
    const long long items = ((long long)p.T * p.G / item_rows(D, p) + p.B) * p.Hkv;
    const long long places = keys / kPgTile + 1 + kPgFixed;
    return keys <= 0x7fffffff && items < (1ll << 31) && items * places < (1ll << 31) - (1 << 20);
}

cudaError_t launch_fwd_paged(int D, const PagedParams &params, int num_sms, cudaStream_t stream) {
    PagedParams p = params;
    p.max_len = (int)std::min<long long>((long long)p.max_pages << p.page_log2, kPgMaxLen);
    const int rows = item_rows(D, p);
    if (D == 64)
        return rows == 8 ? launch_paged<64, 1>(p, num_sms, stream)
                         : rows == 16 ? launch_paged<64, 2>(p, num_sms, stream) : launch_paged<64, 4>(p, num_sms, stream);
    return rows == 8 ? launch_paged<128, 1>(p, num_sms, stream)
                     : rows == 16 ? launch_paged<128, 2>(p, num_sms, stream) : launch_paged<128, 4>(p, num_sms, stream);
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
