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
// Everything enters the products as fp16, which holds codes exactly (multiples of 2^-9 up to 448):
//   q_r as bf16 scaled by a power of two to a largest element in [1, 2) (elements below 2^-17 of
//   it are rounded, to steps of 2^-24 of it);
//   k_j as code * 2^(e_j - e), e the largest exponent of the key scales in the tile, which is exact to
//   2^-15 of the largest scale;
//   v_j as code * 2^(e_j - e), e the largest exponent of the value scales in the first tile that has a finite one
//   (rows that see the tiles before it are NaN; others do not, and must not be measured by them).  O's sums are in
//   units of 2^e; a tile with a scale more than 2^kCkLift units takes e up to its own, and O is rescaled, so that sums of any
//   number of keys stay finite.
// The powers of two are put back into c (by row and tile) and into O.  A tile with a scale that is no
// power of two, or a key scale below 2^-15 of its largest, goes another way: the codes of keys are taken as they are and scores take
// the key scale over 2^e in fp32, and weights take the rest of the value scale in fp32, before they go to fp16.
// In one with a value scale not within 2^-15 to 2^7 units weights times the value scale go to bf16
// (2^-8 of each), which has the range of fp32, beside the codes themselves.
//
// What bounds it: 4 D operations for a row and a key on the tensor cores, with enough rows
// (256 rows share a tile of 128 keys: 2 D bytes a key for 1024 D operations); the conversion
// of the codes, which the tensor cores cannot read beside 16-bit queries, is 2 D elements a key
// and 256 rows.
//
// Roles of a block (one an SM, persistent):
//   warps 0-3, 4-7   softmax of row sub-tile 0 and 1 (128 rows each): the rows' queries into shared
//                    memory, S from tensor memory, P back over it, O out of it at the end;
//   warps 8-15       codes: each takes 16 keys of a tile, reads them from global memory a tile ahead (into
//                    registers), converts them and writes them to shared memory in the layout
//                    that the MMAs read (128-byte swizzle).  What they issue is what the others have to
//                    wait for, so they do nothing else;
//   warps 16, 19     issue the MMAs of sub-tile 0 and 1: S_j, then O += P V_j as the softmax hands P over, so
//                    that one sub-tile's products run while the other's softmax does.  (One warp for
//                    both, in turns, was itself what a tile waited for: 4500 cycles a tile.)
//   warp 17          the block's work, segment by segment, a ring of four ahead of the others;
//   warp 18          tiles: pages and scales looked up, a ring of eight ahead of the code warps.
//
// Split.  Items (sequence, key/value head, 256 rows) are laid end to end, each as long as its
// keys and a fixed cost, and the line is cut into equal shares, one a block.  What a block has of
// an item is a segment of its tiles.  An item that is cut leaves its parts (normalised sums, m, l; l = 0
// of a block whose share is less than a tile) in the workspace, and a second kernel joins them in order.  Lengths are read on the device.
//
// Every wait is bounded in time; one that gives up records a status code and the block winds down.
//
// Measured, D = 128: 1024 tokens behind 65536, 8 of 32 heads 770 to 800 us, 1,440 to 1,385 TFLOP/s (75 to 72% of the measured bf16 rate); 512 behind
// 16384 129 us, 56%; 4 prompts of 4096, 16 heads 295 us, 48%; 32 sequences of 1 to 1024 tokens behind 50 to 8000, 8 of 64 heads, pages
// of 16 570 us, 46%.  D = 64: 4 prompts of 2048, 16 heads 86 to 92 us, a fifth of the rate.  A tile takes 3,160 to 3,500 cycles, of which the tensor pipe has
// work for 2,050 (64 for each of 32 steps) and the exponentials take 1,024 (32 a cycle, measured); the rest is the way from S
// through the softmax to the next S: 1,630 cycles from S to the second half of P, 1,070 more until the softmax waits for the next S no longer.  (A copy
// with a multiply-add in the place of each exponential was no faster.)  An item's ends cost four to five tiles more, the cut and first
// tile 6 to 11 us, the join 2.5 to 7.  Where scales are no powers of two every tile takes its maximum again: 1.8 to 2.0 times these times.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_chunk = 0;

constexpr int kCkThreads = 640;
constexpr int kCkCodeWarps = 8;
constexpr int kCkRows = 256;        // rows of an item, two sub-tiles of 128
constexpr int kCkTile = 128;        // keys a tile
constexpr int kCkFixed = 576;       // keys that an item's fixed cost stands for (512: the mixed batch above 582 us when this took 567; 640: the prompts 303 when this took 296)
constexpr int kCkMinShare = 768;    // of a block, in keys
constexpr int kCkSegs = 4;          // segments in the ring
constexpr int kCkTiles = 8;         // tiles in theirs
constexpr float kCkShift = 4.f;     // exponent of a weight at the maximum in use
constexpr float kCkMost = 32768.f;  // of a half tile's sum
constexpr int kCkUp = 7, kCkDown = 15;  // how far a scale's exponent may lie above or below the unit for fp16 beside codes
constexpr int kCkLift = 40;         // how far above it takes the unit up
constexpr unsigned long long kCkDrainNs = 20ull * 1000 * 1000;
// Registers: 640 x 96 at launch; what the code warps and the last four give goes to the softmax.  None of
// the loops may spill much (D = 128 does not, D = 64 a word): beside this much shared memory the cache that holds spilled registers is small, and
// they would come from the L2.  (The launch checks that the kernel has as many as the split assumes.)
constexpr int kCkRegsLaunch = 96;
constexpr uint32_t kCkRegsSoftmax = 144, kCkRegsCodes = 64, kCkRegsOther = 64;
static_assert(256 * kCkRegsSoftmax + 256 * kCkRegsCodes + 128 * kCkRegsOther <= kCkThreads * kCkRegsLaunch, "register split");

template <int D>
struct CkCfg {
    static constexpr int ST = D == 128 ? 2 : 3;               // stages of K and of V
    static constexpr uint32_t QT_BYTES = 128 * D * 2;         // a sub-tile's queries
    static constexpr uint32_t KV_BYTES = kCkTile * D * 2;
    static constexpr uint32_t CHUNK = 128 * 128;              // 128 rows x 128 bytes
    static constexpr uint32_t OFF_K = 2 * QT_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + ST * KV_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_V + ST * KV_BYTES;
    static constexpr uint32_t SMEM = OFF_BAR + 4096 + 1024;   // barriers, segments, tiles; alignment
    static constexpr uint32_t TM_O = 256;
    static constexpr uint32_t F16 = ~((7u << 7) | (7u << 10));  // fp16 operands: format 0
    static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kCkTile, false) & F16;
    static constexpr uint32_t IDESC_PV_BF16 = idesc_bf16_f32(128, D, true);
    static constexpr uint32_t IDESC_PV = IDESC_PV_BF16 & F16;
    static constexpr int LOADS = D / 32;                      // 16-byte loads a lane for 16 keys
    static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_BAR % 1024 == 0, "atoms");
    static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one block an SM");
};

// barriers (8 bytes each) in the block's last four kilobytes of shared memory
enum : uint32_t {
    C_Q_FULL = 0,    // + sub-tile
    C_K_FULL = 2,    // + stage (up to 3)
    C_K_EMPTY = 5,
    C_V_FULL = 8,
    C_V_EMPTY = 11,
    C_S_FULL = 14,   // + sub-tile
    C_P_HALF = 16,
    C_P_FULL = 18,   // C_P_HALF + 2
    C_PH_DONE = 20,
    C_O_DONE = 22,
    C_O_FREE = 24,
    C_SEG_FULL = 26,  // + ring place
    C_SEG_FREE = 30,
    C_TILE_FULL = 34,
    C_TILE_FREE = 42,
    C_DRAIN = 50,
    C_COUNT = 51
};
constexpr uint32_t kSlotTmem = 408, kSlotAbort = 412;
constexpr uint32_t kSlotExp = 416;     // 4 words: e of a segment's values, behind its last tile
constexpr uint32_t kSlotNan = 432;     // 4 words: number + 1 of a segment with NaN among masked tiles' values
constexpr uint32_t kSlotSegs = 448;    // 4 segments of 64 bytes
// By the tile's number modulo 16 (the softmax may be ten tiles behind what is looked up):
constexpr uint32_t kSlotWide = 704;    // whether a tile's weights are bf16
constexpr uint32_t kSlotKeyExp = 768;  // 2^e of a tile's keys, negative where it goes the other way
constexpr uint32_t kSlotRest = 832;    // what scores and weights are multiplied with in fp32, of 8 pieces: 64 bytes a tile
// and modulo 8: flags, and 16 bytes for each 16 keys
constexpr uint32_t kSlotFlags = 1856;
constexpr uint32_t kSlotPieces = 2048;
// and modulo 16 again, of a tile that goes the other way: what O is multiplied with before it, where the unit goes up
constexpr uint32_t kSlotLift = kSlotPieces + kCkTiles * 128;
static_assert(C_COUNT * 8 <= kSlotTmem && kSlotRest + 16 * 64 <= kSlotFlags && kSlotFlags + kCkTiles * 4 <= kSlotPieces && kSlotLift + 16 * 4 <= 4096, "");

// What a block does of one item.
struct __align__(16) Seg {
    int q0, rows, row0, c;     // first token; rows of the (sequence, head); the item's first; keys before the step's tokens
    int b, h, len, t0;         // sequence, head, its keys; tiles [t0, t1)
    int t1, first[2], act1;    // load order (from t1 - 1 down) in which each sub-tile begins; whether there is a second one
    int slot, end, pad[2];     // partial result: -1 none (the item is whole), 0 begun before, 1 left off; no more work
};
static_assert(sizeof(Seg) == 64, "");

// Of 16 keys of a tile: their first row of the cache, how many rows have keys, and the factors in fp16 that
// K's and V's codes are multiplied with, in both halves of a word (K's: NaN for a page outside the cache or with a scale that is not finite).
struct __align__(16) Piece {
    uint32_t row;
    int valid;
    uint32_t kf, vf;
};

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
// keys before the step's tokens and those up to its last row's token (about 256 / G more for each item).
__device__ __forceinline__ long long ck_begin(const ChunkParams &p, long long i, int c) {
    return i * (kCkFixed + max(c, 0)) + p.item_keys * (i * (i + 1) >> 1);
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
    const bool whole = w <= share / 4 || tiles <= 3 || (tiles <= 16 && w > share && w <= share + share / 3);
    if (whole) return 2 * in < w ? 0 : tiles;
    const int done = (int)((double)(in - kCkFixed) * tiles / (double)(w - kCkFixed) + 0.5);
    return done < 2 ? 0 : (done > tiles - 2 ? tiles : done);
}

// The cut at place pos, which lies in sequence b that begins at `base`.
__device__ __noinline__ Cut ck_cut(const ChunkParams &p, int b, long long base, long long pos, long long share) {
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
// Loads that stay where they are written: the compiler would move them down to where their
// values are used, a whole phase of a code warp later.
__device__ __forceinline__ uint4 ck_load16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float ck_load4(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int ck_load4(const int *p) {
    int v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ck_codes_f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
// 16 codes in bf16
__device__ __forceinline__ void ck_bf16(const uint4 w, uint32_t (&y)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = ck_codes_f16x2(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        y[i] = pack_bf16x2(f.x, f.y);
    }
}
// 16 codes times a factor (in both halves of a word), in fp16
__device__ __forceinline__ void ck_f16(const uint4 w, uint32_t factor, uint32_t (&y)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = ck_codes_f16x2(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&factor));
        y[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
}
// 16 codes times 1: half of the conversion's instructions less
__device__ __forceinline__ void ck_f16(const uint4 w, uint32_t (&y)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = ck_codes_f16x2(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
}
constexpr uint32_t kCkOnes = 0x3c003c00u;
// 2^e in fp16 (0 below 2^-24), in both halves of a word; e <= 15
__device__ __forceinline__ uint32_t ck_f16_two_to(int e) {
    const uint32_t h = e >= -14 ? (uint32_t)(e + 15) << 10 : (e >= -24 ? 1u << (e + 24) : 0u);
    return h | h << 16;
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
// registers -> TMEM, 8 consecutive columns per thread, and its wait
__device__ __forceinline__ void ck_tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t ck_pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Words of shared memory by their 32-bit addresses (pointers would be two registers each, in every role).
__device__ __forceinline__ uint32_t ck_get(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void ck_put(uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }

// Raises the block's abort flag, which makes its other waits give up, and the status word.
__device__ __forceinline__ bool ck_give_up(uint32_t abort_flag) {
    ck_put(abort_flag, 1u);
    atomicExch(&g_status_chunk, (int)FA_ERR_TIMEOUT);
    return false;
}
// A wait bounded in time.  The clock is read every 64 tries only, so that the thirty of them are a few instructions each.
__device__ __forceinline__ bool ck_wait(uint32_t bar, uint32_t parity, uint32_t abort_flag, uint32_t limit_us) {
    uint32_t tries = 0, since = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (ck_get(abort_flag) != 0u) return false;
        if ((++tries & 63u) == 0u) {
            const uint32_t now = (uint32_t)(global_timer_ns() >> 10);  // about microseconds
            if (tries == 64u) since = now;
            if (now - since > limit_us) return ck_give_up(abort_flag);
        }
    }
    return true;
}
// 16 bytes from global to shared memory, or zeros in place of what lies behind the first `bytes`
__device__ __forceinline__ void ck_copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ck_copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float ck_two_to(int e) { return __uint_as_float((uint32_t)(max(-126, min(127, e)) + 127) << 23); }

// Of 32 columns of a row, from column 32 c on, those that are NaN because one of the keys [from, to) has a NaN
// value there (the MMA had zeros in their place: another row may not see the key).  Rare.
template <int D>
__device__ __forceinline__ uint32_t ck_nan_columns(const ChunkParams &p, int b, int h, int from, int to, int c) {
    uint32_t mask = 0;
#pragma unroll 1
    for (int j = from; j < to; ++j) {
        const int pg = p.table[(long long)b * p.max_pages + (j >> p.page_log2)];
        if (pg < 0 || pg >= p.num_pages) continue;
        const unsigned long long row = ((unsigned long long)((uint32_t)pg * p.Hkv + h) << p.page_log2) + (j & ((1 << p.page_log2) - 1));
        const uint32_t *const v = reinterpret_cast<const uint32_t *>(p.v_pages + row * D + c * 32);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint32_t nan = ck_nan_codes(v[i]) >> 7;  // a bit a byte
            mask |= ((nan & 1u) | (nan >> 7 & 2u) | (nan >> 14 & 4u) | (nan >> 21 & 8u)) << (4 * i);
        }
    }
    return mask;
}

// Several MMAs in a row, issued by one elected lane of a converged warp under one election (one for each, with
// its operands brought into uniform registers one by one, took twice the instructions, and the issuing warp is
// on the critical path of every tile).
// S (128 x 128, fresh) = Q K^T over D = 64 C: C chunks of 64 columns, four steps of 32 bytes each.
template <int D>
__device__ __forceinline__ void ck_mma_s(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
            "elect.sync _|p, 0xffffffff;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\tadd.s64 a5, %1, 1026;\n\t"
            "add.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 1024;\n\tadd.s64 b5, %2, 1026;\n\t"
            "add.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, 1;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "elect.sync _|p, 0xffffffff;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    }
}
// O (+)= P V over 64 keys: four steps of 16 keys (8 columns of P, 2048 bytes of V)
__device__ __forceinline__ void ck_mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = sbase + C::OFF_BAR;
    auto bar = [&](uint32_t i) { return bars + 8u * i; };
    // words of it: flags and exponents of tiles and segments
    const uint32_t abort_flag = bars + kSlotAbort;
    auto wide_at = [&](int tile) { return bars + kSlotWide + (tile & 15) * 4; };
    auto key_exp_at = [&](int tile) { return bars + kSlotKeyExp + (tile & 15) * 4; };
    auto rest_at = [&](int tile) { return bars + kSlotRest + (tile & 15) * 64; };  // [k, v][8 pieces]
    auto lift_at = [&](int tile) { return bars + kSlotLift + (tile & 15) * 4; };
    auto flags_at = [&](int tile) { return bars + kSlotFlags + tile % kCkTiles * 4; };
    auto pieces_at = [&](int tile) { return bars + kSlotPieces + tile % kCkTiles * 128; };
    auto exp_at = [&](int seg) { return bars + kSlotExp + seg % kCkSegs * 4; };
    auto nan_at = [&](int seg) { return bars + kSlotNan + seg % kCkSegs * 4; };
    auto seg_at = [&](int seg) { return bars + kSlotSegs + seg % kCkSegs * (uint32_t)sizeof(Seg); };
#define CK_SEG(at, field) ((int)ck_get((at) + (uint32_t)offsetof(Seg, field)))

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(C_Q_FULL + t), 128);
            mbar_init(bar(C_S_FULL + t), 1);
            mbar_init(bar(C_P_HALF + t), 128);
            mbar_init(bar(C_P_FULL + t), 128);
            mbar_init(bar(C_PH_DONE + t), 1);
            mbar_init(bar(C_O_DONE + t), 1);
            mbar_init(bar(C_O_FREE + t), 128);
        }
        for (int s = 0; s < C::ST; ++s) {
            mbar_init(bar(C_K_FULL + s), kCkCodeWarps);  // a lane of each warp
            mbar_init(bar(C_K_EMPTY + s), 2);    // both MMA warps
            mbar_init(bar(C_V_FULL + s), kCkCodeWarps);
            mbar_init(bar(C_V_EMPTY + s), 2);
        }
        for (int s = 0; s < kCkSegs; ++s) {
            mbar_init(bar(C_SEG_FULL + s), 1);
            mbar_init(bar(C_SEG_FREE + s), 8 + 2 + 1);  // softmax, MMA, tiles
            ck_put(nan_at(s), 0u);
        }
        for (int s = 0; s < kCkTiles; ++s) {
            mbar_init(bar(C_TILE_FULL + s), 1);
            mbar_init(bar(C_TILE_FREE + s), kCkCodeWarps);
        }
        mbar_init(bar(C_DRAIN), 2);
        ck_put(abort_flag, 0u);
        fence_mbar_init();
    }
    if (warp == 16) {
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
            cut_sm[e].b = b;
            cut_sm[e].begin = base;
        }
        __syncthreads();
        if (lane == 0 && warp < 2 && cut_sm[warp].begin != LLONG_MAX)
            cut_sm[warp] = ck_cut(p, cut_sm[warp].b, cut_sm[warp].begin, ((long long)blockIdx.x + warp) * share, share);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ck_get(bars + kSlotTmem);
    const uint32_t limit_us = p.limit_us;
    auto wait = [&](uint32_t b, uint32_t parity) {
        return ck_wait(bar(b), parity, abort_flag, limit_us);
    };
    auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
    // Segment n of the block, once it is there.  With a limit of 0 nobody waits for one, whatever has happened by then (a single
    // try may itself wait, so that whether it fails says little; all roles come by here, and not in their loops over tiles).
    auto segment = [&](int n) -> int {
        if (limit_us == 0u) return ck_give_up(abort_flag);
        return wait_all(C_SEG_FULL + n % kCkSegs, (uint32_t)(n / kCkSegs) & 1u);
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C_SEG_FREE + n % kCkSegs));
    };

    if (warp >= 16) {
        regs_decrease<kCkRegsOther>();
        if (warp == 17) {
            // ================================================= segments
            Cut at = cut_sm[0];
            const Cut end = cut_sm[1];
            const long long share = share_sm;
            // Both cuts before the same tile inside an item (the line weighs rows that see no key too, so that a share may be less
            // than a tile): the join counts this block's part all the same, and is to find that it holds nothing.
            if (at.begin == end.begin && at.begin != LLONG_MAX && at.done > 0 && at.done == end.done)
                for (int r = lane; r < kCkRows; r += 32) ck_slot(p.ws, gridDim.x, blockIdx.x, 0, D)[(size_t)kCkRows * (D + 1) + r] = 0.f;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int place = n % kCkSegs;
                if (n >= kCkSegs) ok = wait_all(C_SEG_FREE + place, (uint32_t)(n / kCkSegs - 1) & 1u);
                if (!ok) break;
                const bool more = at.begin < end.begin || (at.begin == end.begin && at.begin != LLONG_MAX && at.done < end.done);
                const long long begin = at.begin;
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
                    if (at.begin == end.begin)
                        at = end;
                    else
                        ck_next(p, at);
                }
                if (lane == 0) {
                    *reinterpret_cast<Seg *>(smem_raw + (seg_at(n) - raw)) = g;
                    mbar_arrive(bar(C_SEG_FULL + place));
                }
                __syncwarp();
                if (more && g.slot == 1) {  // how many blocks have a part of it
                    const int i = g.row0 / kCkRows, tiles = ck_tiles(p, g.c, min(g.rows, g.row0 + kCkRows) - 1);
                    const long long w = ck_begin(p, i + 1, g.c) - ck_begin(p, i, g.c);
                    int parts = 0;
                    for (int j0 = 1; parts == 0; j0 += 32) {
                        const int j = j0 + lane;  // the j-th block behind has its last part, if its end is not in it
                        const long long pos = ((long long)blockIdx.x + j + 1) * share;
                        const bool last_one = pos >= begin + w || (int)blockIdx.x + j + 1 >= (int)gridDim.x ||
                                              ck_done(pos, begin, w, tiles, share) >= tiles;
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
                if (!more) break;
            }
        } else if (warp == 18) {
            // ================================================= tiles
            // Four tiles of a segment at a time, lane 8 j + i for piece i of the j-th.
            const int j = lane >> 3, i = lane & 7;
            auto exponent = [](float x) { return max((int)(__float_as_uint(x) >> 23 & 0xffu) - 127, -126); };
            constexpr int kNone = -127;  // below every exponent
            auto top_of_tile = [](int x) {
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
                return x;
            };
            int tile = 0;
            bool ok = true, end = false;
            for (int n = 0; ok && !end; ++n) {
                ok = segment(n);
                if (!ok) break;
                const uint32_t g = seg_at(n);
                end = CK_SEG(g, end) != 0;
                const int N = CK_SEG(g, t1) - CK_SEG(g, t0), t1 = CK_SEG(g, t1), len = CK_SEG(g, len), h = CK_SEG(g, h);
                const int edge = CK_SEG(g, c) + CK_SEG(g, row0) / p.G + 1;  // keys that the item's first row sees
                const int *const table = p.table + (long long)CK_SEG(g, b) * p.max_pages;
                release(n);
                int e_ref = kNone;
                for (int it = 0; it < N || end; it += 4) {  // (behind the last segment: one more "tile" that says so)
                    const int some = end ? 1 : min(4, N - it), key = (t1 - 1 - it - j) * kCkTile + 16 * i;
                    int ph = -2;  // page * Hkv + head; -2: no keys, -1: outside the cache
                    bool nan = false;  // keys that make the rows that see them NaN
                    float ks = 1.f, vs = 1.f;
                    if (!end && j < some && key < len) {
                        ph = table[key >> p.page_log2];
                        if (ph >= 0 && ph < p.num_pages) {
                            ph = ph * p.Hkv + h;
                            ks = p.k_scale[ph];
                            vs = p.v_scale[ph];
                            nan = !(fabsf(ks) < INFINITY);
                            if (nan) ks = 1.f;
                        } else {
                            ph = -1, nan = true;
                            atomicExch(&g_status_chunk, (int)FA_ERR_BAD_PAGE);
                        }
                    }
                    const bool there = ph >= 0;
                    const int ek = exponent(ks), ev = exponent(vs);
                    const int e_tile = top_of_tile(there && !nan ? ek : -126), v_tile = top_of_tile(there && vs > 0.f && vs < INFINITY ? ev : kNone);
                    if (e_ref == kNone) {
                        const uint32_t has = __ballot_sync(0xffffffffu, v_tile != kNone);
                        if (has) e_ref = __shfl_sync(0xffffffffu, v_tile, __ffs((int)has) - 1);
                    }
                    int unit = e_ref == kNone ? 0 : e_ref, before = unit;  // of this lane's tile, and of the one before it
                    if (__any_sync(0xffffffffu, e_ref != kNone && v_tile - e_ref > kCkLift)) {
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const int last = e_ref, top = __shfl_sync(0xffffffffu, v_tile, 8 * k);
                            if (top - e_ref > kCkLift) e_ref = top;
                            if (k == j) unit = e_ref, before = last;
                        }
                    }
                    // 2: weights times value scales need bf16's range, 1: other than powers of two, keys' far apart, or a unit that goes up
                    const int other = top_of_tile(!there ? 0 : ev - unit > kCkUp || unit - ev > kCkDown || !(vs < INFINITY) ? 2 :
                                                  ks * ck_two_to(-ek) != 1.f || e_tile - ek > kCkDown || vs * ck_two_to(-ev) != 1.f || before != unit ? 1 : 0);
                    const bool wide = other == 2;
                    // the tiles' places in the rings
#pragma unroll 1
                    for (int k = 0; ok && k < some; ++k)
                        if (tile + k >= kCkTiles) ok = wait_all(C_TILE_FREE + (tile + k) % kCkTiles, (uint32_t)((tile + k) / kCkTiles - 1) & 1u);
                    if (!ok) break;
                    const int m = tile + j;
                    if (j < some) {
                        const uint32_t row = ((uint32_t)max(ph, 0) << p.page_log2) + (key & ((1 << p.page_log2) - 1));
                        const uint32_t kf = nan ? 0x7e007e00u : other ? kCkOnes : ck_f16_two_to(min(ek - e_tile, 0));
                        st_shared_v4(pieces_at(m) + i * (uint32_t)sizeof(Piece), row, there ? min(len - key, 16) : 0, kf, ck_f16_two_to(min(ev - unit, kCkUp)));
                        if (other) {
                            ck_put(rest_at(m) + i * 4, __float_as_uint(ks * ck_two_to(-e_tile)));
                            ck_put(rest_at(m) + 32 + i * 4, __float_as_uint(there ? vs * ck_two_to(wide ? -unit : -ev) : 1.f));
                            if (i == 0) ck_put(lift_at(m), __float_as_uint(ck_two_to(before - unit)));
                        }
                        if (i == 0) {
                            ck_put(wide_at(m), wide);
                            ck_put(key_exp_at(m), __float_as_uint(other ? -ck_two_to(e_tile) : ck_two_to(e_tile)));
                            // 1: no more tiles, 2: a row does not see some of its keys, 4: values as they are, 8 *: its segment
                            ck_put(flags_at(m), (end ? 1u : 0u) | (key + kCkTile > edge ? 2u : 0u) | (wide ? 4u : 0u) | (uint32_t)n << 3);
                            if (j == 0) ck_put(exp_at(n), e_ref == kNone ? 0u : (uint32_t)e_ref);  // (read when the segment's last tile is through)
                        }
                    }
                    __syncwarp();
                    if (j < some && i == 0) mbar_arrive(bar(C_TILE_FULL + m % kCkTiles));
                    tile += some;
                    if (end) break;
                }
            }
        } else {
            // ================================================= MMA issuers
            const int t = warp == 16 ? 0 : 1;
            const uint64_t dq = sw128_desc(sbase + t * C::QT_BYTES, 16, 1024);
            const uint64_t dk = sw128_desc(sbase + C::OFF_K, 16, 1024);
            const uint64_t dv = sw128_desc(sbase + C::OFF_V, C::CHUNK, 1024);
            const uint32_t s_tm = tmem + t * 128, o_tm = tmem + C::TM_O + t * D;
            int items = 0, stage = 0, tile = 0;  // items that the sub-tile took part in; stage of K and V; tiles so far
            uint32_t phase = 0, pv_phase = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = segment(n);
                if (!ok) break;
                const uint32_t g = seg_at(n);
                const int N = CK_SEG(g, t1) - CK_SEG(g, t0), end = CK_SEG(g, end), first = t ? CK_SEG(g, first[1]) : CK_SEG(g, first[0]);
                release(n);
                if (end) break;
                // Tiles that the sub-tile sees nothing of: it waits for both fills, so that its arrivals are for this use.
                int it = 0;
#pragma unroll 1
                for (; it < min(first, N); ++it, ++tile) {
                    ok = wait_all(C_K_FULL + stage, phase) && wait_all(C_V_FULL + stage, phase);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive(bar(C_K_EMPTY + stage));
                        mbar_arrive(bar(C_V_EMPTY + stage));
                    }
                    __syncwarp();
                    if (++stage == C::ST) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                if (it == N) continue;
                // The others: S of the first; then for each O += P V in two halves of 64 keys, the first as soon as the softmax
                // has written it, and S of the next right behind the second half.  Whatever else is waited
                // for is waited for while the softmax works.  (An item's first product overwrites O, which has been
                // read out.)
                ok = wait_all(C_K_FULL + stage, phase) && wait_all(C_Q_FULL + t, (uint32_t)items & 1u);
                if (!ok) break;
                tc_fence_after();
                ck_mma_s<D>(s_tm, dq, dk + ((stage * C::KV_BYTES) >> 4), C::IDESC_S);
                tc_commit(bar(C_S_FULL + t));
                tc_commit(bar(C_K_EMPTY + stage));
                if (items > 0) ok = wait_all(C_O_FREE + t, (uint32_t)(items - 1) & 1u);
                if (!ok) break;
                uint32_t more = 0;
#pragma unroll 1
                for (; it < N; ++it, ++tile) {
                    const int next = stage + 1 == C::ST ? 0 : stage + 1;
                    const uint32_t next_phase = next ? phase : phase ^ 1u;
                    const bool last = it == N - 1;
                    const uint32_t idesc = ck_get(wide_at(tile)) ? C::IDESC_PV_BF16 : C::IDESC_PV;
                    const uint64_t dvs = dv + ((stage * C::KV_BYTES) >> 4), dks = dk + ((next * C::KV_BYTES) >> 4);
                    ok = wait_all(C_V_FULL + stage, phase) && wait_all(C_P_HALF + t, pv_phase);
                    if (!ok) break;
                    tc_fence_after();
                    ck_mma_pv(o_tm, s_tm, dvs, idesc, more);
                    tc_commit(bar(C_PH_DONE + t));
                    // (the next tile's codes may not be looked up before this one's segment ends: waited for only within it)
                    if (!last) ok = wait_all(C_K_FULL + next, next_phase);
                    ok = ok && wait_all(C_P_FULL + t, pv_phase);
                    if (!ok) break;
                    tc_fence_after();
                    ck_mma_pv(o_tm, s_tm + 32, dvs + ((64 * 128) >> 4), idesc, 1u);
                    if (!last) {
                        ck_mma_s<D>(s_tm, dq, dks, C::IDESC_S);
                        tc_commit(bar(C_S_FULL + t));
                        tc_commit(bar(C_K_EMPTY + next));
                    } else {
                        tc_commit(bar(C_O_DONE + t));
                    }
                    tc_commit(bar(C_V_EMPTY + stage));
                    pv_phase ^= 1u;
                    more = 1;
                    stage = next, phase = next_phase;
                }
                if (!ok) break;
                ++items;
            }
            tc_commit(bar(C_DRAIN));
            mbar_wait_drain(bar(C_DRAIN), 0, kCkDrainNs);
        }
    } else if (warp >= 8) {
        // ===================================================== codes
        regs_decrease<kCkRegsCodes>();
        const int cw = warp - 8;  // takes the tile's keys 16 cw .. 16 cw + 15, which are in one page
        // A load's lanes: pairs of rows in which eight lanes cover the same 64 columns (four
        // pieces of 16 codes), so that what they write falls into different banks.
        const int ld_row = 2 * (D == 128 ? lane >> 4 : lane >> 3) + ((lane >> 2) & 1);
        const int ld_piece = (lane & 3) + (D == 128 ? (lane >> 3 & 1) * 4 : 0);
        constexpr int LD_ROWS = D == 128 ? 4 : 8;
        // (Spilled registers would go to the L2: the cache beside this much shared memory is small.)
        uint32_t flags = 0, row = 0, kf = 0, vf = 0;   // of the tile being worked on
        int valid = 0;
        uint4 kr[C::LOADS], vr[C::LOADS];
        const uint32_t lane_at = ld_row * D + ld_piece * 16;
        auto load = [&](const uint8_t *pages, uint4 (&r)[C::LOADS]) {
            const uint8_t *const src = pages + (unsigned long long)row * D + lane_at;
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                r[i] = make_uint4(0, 0, 0, 0);
                if (i * LD_ROWS + ld_row < valid) r[i] = ck_load16(src + i * LD_ROWS * D);
            }
        };
        // Where this lane's 32 bytes of a row go: two pieces of 16, swapped within 128 bytes by the row.  Its rows are LD_ROWS
        // (a multiple of 4) apart, so that their swaps differ in one bit at most.
        const uint32_t to = (ld_piece >> 2) * C::CHUNK + (16 * cw + ld_row) * 128, piece = 2 * (ld_piece & 3);
        const uint32_t to0 = to + ((piece ^ (ld_row & 7)) << 4), to1 = to + (((piece + 1) ^ (ld_row & 7)) << 4);
        auto store = [&](uint32_t base, int i, const uint32_t (&y)[8]) {
            const uint32_t flip = (i * LD_ROWS & 7) << 4, down = i * LD_ROWS * 128;
            st_shared_v4(base + (to0 ^ flip) + down, y[0], y[1], y[2], y[3]);
            st_shared_v4(base + (to1 ^ flip) + down, y[4], y[5], y[6], y[7]);
        };
        auto hand_over = [&](uint32_t b) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        // Takes up tile m, which has been looked up: asks for its K.  Returns whether there is one.
        auto take_up = [&](int m) {
            flags = ck_get(flags_at(m));
            uint32_t some;
            ld_shared_v4(pieces_at(m) + cw * (uint32_t)sizeof(Piece), row, some, kf, vf);
            valid = (int)some;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_TILE_FREE + m % kCkTiles));
            if (flags & 1u) return false;
            load(p.k_pages, kr);
            return true;
        };
        bool ok = wait_all(C_TILE_FULL, 0);
        bool have = ok && take_up(0);
        if (have) load(p.v_pages, vr);
        int st = 0;
        uint32_t use = 1;   // parity of what the stage's last use leaves when it is done (passes at the first)
#pragma unroll 1
        for (int n = 0; have; ++n) {
            // ---- K of the tile; then the next one's is asked for, if it has been looked up (it may not be before this
            // tile is done: segments' places in the ring are free when the softmax is through with them)
            ok = wait_all(C_K_EMPTY + st, use);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                uint32_t y[8];
                if (kf == kCkOnes)  // (the tile's largest scale, as mostly: 744 us instead of 754 for 1,024 tokens behind 65,536 keys)
                    ck_f16(kr[i], y);
                else
                    ck_f16(kr[i], kf, y);
                store(sbase + C::OFF_K + st * C::KV_BYTES, i, y);
            }
            hand_over(C_K_FULL + st);
            const uint32_t now = flags, v_factor = vf;
            const uint32_t next = C_TILE_FULL + (n + 1) % kCkTiles, next_phase = (uint32_t)((n + 1) / kCkTiles) & 1u;
            const bool early = __all_sync(0xffffffffu, mbar_try_wait(bar(next), next_phase));
            if (early) have = take_up(n + 1);
            // ---- V of the tile
            ok = wait_all(C_V_EMPTY + st, use);
            if (!ok) break;
            if (__builtin_expect((now & 6u) == 0, 1)) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    uint32_t y[8];
                    ck_f16(vr[i], v_factor, y);
                    store(sbase + C::OFF_V + st * C::KV_BYTES, i, y);
                }
            } else {
                bool nan = false;
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    uint32_t y[8];
                    if (now & 2u) nan |= ck_without_nan(vr[i]);  // they must not reach the rows that do not see them
                    if (now & 4u)
                        ck_bf16(vr[i], y);
                    else
                        ck_f16(vr[i], v_factor, y);
                    store(sbase + C::OFF_V + st * C::KV_BYTES, i, y);
                }
                if (nan) ck_put(nan_at(now >> 3), (now >> 3) + 1u);
            }
            hand_over(C_V_FULL + st);
            if (!early) {
                ok = wait_all(next, next_phase);
                if (!ok) break;
                have = take_up(n + 1);
            }
            if (have) load(p.v_pages, vr);
            if (++st == C::ST) st = 0, use ^= 1u;
        }
    } else {
        // ============================================ softmax warpgroups
        regs_increase<kCkRegsSoftmax>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lane_off + t * 128;
        const uint32_t o_tm = tmem + lane_off + C::TM_O + t * D;
        int ns = 0, od = 0, tile = 0;  // S tiles and items of this sub-tile, tiles of the block so far
        bool ok = true;
        // The row's query of segment n, scaled to fp16, into shared memory, where the last S of the segment before (or of
        // the one before that) has read the one that was there.  Returns the row's factor of the scores.
        auto load_query = [&](int n) -> float {
            float c_row = p.scale_log2;
            ok = segment(n);
            if (!ok) return c_row;
            const uint32_t g = seg_at(n);
            const int first = t ? CK_SEG(g, first[1]) : CK_SEG(g, first[0]);
            if (CK_SEG(g, end) || first >= CK_SEG(g, t1) - CK_SEG(g, t0)) return c_row;
            // The warp's 32 rows into shared memory as they are, two to four whole rows with each load; then each lane
            // scales its own row there.  (A row a lane, whose loads touch 32 lines each: 311 us for the prompts instead of 303, 132 instead of 128
            // for 512 tokens behind 16384.)
            constexpr int LANES = D / 8, ROWS = 32 / LANES;
            const int rows = CK_SEG(g, rows), piece = lane % LANES, from = (warp & 3) * 32 + lane / LANES, R = CK_SEG(g, row0) + t * 128 + from;
            int tok = R / p.G, head = R - tok * p.G;
            const int more_tok = ROWS / p.G, more_head = ROWS - more_tok * p.G;
            const __nv_bfloat16 *const src = static_cast<const __nv_bfloat16 *>(p.q) + (long long)CK_SEG(g, q0) * p.q_stride + (long long)CK_SEG(g, h) * p.G * D + piece * 8;
            const uint32_t at = sbase + t * C::QT_BYTES + (piece >> 3) * C::CHUNK + from * 128;
#pragma unroll 2
            for (int i = 0; i < LANES; ++i) {
                const bool there = R + i * ROWS < rows;  // zeros behind the last row
                ck_copy16(at + i * ROWS * 128 + (((piece ^ (from + i * ROWS)) & 7) << 4), src + (there ? tok * p.q_stride + (long long)head * D : 0), there ? 16 : 0);
                tok += more_tok, head += more_head;
                if (head >= p.G) head -= p.G, ++tok;
            }
            ck_copies_wait();
            __syncwarp();
            const uint32_t dst = sbase + t * C::QT_BYTES + row * 128;
            uint32_t am = 0;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint32_t w[4];
                ld_shared_v4(dst + (i >> 3) * C::CHUNK + (((i ^ row) & 7) << 4), w[0], w[1], w[2], w[3]);
                am = __vmaxu2(am, __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu)));
            }
            am = max(am & 0xffffu, am >> 16);
            const int e = am ? max(-126, min(126, (int)(am >> 7) - 127)) : 0;
            const float down = ck_two_to(-e);
            c_row *= ck_two_to(e);
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t to = dst + (i >> 3) * C::CHUNK + (((i ^ row) & 7) << 4);
                uint32_t w[4];
                ld_shared_v4(to, w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = ck_pack_f16(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xffff0000u) * down);
                st_shared_v4(to, w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(C_Q_FULL + t));
            return c_row;
        };
        float c_row = 0.f, c_next;
        for (int n = -1; ok; ++n, c_row = c_next) {  // (a first pass takes the first segment's query only)
            const uint32_t g = seg_at(max(n, 0));    // (released behind the epilogue, which reads it again)
            const int N = n < 0 ? 0 : CK_SEG(g, t1) - CK_SEG(g, t0), first = n < 0 ? 0 : t ? CK_SEG(g, first[1]) : CK_SEG(g, first[0]);
            // (What only the rarer paths need is read again there: registers are short in this loop.)
            auto limit_of_row = [&]() {  // keys that this row sees
                return CK_SEG(g, c) + min(CK_SEG(g, row0) + t * 128 + row, CK_SEG(g, rows) - 1) / p.G + 1;
            };
            // from which tile on every row of the sub-tile sees all keys: those up to its first row's limit
            const int plain_from = CK_SEG(g, t1) - max(0, CK_SEG(g, c) + (CK_SEG(g, row0) + t * 128) / p.G + 1) / kCkTile;
            tile += min(first, N);
            float m_used = -INFINITY, l_run = 0.f;
            bool ready = false;  // every row of the warp has a maximum
            for (int it = first; it < N; ++it, ++tile) {
                ok = wait_all(C_S_FULL + t, (uint32_t)ns & 1u);
                if (!ok) break;
                ++ns;
                tc_fence_after();
                // ---- the ordinary tile: no mask, fp16, and a maximum that holds.  S goes through the registers 16
                // keys at a time, the next two times 16 on their way; P is handed over in halves of 64 keys.
                // (The loops of all roles have to stay in the instruction cache together, so that this
                // one has nothing else in it.)
                const float key_exp = __uint_as_float(ck_get(key_exp_at(tile)));  // negative: the tile goes the other way
                const bool masked = it < plain_from, other = key_exp < 0.f;
                float c_tile = c_row * fabsf(key_exp);
                int half = 0;
                if (!(masked || other) && ready) {
                    uint32_t s[3][16], pk[32];
                    const float nm = kCkShift - m_used;
                    const uint64_t c2 = f2_pack(c_tile, c_tile), nm2 = f2_pack(nm, nm);
                    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
                    tmem_ld16(s_tm, s[0]);
                    half = [&]() {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if (c == 0) tmem_ld16(s_tm + 16, s[1]);
                            if (c < 6) tmem_ld16(s_tm + (c + 2) * 16, s[(c + 2) % 3]);
                            tmem_ld_wait16(s[c % 3]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c % 3][2 * e]), __uint_as_float(s[c % 3][2 * e + 1])), c2, nm2), x0, x1);
                                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                                acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
                                pk[c % 4 * 8 + e] = ck_pack_f16(p0, p1);
                            }
                            if (c % 4 == 3) {
                                float a0, a1, b0, b1;
                                f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
                                f2_unpack(f2_add(acc[2], acc[3]), b0, b1);
                                const float sum = (a0 + a1) + (b0 + b1);
                                // scores have grown past the maximum in use?
                                if (__any_sync(0xffffffffu, !(sum <= kCkMost))) return c / 4;
                                l_run += sum;
                                acc[0] = acc[1] = acc[2] = acc[3] = 0ull;
                                tmem_st16(s_tm + c / 4 * 32, pk);
                                tmem_st16(s_tm + c / 4 * 32 + 16, pk + 16);
                                tmem_st_wait(pk);
                                tc_fence_before();
                                mbar_arrive(bar((c == 3 ? C_P_HALF : C_P_FULL) + t));
                            }
                        }
                        return 2;
                    }();
                    if (half == 2) continue;
                    tmem_ld_wait16(s[0]);
                    tmem_ld_wait16(s[1]);
                    tmem_ld_wait16(s[2]);
                }
                const int lim = limit_of_row() - (CK_SEG(g, t1) - 1 - it) * kCkTile;
                // ---- the others, or the second half of one: the maximum first, then P, 16 keys at a time.  Tiles that go the other
                // way have this code to themselves (with both in one, branches at every 16 keys: prompts 301 us instead of 295, and 697 instead
                // of 518 with scales that are no powers of two).
                // (A factor of 0 would make NaN of masked keys' -infinity.  The sum is another than c_tile only where scores are 0 either way.)
                c_tile += FLT_MIN;
                auto slowly = [&](auto tag) {
                    constexpr bool OTHER = decltype(tag)::value;
                    uint32_t x[16];
                    auto piece = [&](int c) {
                        tmem_ld16(s_tm + c * 16, x);
                        tmem_ld_wait16(x);
                        if constexpr (OTHER) {
                            const float f = __uint_as_float(ck_get(rest_at(tile) + c * 4));
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                        }
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c * 16 + e >= lim) x[e] = __float_as_uint(-INFINITY);
                        }
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = OTHER ? 0 : 4 * half; c < 8; ++c) {
                        piece(c);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) top = max3f(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    }
                    const float m_new = fmaxf(m_used, top * c_tile);
                    ready = __all_sync(0xffffffffu, m_new != -INFINITY);
                    const float factor = m_new == -INFINITY ? 1.f : ex2_approx(m_used - m_new);  // 0 on a row's first keys
                    m_used = m_new;
                    l_run *= factor;
                    const float factor_o = OTHER ? factor * __uint_as_float(ck_get(lift_at(tile))) : factor;
                    if (!OTHER && half == 1) {  // the first half's product must be in O before O is rescaled
                        ok = wait_all(C_PH_DONE + t, (uint32_t)(ns - 1) & 1u);
                        if (!ok) return false;
                        tc_fence_after();
                    }
                    if (((!OTHER && half == 1) || it > first) && __any_sync(0xffffffffu, factor_o != 1.f)) {  // O holds what came before at the old maximum and in the old unit
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            tmem_ld16(o_tm + c * 16, x);
                            tmem_ld_wait16(x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * factor_o);
                            tmem_st16(o_tm + c * 16, x);
                            tmem_st_wait16(x);
                        }
                    }
                    const float nm = m_used == -INFINITY ? 0.f : kCkShift - m_used;  // no key yet: p = 0
#pragma unroll 1
                    for (int c = OTHER ? 0 : 4 * half; c < 8; ++c) {
                        piece(c);
                        uint32_t y[8];
                        float sum = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            x[e] = __float_as_uint(ex2_approx(fmaf(__uint_as_float(x[e]), c_tile, nm)));
                            sum += __uint_as_float(x[e]);
                        }
                        l_run += sum;
                        if constexpr (OTHER) {
                            const float f = __uint_as_float(ck_get(rest_at(tile) + 32 + c * 4));
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                            if (!(fabsf(f) < INFINITY)) {  // keys that the row does not see: 0, whatever their scale
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (c * 16 + e >= lim) x[e] = 0u;
                            }
                        }
                        if (OTHER && ck_get(wide_at(tile))) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = ck_pack_f16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                        }
                        ck_tmem_st8(s_tm + c * 8, y);  // (over scores that are read already)
                        if (c == 3) {
                            tc_fence_before();
                            mbar_arrive(bar(C_P_HALF + t));
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(bar(C_P_FULL + t));
                    return true;
                };
                if (!(other ? slowly(std::true_type()) : slowly(std::false_type()))) break;
            }
            if (!ok) break;
            c_next = load_query(n + 1);  // so that the next segment's first S runs beside what follows
            if (!ok) break;
            if (n < 0) {
                if (CK_SEG(seg_at(0), end)) break;
                continue;
            }
            // ---- the rows' results, 32 columns at a time
            const bool some = first < N;  // the sub-tile has tiles here
            float unit = 1.f;
            bool nan_there = false;
            if (some) {
                ok = wait_all(C_O_DONE + t, (uint32_t)od & 1u);
                if (!ok) break;
                ++od;
                tc_fence_after();
                unit = ck_two_to((int)ck_get(exp_at(n)));
                nan_there = ck_get(nan_at(n)) == (uint32_t)n + 1u;
            }
            const int R = CK_SEG(g, row0) + t * 128 + row, slot = CK_SEG(g, slot);
            const bool there = R < CK_SEG(g, rows), empty = l_run == 0.f;  // empty: no key
            const float inv = empty ? 0.f : 1.f / l_run;
            const int tok = min(R, CK_SEG(g, rows) - 1) / p.G;
            const long long at = (long long)(CK_SEG(g, q0) + tok) * (p.Hkv * p.G) + CK_SEG(g, h) * p.G + (R - tok * p.G);
            float *const part = ck_slot(p.ws, gridDim.x, blockIdx.x, max(slot, 0), D);
            const int r = t * 128 + row;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (some) {
                    tmem_ld32(o_tm + c * 32, o);
                    tmem_ld_wait(o);
                }
                uint32_t nan = 0;
                if (nan_there) {
                    const int from = max(CK_SEG(g, t0), max(0, CK_SEG(g, c) + CK_SEG(g, row0) / p.G + 1) / kCkTile) * kCkTile;
                    nan = ck_nan_columns<D>(p, CK_SEG(g, b), CK_SEG(g, h), from, min(min(limit_of_row(), CK_SEG(g, len)), CK_SEG(g, t1) * kCkTile), c);
                }
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
            if (CK_SEG(seg_at(n + 1), end)) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- the join
// O = sum_s w_s o_s / sum_s w_s with w_s = l_s 2^(m_s - max m), LSE = ln2 (max m - 4 + log2 sum_s w_s), the
// parts in order: a warp a row, D / 32 columns a lane.
constexpr int kCkJoinWarps = 8, kCkJoinBlocks = 16;  // blocks an item, of 8 warps: two rows each (with 8 blocks the chunk of 512 tokens took 7 us more)
template <int D>
__global__ void __launch_bounds__(32 * kCkJoinWarps) fa_fwd_paged_chunk_join(const __grid_constant__ ChunkParams p) {
    grid_wait();
    const CkTail tail = *ck_tail(p.ws, blockIdx.x);
    const int lane = threadIdx.x & 31;
    if (tail.parts == 0) return;
    auto part = [&](int j) { return ck_slot(p.ws, gridDim.x, (int)blockIdx.x + j, j == 0 ? 1 : 0, D); };
#pragma unroll 1
    for (int r = blockIdx.y * kCkJoinWarps + (threadIdx.x >> 5), row = tail.row0 + r; r < kCkRows && row < tail.rows;
         r += kCkJoinWarps * kCkJoinBlocks, row += kCkJoinWarps * kCkJoinBlocks) {
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
}

size_t paged_chunk_workspace_bytes(int D, int num_sms) {
    return (size_t)num_sms * (sizeof(CkTail) + 2 * (size_t)kCkRows * (D + 2) * sizeof(float));
}

template <int D>
static cudaError_t launch_chunk(const ChunkParams &p, int num_sms, cudaStream_t stream) {
    // With fewer registers at launch than the split counts on, the warps that ask for more would wait for ever.  (What was found once
    // holds: the kernel is compiled for one architecture.  A look-up that failed says nothing of the next call's.)
    static std::atomic<bool> split_holds{false};
    cudaError_t e;
    if (!split_holds.load(std::memory_order_relaxed)) {
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, fa_fwd_paged_chunk_kernel<D>);
        if (e != cudaSuccess) return e;
        if (a.numRegs != kCkRegsLaunch) return cudaErrorLaunchOutOfResources;
        split_holds.store(true, std::memory_order_relaxed);
    }
    e = cudaFuncSetAttribute(fa_fwd_paged_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CkCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_early(fa_fwd_paged_chunk_kernel<D>, dim3((unsigned)num_sms), kCkThreads, CkCfg<D>::SMEM, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_early(fa_fwd_paged_chunk_join<D>, dim3((unsigned)num_sms, kCkJoinBlocks), 32 * kCkJoinWarps, 0, stream, 1, p);
}

cudaError_t launch_fwd_paged_chunk(int D, ChunkParams p, int num_sms, cudaStream_t stream) {
    p.max_len = p.max_pages << p.page_log2;
    p.item_keys = (kCkRows + p.G - 1) / p.G;
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
