// fa_paged.cu -- attention of a few query tokens over the paged 8-bit cache
// on GB300 (sm_103a): O = softmax(scale q K^T) V and the row log-sum-exp, K and
// V read as e4m3 codes with one scale for each page and head.
//
// Mathematics.  For a query row r and key j with codes k_j, v_j and their pages'
// scales ks_j, vs_j, in base 2 (c = scale log2 e):
//   x_rj = c ks_j (q_r . k_j) + log2 vs_j,      m_r = max_j x_rj,
//   w_rj = 2^(x_rj - m_r + 14)                   (the weight of the CODES v_j)
//   O_r  = sum_j w_rj v_j / l_r,   l_r = sum_j w_rj / vs_j,
//   LSE_r = ln2 (m_r - 14 + log2 l_r).
// With the value scale inside the exponent the weights are at most 2^14 however
// unevenly the pages are scaled, so they can be rounded to fp16 (to 2^-12 of
// each) with the smallest ones still above fp16's subnormals 2^-24, i.e. 2^-38 of
// the largest; bf16 would keep three bits less.  l sums the unrounded weights in
// fp32.  e4m3 codes are exact in fp16, and a query row is scaled by a power of two
// to a largest element in [1, 2), so that its bf16 values are exact too: both
// products run on fp16 operands with fp32 accumulators, and nothing but w and O is
// rounded.
//
// What bounds it: 2 D bytes read for a key and key/value head and 2 FLOP a byte
// for each query row, so for a few rows (grouped heads, drafts) the HBM stream.
// The products are computed transposed, S^T = K Q^T and O^T = V^T W^T, so that
// the long side of the MMA tile (16) lies along the keys or the head dimension
// and the short one (8) along the few query rows; the tensor cores' 128-row
// tcgen05 tiles would be filled to a sixteenth, wait on TMEM for every tile, and
// need the softmax's row sums across lanes.  Here each warp streams its own
// tiles of 32 keys through a private ring of asynchronous copies and keeps its own
// running maximum and sums: nothing waits for another warp before the end of an
// item.
//
// Split.  The tiles of all items (sequence, key/value head, 8 or 16 query rows)
// are laid end to end and cut into equal shares, one a CTA, whatever the lengths:
// a long sequence is cut over many CTAs, short ones are packed into one.  Lengths
// are read on the device (a scan of a few hundred integers).  An item that is cut
// leaves partial results in the workspace, which a second kernel joins; a CTA has
// at most two of them (the item that it continues, the item that it leaves off).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

static __device__ int g_status_paged = 0;

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgTile = 32;         // keys a tile; two halves of 16, each in one page
constexpr int kPgCtasPerSm = 2;
constexpr int kPgMinShare = 8;      // tiles: two for each warp
constexpr int kPgMaxLen = 0x7fffff00;
constexpr float kPgShift = 14.f;

template <int D>
struct PgCfg {
    static constexpr int CHUNKS = D / 16;                    // 16-byte pieces of a row
    static constexpr int HALF_BYTES = 16 * D;                // 16 rows of K or of V
    static constexpr int STAGE_BYTES = 4 * HALF_BYTES;       // K and V of a tile
    static constexpr int ST = D == 128 ? 3 : 6;              // stages a warp: 96 KB a CTA
    static constexpr int META = 8;                           // words a stage
    static constexpr int OFF_META = kPgWarps * ST * STAGE_BYTES;
    static constexpr int SMEM = OFF_META + kPgWarps * ST * META * 4;
    static constexpr int ROW = D + 4;                        // floats a row of the join buffers
};

// A place in the line of tiles.
struct Place {
    int entry;        // sequence, or sequence * Hkv + head where pages are selected
    long long base;   // first tile of the entry
};

struct Seq {
    int q0, nq, len;
};

__device__ __forceinline__ Seq sequence(const PagedParams &p, int b) {
    Seq s;
    s.q0 = max(0, min(p.cu_q[b], p.T));
    s.nq = max(s.q0, min(p.cu_q[b + 1], p.T)) - s.q0;
    const long long most = min((long long)p.max_pages << p.page_log2, (long long)kPgMaxLen);
    s.len = (int)max(0ll, min((long long)p.seq_lens[b], most));
    return s;
}

// Tiles of one item of (b, h), at least one: an item without keys still writes its rows.
__device__ __forceinline__ int item_tiles(const PagedParams &p, int b, int h, int len) {
    long long keys = len;
    if (p.sel) keys = (long long)max(0, min(p.sel_count[(long long)b * p.Hkv + h], p.sel_width)) << p.page_log2;
    return max(1, (int)((keys + kPgTile - 1) / kPgTile));
}

__device__ __forceinline__ long long entry_weight(const PagedParams &p, int e, int nr) {
    const int b = p.sel ? e / p.Hkv : e, h = p.sel ? e % p.Hkv : 0;
    const Seq s = sequence(p, b);
    if (s.nq == 0) return 0;
    const long long rt = ((long long)s.nq * p.G + nr - 1) / nr;
    return rt * (p.sel ? 1 : p.Hkv) * item_tiles(p, b, h, s.len);
}

// The line of tiles, known to every thread of a block: total and share, and the
// place of one position (given as a function of the share).
struct Line {
    long long total, share;
};

template <class PosOf>
__device__ __forceinline__ Line scan_line(const PagedParams &p, int nr, int ctas, PosOf pos_of, Place &place,
                                          long long *warp_sums, Place *found) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = p.sel ? p.B * p.Hkv : p.B;
    const int per = (n + kPgThreads - 1) / kPgThreads;
    const int e0 = min(n, tid * per), e1 = min(n, e0 + per);
    long long mine = 0;
    for (int e = e0; e < e1; ++e) mine += entry_weight(p, e, nr);
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    Line line;
    line.total = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) x += warp_sums[w];
        line.total += warp_sums[w];
    }
    line.share = (line.total + ctas - 1) / ctas;
    if (line.share < kPgMinShare) line.share = kPgMinShare;
    const long long pos = pos_of(line);
    long long lo = x - mine;
    if (pos >= lo && pos < x) {
        int e = e0;
        for (; e < e1 - 1; ++e) {
            const long long w = entry_weight(p, e, nr);
            if (pos < lo + w) break;
            lo += w;
        }
        found->entry = e;
        found->base = lo;
    }
    __syncthreads();
    place = *found;
    return line;
}

// ------------------------------------------------------------- instructions
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// four 8x8 tiles of 16-bit pairs, transposed: lane l's address is row l of the 32
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where partial results of CTA c lie: slot 0 for the item that it continues, 1
// for the one that it leaves off.  [rows] m, [rows] l, [rows][D] sums.
__device__ __forceinline__ float *slot_of(float *ws, int c, int slot, int nr, int D) {
    return ws + (2ll * c + slot) * nr * (D + 2);
}

__device__ __forceinline__ void write_row(const PagedParams &p, const Seq &s, int h, long long row, int D, int d,
                                          float o, float m, float l) {
    const long long at = (s.q0 + row / p.G) * ((long long)p.Hkv * p.G) + (long long)h * p.G + row % p.G;
    static_cast<__nv_bfloat16 *>(p.o)[at * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
    if (d == 0) {
        // l's exponent is added to m before its mantissa's logarithm: both are near
        // what LSE is not, and would cost it their rounding
        const uint32_t u = __float_as_uint(l);
        const float whole = (float)((int)(u >> 23) - 127) - kPgShift;
        const float frac = log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
        float y = ((m + whole) + frac) * 0.69314718055994531f;
        if (l == 0.f) y = -INFINITY;
        if (!(l < INFINITY)) y = m + l;
        p.lse[at] = y;
    }
}

// --------------------------------------------------------------- the kernel
template <int D, int NT>
__global__ void __launch_bounds__(kPgThreads, kPgCtasPerSm) fa_fwd_paged_kernel(const PagedParams p) {
    using C = PgCfg<D>;
    constexpr int NR = 8 * NT;
    constexpr int KG = D / 64;  // groups of four 16-byte pieces of a row
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ long long warp_sums[kPgWarps];
    __shared__ Place found;
    __shared__ float join_m[kPgWarps][NR], join_l[kPgWarps][NR];
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int page = 1 << p.page_log2;
    const uint32_t ring = smem_u32(sm) + warp * C::ST * C::STAGE_BYTES;
    int *const meta_of = reinterpret_cast<int *>(sm + C::OFF_META) + warp * C::ST * C::META;

    Place place;
    const Line line = scan_line(
        p, NR, gridDim.x, [](const Line &l) { return (long long)blockIdx.x * l.share; }, place, warp_sums, &found);
    long long pos = blockIdx.x * line.share;
    const long long end = min(pos + line.share, line.total);
    while (pos < end) {
        // ---- the item at pos
        int b = place.entry, h = 0;
        if (p.sel) b = place.entry / p.Hkv, h = place.entry % p.Hkv;
        const Seq s = sequence(p, b);
        const long long weight = entry_weight(p, place.entry, NR);
        if (pos >= place.base + weight) {
            place.base += weight;
            ++place.entry;
            continue;
        }
        const int tiles = item_tiles(p, b, h, s.len);
        const long long rts = ((long long)s.nq * p.G + NR - 1) / NR, nth = (pos - place.base) / tiles;
        const int t0 = (int)((pos - place.base) - nth * tiles), t1 = (int)min((long long)tiles, t0 + (end - pos));
        long long rt = nth;
        if (!p.sel) h = (int)(nth / rts), rt = nth % rts;
        const long long row0 = rt * NR, rows = (long long)s.nq * p.G;
        const int n_pages = (s.len + page - 1) >> p.page_log2;
        const long long bh = (long long)b * p.Hkv + h;
        const int n_sel = p.sel ? max(0, min(p.sel_count[bh], p.sel_width)) : 0;
        const int *const table = p.table + (long long)b * p.max_pages;
        const int *const sel = p.sel ? p.sel + bh * p.sel_width : nullptr;
        const int mine = t1 - t0 > warp ? (t1 - t0 - warp + kPgWarps - 1) / kPgWarps : 0;  // this warp's tiles

        // ---- pages: 16 tiles (32 halves) looked up at a time, a half a lane
        // key: the half's first key, kPgMaxLen for none; pg: its page, -1 for one outside the cache
        auto look_up = [&](int i, int &pg, int &key) {
            const int tile = t0 + warp + (i + (lane >> 1)) * kPgWarps;
            const long long at = (long long)tile * kPgTile + (lane & 1) * 16;
            pg = 0;
            key = kPgMaxLen;
            if (tile >= t1) return;
            int pos_in = (int)(at >> p.page_log2);
            if (sel) {
                if (pos_in >= n_sel) return;
                pos_in = sel[pos_in];
                if (pos_in < 0 || pos_in >= n_pages) {
                    pg = -1, key = 0;
                    return;
                }
                key = (pos_in << p.page_log2) + (int)(at & (page - 1));
                if (key >= s.len) {
                    key = kPgMaxLen;
                    return;
                }
            } else {
                if (at >= s.len) return;
                key = (int)at;
            }
            pg = table[pos_in];
            if (pg < 0 || pg >= p.num_pages) pg = -1;
        };
        int pg_now, key_now, pg_next, key_next;
        look_up(0, pg_now, key_now);
        look_up(16, pg_next, key_next);
        int issued = 0;
        auto issue = [&]() {
            if (issued < mine) {
                const uint32_t st = ring + (issued % C::ST) * C::STAGE_BYTES;
                int *const meta = meta_of + (issued % C::ST) * C::META;
                if (issued > 0 && (issued & 15) == 0) {
                    pg_now = pg_next, key_now = key_next;
                    look_up(issued + 16, pg_next, key_next);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int src = ((issued & 15) << 1) + half;
                    const int pg = __shfl_sync(0xffffffffu, pg_now, src), key = __shfl_sync(0xffffffffu, key_now, src);
                    const long long ph = (long long)max(pg, 0) * p.Hkv + h;
                    const long long at = ((ph << p.page_log2) + (key & (page - 1))) * D + lane * 16;
                    const bool none = pg < 0 || key == kPgMaxLen;
                    constexpr int PER = C::HALF_BYTES / 512;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int r = j * (16 / PER) + lane / C::CHUNKS, c = lane % C::CHUNKS;
                        const int n = !none && key + r < s.len ? 16 : 0;  // rows behind the sequence read as 0
                        const int kx = D == 128 ? c ^ ((r & 1) << 2) : c;
                        const int vx = D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
                        cp_async16(st + half * C::HALF_BYTES + r * D + kx * 16, p.k_pages + (none ? 0 : at + j * 512), n);
                        cp_async16(st + (2 + half) * C::HALF_BYTES + r * D + vx * 16, p.v_pages + (none ? 0 : at + j * 512), n);
                    }
                    if (lane < 2) cp_async4(smem_u32(meta + 4 + half * 2 + lane), (lane ? p.v_scale : p.k_scale) + ph);
                    if (lane == 2) meta[half * 2] = key;
                    if (lane == 3) meta[half * 2 + 1] = pg;
                }
            }
            cp_commit();
            ++issued;
        };
#pragma unroll
        for (int i = 0; i < C::ST - 1; ++i) issue();

        // ---- query rows: fragments of Q^T (lane: row g of each tile of 8)
        uint32_t qf[NT][KG][4][2];
        float fac[NT][2];   // c 2^e of the rows 2t, 2t+1, which this lane holds in accumulators
        int lim[NT][2];     // the first key that they do not see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const long long row = row0 + nt * 8 + g;
            uint4 w[KG][2];
            uint32_t am = 0;
#pragma unroll
            for (int i = 0; i < KG; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[i][j] = make_uint4(0, 0, 0, 0);
                    if (row < rows) {
                        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                                 (s.q0 + row / p.G) * p.q_stride +
                                                 ((long long)h * p.G + row % p.G) * D + 16 * (t + 4 * i) + 8 * j;
                        w[i][j] = __ldg(reinterpret_cast<const uint4 *>(q));
                    }
                    const uint32_t u[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) am = max(am, max(u[c] & 0x7fffu, (u[c] >> 16) & 0x7fffu));
                }
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int e = max(-126, min(126, (int)(am >> 7) - 127));
            const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < KG; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t u[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        qf[nt][i][2 * j + c / 2][c & 1] =
                            pack_f16x2(__uint_as_float(u[c] << 16) * down, __uint_as_float(u[c] & 0xffff0000u) * down);
                }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fac[nt][j] = p.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
                const long long r = row0 + nt * 8 + 2 * t + j;
                lim[nt][j] = r < rows ? s.len - s.nq + (int)(r / p.G) + 1 : s.len;
            }
        }
        const int lim_min = s.len - s.nq + (int)(row0 / p.G) + 1;

        float m[NT][2], l[NT][2], acc[C::CHUNKS][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[c][nt][j] = 0.f;
        }

        for (int i = 0; i < mine; ++i) {
            cp_wait<C::ST - 2>();
            __syncwarp();
            issue();  // into the stage that the tile before was read from
            const uint32_t st = ring + (i % C::ST) * C::STAGE_BYTES;
            const int *const meta = meta_of + (i % C::ST) * C::META;

            // ---- S^T = K Q^T: a half of 16 keys an MMA tile.  The order of d within the
            // contraction is free as long as Q's is the same: lane t takes whole 16-byte
            // pieces t and t + 4 of its keys' rows, four MMAs' worth each.
            float sc[2][NT][4];
            float lv[2], inv_vs[2];
            int key[2];
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[half][nt][j] = 0.f;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
                    const int c = t + 4 * kg, x = D == 128 ? c ^ ((g & 1) << 2) : c;
                    const uint32_t at = st + half * C::HALF_BYTES + g * D + x * 16;
                    uint32_t a[4], b8[4];
                    ld_shared_v4(at, a[0], a[1], a[2], a[3]);
                    ld_shared_v4(at + 8 * D, b8[0], b8[1], b8[2], b8[3]);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = codes_f16x2(a[w]), a1 = codes_f16x2(b8[w]);
                        const uint32_t a2 = codes_f16x2(a[w] >> 16), a3 = codes_f16x2(b8[w] >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(sc[half][nt], a0, a1, a2, a3, qf[nt][kg][w][0], qf[nt][kg][w][1]);
                    }
                }
                key[half] = meta[half * 2];
                const bool bad = meta[half * 2 + 1] < 0;
                float ks = __int_as_float(meta[4 + half * 2]);
                if (bad) {
                    ks = __int_as_float(0x7fc00000);
                    if (lane == 0) atomicExch(&g_status_paged, (int)FA_ERR_BAD_PAGE);
                }
                {   // log2 of the value scale, exact for powers of two
                    const int u = bad ? 0x3f800000 : meta[5 + half * 2];
                    lv[half] = fmaxf((float)((u >> 23) - 127) + lg2_approx(__int_as_float((u & 0x7fffff) | 0x3f800000)), -100.f);
                }
                inv_vs[half] = ex2_approx(-lv[half]);
                const bool masked = key[half] + 16 > lim_min;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float y = fmaf(sc[half][nt][j], fac[nt][j & 1] * ks, lv[half]);
                        if (masked && key[half] + g + (j >> 1) * 8 >= lim[nt][j & 1]) y = -INFINITY;
                        sc[half][nt][j] = y;
                        mx[nt][j & 1] = fmaxf(mx[nt][j & 1], y);
                    }
            }
            // ---- running maximum; the sums are scaled where it grew
            bool grew = false;
            float corr[NT][2], off[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y = mx[nt][j];
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                    y = fmaxf(y, m[nt][j]);
                    const float base = y == -INFINITY ? 0.f : y;
                    grew |= y > m[nt][j];
                    corr[nt][j] = ex2_approx(m[nt][j] - base);
                    off[nt][j] = kPgShift - base;
                    m[nt][j] = y;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt][0] *= corr[nt][0];
                    l[nt][1] *= corr[nt][1];
#pragma unroll
                    for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[c][nt][j] *= corr[nt][j & 1];
                }
            }
            // ---- weights, and their transpose as the B operand (keys x rows)
            uint32_t wf[2][NT][2];
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[j] = ex2_approx(sc[half][nt][j] + off[nt][j & 1]);
                        l[nt][j & 1] = fmaf(w[j], inv_vs[half], l[nt][j & 1]);
                    }
                    wf[half][nt][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
                    wf[half][nt][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
                }
            // ---- O^T += V^T W^T.  A pair of bytes is one 16-bit element for ldmatrix, so
            // a transposed tile holds d = 2g, 2g+1 of two neighbouring keys in a register;
            // their bytes are sorted by d before the conversion.
            auto accumulate = [&](auto keep, auto settle) {
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) {
                    float was[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) was[nt][j] = acc[c][nt][j];
                    const int x = D == 128 ? c ^ (lane & 7) : c ^ ((lane >> 1) & 3);
                    uint32_t r[4];
                    ldmatrix_x4_trans(st + 2 * C::HALF_BYTES + lane * D + x * 16, r);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t lo = __byte_perm(keep(r[2 * half], half, 0), 0, 0x3120);
                        const uint32_t hi = __byte_perm(keep(r[2 * half + 1], half, 1), 0, 0x3120);
                        const uint32_t a0 = codes_f16x2(lo), a1 = codes_f16x2(lo >> 16);
                        const uint32_t a2 = codes_f16x2(hi), a3 = codes_f16x2(hi >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(acc[c][nt], a0, a1, a2, a3, wf[half][nt][0], wf[half][nt][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[c][nt][j] = settle(acc[c][nt][j], was[nt][j], nt, j & 1);
                }
            };
            if (max(key[0], key[1]) + 16 <= lim_min || lim_min >= s.len) {
                accumulate([](uint32_t r, int, int) { return r; }, [](float now, float, int, int) { return now; });
            } else {
                // Some rows do not see all of these keys: a weight of 0 would still turn a
                // NaN among the values into NaN, so the values that a token does not see
                // are cleared, a token at a time, and only that token's rows take the
                // result (only the last tiles of a sequence come here).
                const int tok0 = (int)(row0 / p.G), tok1 = (int)min((long long)s.nq - 1, (row0 + NR - 1) / p.G);
                for (int tok = tok0; tok <= tok1; ++tok) {
                    const int limit = s.len - s.nq + tok + 1;
                    bool my[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) my[nt][j] = (row0 + nt * 8 + 2 * t + j) / p.G == tok;
                    accumulate(
                        [&](uint32_t r, int half, int up) {
                            const int k = key[half] + up * 8 + 2 * t;
                            return r & ((k < limit ? 0xffffu : 0u) | (k + 1 < limit ? 0xffff0000u : 0u));
                        },
                        [&](float now, float before, int nt, int j) { return my[nt][j] ? now : before; });
                }
            }
        }
        cp_wait<0>();

        // ---- join the warps
        __syncthreads();
        float *const join = reinterpret_cast<float *>(sm);  // [warp][NR][ROW], over the ring
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y = l[nt][j];
                y += __shfl_xor_sync(0xffffffffu, y, 4);
                y += __shfl_xor_sync(0xffffffffu, y, 8);
                y += __shfl_xor_sync(0xffffffffu, y, 16);
                const int r = nt * 8 + 2 * t + j;
                if (g == 0) {
                    join_m[warp][r] = m[nt][j];
                    join_l[warp][r] = y;
                }
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c)
                    *reinterpret_cast<float2 *>(join + (warp * NR + r) * C::ROW + 16 * c + 2 * g) =
                        make_float2(acc[c][nt][j], acc[c][nt][j + 2]);
            }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        float *const part = slot_of(p.ws, blockIdx.x, t0 == 0 ? 1 : 0, NR, D);
        for (int i = tid; i < NR * D; i += kPgThreads) {
            const int r = i / D, d = i % D;
            float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, join_m[w][r]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kPgWarps; ++w) {
                const float f = ex2_approx(join_m[w][r] - base);
                L = fmaf(join_l[w][r], f, L);
                O = fmaf(join[(w * NR + r) * C::ROW + d], f, O);
            }
            if (whole) {
                if (row0 + r < rows) write_row(p, s, h, row0 + r, D, d, O, base, L);
            } else {
                part[2 * NR + i] = O;
                if (d == 0) part[r] = base, part[NR + r] = L;
            }
        }
        __syncthreads();
        pos += t1 - t0;
    }
}

// Joins the partial results of an item that was cut: block (c, r) has row r of
// the item that CTA c left off, whose other parts are with the CTAs behind it.
template <int D, int NT>
__global__ void __launch_bounds__(kPgThreads) fa_paged_join_kernel(const PagedParams p, int ctas) {
    constexpr int NR = 8 * NT;
    extern __shared__ float weight_of[];  // [ctas]
    __shared__ long long warp_sums[kPgWarps];
    __shared__ Place found;
    __shared__ float red[kPgWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x, r = blockIdx.y;
    Place place;
    const Line line = scan_line(
        p, NR, ctas, [c](const Line &l) { return (c + 1) * l.share - 1; }, place, warp_sums, &found);
    grid_wait();
    const long long edge = (c + 1) * line.share;  // where CTA c ends
    if (edge >= line.total) return;
    int b = place.entry, h = 0;
    if (p.sel) b = place.entry / p.Hkv, h = place.entry % p.Hkv;
    const Seq s = sequence(p, b);
    const int tiles = item_tiles(p, b, h, s.len);
    const long long rts = ((long long)s.nq * p.G + NR - 1) / NR, nth = (edge - 1 - place.base) / tiles;
    const long long first = place.base + nth * tiles, last = first + tiles;  // the item
    if (first < edge - line.share || last <= edge) return;
    long long rt = nth;
    if (!p.sel) h = (int)(nth / rts), rt = nth % rts;
    const long long row = rt * NR + r;
    if (row >= (long long)s.nq * p.G) return;
    const int n = (int)((last - 1) / line.share) - c + 1;  // parts
    float M = -INFINITY;
    for (int i = tid; i < n; i += kPgThreads) {
        const float *part = slot_of(p.ws, c + i, i == 0, NR, D);
        // a part without keys does not count
        const float m = part[NR + r] == 0.f ? -INFINITY : part[r];
        weight_of[i] = m;
        M = fmaxf(M, m);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if (lane == 0) red[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, red[w]);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, O = 0.f;
    const int d = tid;
    for (int i = 0; i < n; ++i) {
        const float *part = slot_of(p.ws, c + i, i == 0, NR, D);
        const float f = ex2_approx(weight_of[i] - base);
        L = fmaf(part[NR + r], f, L);
        if (d < D) O = fmaf(part[2 * NR + r * D + d], f, O);
    }
    if (d < D) write_row(p, s, h, row, D, d, O, base, L);
}

size_t paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int num_sms) {
    (void)B, (void)T, (void)Hq, (void)Hkv;
    return (size_t)num_sms * kPgCtasPerSm * 2 * 16 * (D + 2) * sizeof(float);
}

template <int D, int NT>
static cudaError_t launch_paged(const PagedParams &p, int num_sms, cudaStream_t stream) {
    const int ctas = kPgCtasPerSm * num_sms;
    cudaError_t e = cudaFuncSetAttribute(fa_fwd_paged_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PgCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    fa_fwd_paged_kernel<D, NT><<<ctas, kPgThreads, PgCfg<D>::SMEM, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the join is launched while the first kernel still runs, and waits for its end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 8 * NT);
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = ctas * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_paged_join_kernel<D, NT>, p, ctas);
}

cudaError_t launch_fwd_paged(int D, const PagedParams &p, int num_sms, cudaStream_t stream) {
    // Rows of an item: 8 while a sequence has no more on average, 16 beyond.
    const bool wide = (long long)p.T * p.G > 8ll * p.B;
    if (D == 64) return wide ? launch_paged<64, 2>(p, num_sms, stream) : launch_paged<64, 1>(p, num_sms, stream);
    return wide ? launch_paged<128, 2>(p, num_sms, stream) : launch_paged<128, 1>(p, num_sms, stream);
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
