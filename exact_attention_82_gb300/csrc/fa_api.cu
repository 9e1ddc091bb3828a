// fa_api.cu -- the C ABI declared in include/fa.h: argument checks, TMA
// tensor-map encoding and the launch on the caller's stream.  No device
// memory is allocated here and nothing is synchronised (except in
// fa_device_status, which exists to read the status word).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>

using std::max;
using std::min;

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_paged.h"

namespace {

constexpr unsigned long long kWaitLimitNs = 2ull * 1000 * 1000 * 1000;  // 2 s per wait

thread_local char t_errbuf[256];
thread_local cudaError_t t_last_cuda = cudaSuccess;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

int fail_cuda(cudaError_t e) {
    t_last_cuda = e;
    return FA_ERR_CUDA;
}

bool get_encoder() {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// 3-D map over a [BH, S, D] tensor of bf16 (eb = 2) or 8-bit (eb = 1)
// elements: dims (D, S, BH), box (128 bytes of a row, rows, 1), 128-byte
// swizzle, zero fill outside the tensor.  Being 3-D, a box never reaches into
// the next head's rows.
bool encode_bhsd(CUtensorMap *map, const void *ptr, int D, int S, long long BH, int box_rows, int eb = 2) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {(cuuint64_t)D * eb, (cuuint64_t)S * (cuuint64_t)D * eb};
    const cuuint32_t box[3] = {128u / (cuuint32_t)eb, (cuuint32_t)box_rows, 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = g_encode(map, eb == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                                const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

extern "C" int fa_version(void) { return 100; }  // 0.1.0

extern "C" const char *fa_strerror(int status) {
    const char *s;
    switch (status) {
        case FA_OK: s = "ok"; break;
        case FA_ERR_NULLPTR: s = "a required pointer is NULL"; break;
        case FA_ERR_BAD_SHAPE: s = "bad shape: B, H, Sq, Sk must be >= 1 and sizes in range"; break;
        case FA_ERR_UNSUPPORTED_D: s = "unsupported head dim (64 or 128; 128 for the 8-bit path)"; break;
        case FA_ERR_UNSUPPORTED_CAUSAL: s = "causal must be 0 or 1, and causal needs Sq == Sk"; break;
        case FA_ERR_MISALIGNED: s = "a pointer is not 16-byte aligned"; break;
        case FA_ERR_BAD_SCALE: s = "scale (and each descale) must be finite and > 0"; break;
        case FA_ERR_CUDA: s = "CUDA error"; break;
        case FA_ERR_TIMEOUT: s = "an on-chip wait gave up (bounded-wait timeout)"; break;
        case FA_ERR_ALIAS: s = "an output buffer overlaps an input or the other output"; break;
        case FA_ERR_BAD_WINDOW: s = "window bounds must be >= -1, and a bounded window needs Sq == Sk"; break;
        case FA_ERR_WORKSPACE: s = "workspace missing, not 16-byte aligned, or smaller than required"; break;
        case FA_ERR_BAD_MASK: s = "mask_heads must be 1 or B * H, and pair_stride >= 1"; break;
        case FA_ERR_BAD_PAGE:
            s = "page size must be 16, 32, 64 or 128 (or, from the status word: a page or position outside the cache)";
            break;
        case FA_ERR_SCRATCH_LIMIT:
            s = "needs more scratch than the built-in 16 MiB buffer of fa_fwd_splitkv_noalloc holds; "
                "pass a workspace to fa_fwd_splitkv instead";
            break;
        default: s = "unknown status"; break;
    }
    if (status == FA_ERR_CUDA && t_last_cuda != cudaSuccess)
        snprintf(t_errbuf, sizeof t_errbuf, "%s: %s", s, cudaGetErrorString(t_last_cuda));
    else
        snprintf(t_errbuf, sizeof t_errbuf, "%s", s);
    return t_errbuf;
}

// SMs of the current device (cached per device): persistent forward kernels
// run at most one CTA per SM, and the split-KV heuristic sizes its grid by it.
static int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
        cached[dev] = n;
    }
    return cached[dev];
}

// Checks shared by the forward entry points; FA_OK when the call may launch.
static int check_fwd(const void *q, const void *k, const void *v, const void *o, const float *lse, int B, int H,
                     int Sq, int Sk, int D, float scale) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULLPTR;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA_ERR_MISALIGNED;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1) return FA_ERR_BAD_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED_D;
    if (!isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_SCALE;
    const long long BH = (long long)B * H;
    const long long n_ctas = ((Sq + fa::kCtaRows - 1) / fa::kCtaRows) * BH;
    if (BH > (1ll << 31) || n_ctas > 0x7fffffffll) return FA_ERR_BAD_SHAPE;
    const size_t q_bytes = (size_t)BH * Sq * D * 2, kv_bytes = (size_t)BH * Sk * D * 2;
    const size_t lse_bytes = (size_t)BH * Sq * 4;
    if (overlaps(o, q_bytes, q, q_bytes) || overlaps(o, q_bytes, k, kv_bytes) ||
        overlaps(o, q_bytes, v, kv_bytes) || overlaps(lse, lse_bytes, q, q_bytes) ||
        overlaps(lse, lse_bytes, k, kv_bytes) || overlaps(lse, lse_bytes, v, kv_bytes) ||
        overlaps(lse, lse_bytes, o, q_bytes))
        return FA_ERR_ALIAS;
    return FA_OK;
}

// Encode the maps and launch; arguments already checked.  Key j is allowed
// for query i iff i - wl <= j <= i + wr (a negative bound: unbounded).
static int launch_checked(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Sq,
                          int Sk, int D, float scale, int wl, int wr, void *stream,
                          unsigned long long timeout_ns = kWaitLimitNs, const unsigned char *bmask = nullptr,
                          long long bmask_hstride = 0, int pair_stride = 1) {
    if (!get_encoder()) return fail_cuda(cudaErrorNotSupported);
    const long long BH = (long long)B * H;
    long long n_mblk = (Sq + fa::kCtaRows - 1) / fa::kCtaRows;
    if (bmask) {  // items of one head when query blocks a and a + pair_stride are paired
        const long long n_qb = (Sq + fa::kBlockM - 1) / fa::kBlockM, s = pair_stride;
        const long long whole = n_qb / (2 * s);
        n_mblk = whole * s + (n_qb - 2 * s * whole + 1) / 2;
    }
    CUtensorMap tm_q, tm_k, tm_v;
    if (!encode_bhsd(&tm_q, q, D, Sq, BH, fa::kBlockM) || !encode_bhsd(&tm_k, k, D, Sk, BH, fa::kBlockN) ||
        !encode_bhsd(&tm_v, v, D, Sk, BH, fa::kBlockN))
        return fail_cuda(cudaErrorInvalidValue);
    fa::FwdParams p;
    p.o = o;
    p.lse = lse;
    p.bh_count = (int)BH;
    p.n_items = (int)(n_mblk * BH);
    p.Sq = Sq;
    p.Sk = Sk;
    p.n_mblk = (int)n_mblk;
    p.n_kv = (Sk + fa::kBlockN - 1) / fa::kBlockN;
    p.causal = (wr >= 0 && wl < 0) ? 1 : 0;  // triangular work: longest blocks first
    p.wl = wl < 0 ? -1 : wl;
    p.wr = wr < 0 ? -1 : wr;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_scale = 1.f;
    p.timeout_ns = timeout_ns;
    p.bmask = bmask;
    p.bmask_hstride = bmask_hstride;
    p.pair_stride = pair_stride;
    const cudaError_t e = fa::launch_fwd(D, tm_q, tm_k, tm_v, p, sm_count(), (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    return FA_OK;
}

extern "C" int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Sq,
                      int Sk, int D, float scale, int causal, void *stream) {
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (causal != 0 && causal != 1) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (causal && Sq != Sk) return FA_ERR_UNSUPPORTED_CAUSAL;
    return launch_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, -1, causal ? 0 : -1, stream);
}

extern "C" int fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                             int Sq, int Sk, int D, float scale, int window_left, int window_right,
                             void *stream) {
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (window_left < -1 || window_right < -1) return FA_ERR_BAD_WINDOW;
    if ((window_left >= 0 || window_right >= 0) && Sq != Sk) return FA_ERR_BAD_WINDOW;
    return launch_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, window_left, window_right, stream);
}

extern "C" int fa_fwd_blockmask(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                                int Sq, int Sk, int D, float scale, int window_left, int window_right,
                                const unsigned char *block_mask, int mask_heads, int pair_stride, void *stream) {
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (!block_mask) return FA_ERR_NULLPTR;
    if (window_left < -1 || window_right < -1) return FA_ERR_BAD_WINDOW;
    if ((window_left >= 0 || window_right >= 0) && Sq != Sk) return FA_ERR_BAD_WINDOW;
    const long long BH = (long long)B * H;
    if (mask_heads != 1 && (long long)mask_heads != BH) return FA_ERR_BAD_MASK;
    if (pair_stride < 1) return FA_ERR_BAD_MASK;
    const long long n_qb = (Sq + fa::kBlockM - 1) / fa::kBlockM, n_kb = (Sk + fa::kBlockN - 1) / fa::kBlockN;
    const size_t mask_bytes = (size_t)mask_heads * (size_t)(n_qb * n_kb);
    const size_t o_bytes = (size_t)BH * Sq * D * 2, lse_bytes = (size_t)BH * Sq * 4;
    if (overlaps(block_mask, mask_bytes, o, o_bytes) || overlaps(block_mask, mask_bytes, lse, lse_bytes))
        return FA_ERR_ALIAS;
    // a stride of n_qb or more pairs nothing apart: every block with its neighbour
    const int stride = (int)std::min<long long>(pair_stride, n_qb);
    return launch_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, window_left, window_right, stream, kWaitLimitNs,
                          block_mask, mask_heads == 1 ? 0 : n_qb * n_kb, stride);
}

extern "C" int fa_fwd_fp8(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                          int Sq, int Sk, int D, float scale, int causal, float descale_q, float descale_k,
                          float descale_v, void *stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULLPTR;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA_ERR_MISALIGNED;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1) return FA_ERR_BAD_SHAPE;
    if (D != 128) return FA_ERR_UNSUPPORTED_D;
    if (causal != 0 && causal != 1) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (causal && Sq != Sk) return FA_ERR_UNSUPPORTED_CAUSAL;
    const float sc[4] = {scale, descale_q, descale_k, descale_v};
    for (float x : sc)
        if (!isfinite(x) || !(x > 0.f)) return FA_ERR_BAD_SCALE;
    const float scale_log2 = scale * descale_q * descale_k * 1.4426950408889634f;
    if (!isfinite(scale_log2) || !(scale_log2 > 0.f)) return FA_ERR_BAD_SCALE;
    const long long BH = (long long)B * H;
    const long long n_mblk = (Sq + fa::kCtaRows - 1) / fa::kCtaRows;
    if (BH > (1ll << 31) || n_mblk * BH > 0x7fffffffll) return FA_ERR_BAD_SHAPE;
    const size_t q_bytes = (size_t)BH * Sq * D, kv_bytes = (size_t)BH * Sk * D;
    const size_t o_bytes = 2 * q_bytes, lse_bytes = (size_t)BH * Sq * 4;
    if (overlaps(o, o_bytes, q, q_bytes) || overlaps(o, o_bytes, k, kv_bytes) || overlaps(o, o_bytes, v, kv_bytes) ||
        overlaps(lse, lse_bytes, q, q_bytes) || overlaps(lse, lse_bytes, k, kv_bytes) ||
        overlaps(lse, lse_bytes, v, kv_bytes) || overlaps(lse, lse_bytes, o, o_bytes))
        return FA_ERR_ALIAS;
    if (!get_encoder()) return fail_cuda(cudaErrorNotSupported);
    CUtensorMap tm_q, tm_k, tm_v;
    if (!encode_bhsd(&tm_q, q, D, Sq, BH, fa::kBlockM, 1) || !encode_bhsd(&tm_k, k, D, Sk, BH, fa::kBlockN, 1) ||
        !encode_bhsd(&tm_v, v, D, Sk, BH, fa::kBlockN, 1))
        return fail_cuda(cudaErrorInvalidValue);
    fa::FwdParams p;
    p.o = o;
    p.lse = lse;
    p.bh_count = (int)BH;
    p.n_items = (int)(n_mblk * BH);
    p.Sq = Sq;
    p.Sk = Sk;
    p.n_mblk = (int)n_mblk;
    p.n_kv = (Sk + fa::kBlockN - 1) / fa::kBlockN;
    p.causal = causal;
    p.wl = -1;
    p.wr = causal ? 0 : -1;
    p.scale_log2 = scale_log2;
    p.o_scale = descale_v;
    p.timeout_ns = kWaitLimitNs;
    p.bmask = nullptr;
    p.bmask_hstride = 0;
    p.pair_stride = 1;
    const cudaError_t e = fa::launch_fwd_fp8(tm_q, tm_k, tm_v, p, sm_count(), (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    return FA_OK;
}

// ------------------------------------------------------------- split-KV path
// Keys per split for `splits` ranges: a multiple of the 64-key split tile.
static int split_chunk(int Sk, int splits) {
    const int per = (Sk + splits - 1) / splits;
    return ((per + fa::kSplitTileKeys - 1) / fa::kSplitTileKeys) * fa::kSplitTileKeys;
}

static int resolve_splits(int B, int H, int Sk, int num_splits) {
    const int max_splits = (Sk + fa::kSplitTileKeys - 1) / fa::kSplitTileKeys;
    int s = num_splits;
    if (s <= 0) {
        // Our heuristic: among split counts keeping >= 256 keys per split (up to
        // 256 splits), take the one whose CTAs fill the SMs' last wave best,
        // preferring at least four waves; ties go to fewer splits.
        const long long bh = (long long)B * H;
        const int nsm = sm_count();
        const int cap = max(1, min(256, (Sk + 255) / 256));
        double best = -1.0;
        s = 1;
        for (int c = 1; c <= cap; ++c) {
            const long long ctas = bh * c;
            const long long waves = (ctas + nsm - 1) / nsm;
            double score = (double)ctas / (double)(waves * nsm);
            if (ctas < 4ll * nsm) score *= (double)ctas / (4.0 * nsm);
            if (score > best + 1e-9) {
                best = score;
                s = c;
            }
        }
    }
    s = min(s, max_splits);
    const int chunk = split_chunk(Sk, s);
    return (Sk + chunk - 1) / chunk;  // no empty split
}

static size_t splitkv_bytes(long long BH, int Sq, int D, int splits) {
    const size_t o_bytes = (size_t)BH * splits * Sq * D * sizeof(float);
    const size_t o_pad = (o_bytes + 255) & ~(size_t)255;
    return o_pad + (size_t)BH * splits * Sq * sizeof(float);
}

static bool splitkv_shape_ok(int B, int H, int Sq, int Sk, int D) {
    return B >= 1 && H >= 1 && Sq >= 1 && Sq <= fa::kSplitMaxSq && Sk >= 1 && (D == 64 || D == 128) &&
           (long long)B * H <= 65535;
}

extern "C" int fa_splitkv_num_splits(int B, int H, int Sq, int Sk, int D) {
    if (!splitkv_shape_ok(B, H, Sq, Sk, D)) return FA_ERR_BAD_SHAPE;
    return resolve_splits(B, H, Sk, 0);
}

extern "C" size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int Sq, int Sk, int D, int num_splits) {
    if (!splitkv_shape_ok(B, H, Sq, Sk, D) || num_splits > 256) return 0;
    return splitkv_bytes((long long)B * H, Sq, D, resolve_splits(B, H, Sk, num_splits));
}

static int splitkv_checked(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                           int Sq, int Sk, int D, float scale, int num_splits, void *workspace,
                           size_t workspace_bytes, void *stream, unsigned long long timeout_ns) {
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (Sq > fa::kSplitMaxSq || (long long)B * H > 65535 || num_splits > 256) return FA_ERR_BAD_SHAPE;
    const long long BH = (long long)B * H;
    const int splits = resolve_splits(B, H, Sk, num_splits);
    const size_t need = splitkv_bytes(BH, Sq, D, splits);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t kv_bytes = (size_t)BH * Sk * D * 2, q_bytes = (size_t)BH * Sq * D * 2;
    if (overlaps(workspace, need, q, q_bytes) || overlaps(workspace, need, k, kv_bytes) ||
        overlaps(workspace, need, v, kv_bytes) || overlaps(workspace, need, o, q_bytes) ||
        overlaps(workspace, need, lse, (size_t)BH * Sq * 4))
        return FA_ERR_ALIAS;
    if (!get_encoder()) return fail_cuda(cudaErrorNotSupported);
    CUtensorMap tm_k, tm_v;
    if (!encode_bhsd(&tm_k, k, D, Sk, BH, fa::kSplitTileKeys) || !encode_bhsd(&tm_v, v, D, Sk, BH, fa::kSplitTileKeys))
        return fail_cuda(cudaErrorInvalidValue);
    fa::SplitParams p;
    p.q = q;
    p.o = o;
    p.lse = lse;
    p.o_part = static_cast<float *>(workspace);
    p.lse_part = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                           (((size_t)BH * splits * Sq * D * sizeof(float) + 255) & ~(size_t)255));
    p.Sq = Sq;
    p.Sk = Sk;
    p.chunk = split_chunk(Sk, splits);
    p.splits = splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = timeout_ns;
    const cudaError_t e = fa::launch_splitkv(D, tm_k, tm_v, p, (int)BH, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    return FA_OK;
}

extern "C" int fa_fwd_splitkv(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                              int Sq, int Sk, int D, float scale, int num_splits, void *workspace,
                              size_t workspace_bytes, void *stream) {
    return splitkv_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, num_splits, workspace, workspace_bytes, stream,
                           kWaitLimitNs);
}

extern "C" int fa_selftest_splitkv_timeout(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                                           int H, int Sq, int Sk, int D, float scale, int num_splits,
                                           void *workspace, size_t workspace_bytes,
                                           unsigned long long timeout_ns, void *stream) {
    if (timeout_ns > kWaitLimitNs) return FA_ERR_BAD_SHAPE;
    return splitkv_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, num_splits, workspace, workspace_bytes, stream,
                           timeout_ns);
}

extern "C" int fa_fwd_splitkv_noalloc(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                                      int H, int Sq, int Sk, int D, float scale, int num_splits, void *stream) {
    // Same checks as fa_fwd_splitkv, then the size limit, before any CUDA call.
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (Sq > fa::kSplitMaxSq || (long long)B * H > 65535 || num_splits > 256) return FA_ERR_BAD_SHAPE;
    const size_t need = splitkv_bytes((long long)B * H, Sq, D, resolve_splits(B, H, Sk, num_splits));
    if (need > fa::kNoAllocScratchBytes) return FA_ERR_SCRATCH_LIMIT;
    void *scratch = nullptr;
    const cudaError_t e = fa::splitkv_scratch(&scratch);
    if (e != cudaSuccess) return fail_cuda(e);
    return fa_fwd_splitkv(q, k, v, o, lse, B, H, Sq, Sk, D, scale, num_splits, scratch, fa::kNoAllocScratchBytes,
                          stream);
}

// ------------------------------------------------------------------ backward
static int bwd_checked(const void *q, const void *k, const void *v, const void *o, const float *lse,
                       const void *dout, void *dq, void *dk, void *dv, float *delta, int B, int H, int Sq, int Sk,
                       int D, float scale, int causal, void *stream, unsigned long long timeout_ns) {
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !delta) return FA_ERR_NULLPTR;
    const void *ptrs[10] = {q, k, v, o, lse, dout, dq, dk, dv, delta};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr)) return FA_ERR_MISALIGNED;
    if (B < 1 || H < 1 || Sq < 1 || Sk < 1) return FA_ERR_BAD_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED_D;
    if (causal != 0 && causal != 1) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (causal && Sq != Sk) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (!isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_SCALE;
    const long long BH = (long long)B * H;
    const long long n_qt = (Sq + 127) / 128, n_kt = (Sk + 127) / 128;
    if (n_qt * BH > 0x7fffffffll || n_kt * BH > 0x7fffffffll) return FA_ERR_BAD_SHAPE;
    const size_t qb = (size_t)BH * Sq * D * 2, kb = (size_t)BH * Sk * D * 2, lb = (size_t)BH * Sq * 4;
    // outputs (dq, dk, dv, delta) must not overlap any input or each other
    const void *outs[4] = {dq, dk, dv, delta};
    const size_t out_b[4] = {qb, kb, kb, lb};
    const void *ins[6] = {q, k, v, o, lse, dout};
    const size_t in_b[6] = {qb, kb, kb, qb, lb, qb};
    for (int a = 0; a < 4; ++a) {
        for (int b = 0; b < 6; ++b)
            if (overlaps(outs[a], out_b[a], ins[b], in_b[b])) return FA_ERR_ALIAS;
        for (int b = a + 1; b < 4; ++b)
            if (overlaps(outs[a], out_b[a], outs[b], out_b[b])) return FA_ERR_ALIAS;
    }
    if (!get_encoder()) return fail_cuda(cudaErrorNotSupported);
    CUtensorMap tq, tk, tv, tdo, to, tdq, tdk, tdv;
    if (!encode_bhsd(&tq, q, D, Sq, BH, 128) || !encode_bhsd(&tk, k, D, Sk, BH, 128) ||
        !encode_bhsd(&tv, v, D, Sk, BH, 128) || !encode_bhsd(&tdo, dout, D, Sq, BH, 128) ||
        !encode_bhsd(&to, o, D, Sq, BH, 128) ||
        !encode_bhsd(&tdq, dq, D, Sq, BH, 128) || !encode_bhsd(&tdk, dk, D, Sk, BH, 128) ||
        !encode_bhsd(&tdv, dv, D, Sk, BH, 128))
        return fail_cuda(cudaErrorInvalidValue);
    fa::BwdParams p;
    p.lse = lse;
    p.delta = delta;
    p.Sq = Sq;
    p.Sk = Sk;
    p.n_qt = (int)n_qt;
    p.n_kt = (int)n_kt;
    p.causal = causal;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = timeout_ns;
    const cudaError_t e = fa::launch_bwd(D, tq, tk, tv, tdo, to, tdq, tdk, tdv, p, BH, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    return FA_OK;
}

extern "C" int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                      const void *dout, void *dq, void *dk, void *dv, float *delta, int B, int H, int Sq, int Sk,
                      int D, float scale, int causal, void *stream) {
    return bwd_checked(q, k, v, o, lse, dout, dq, dk, dv, delta, B, H, Sq, Sk, D, scale, causal, stream,
                       kWaitLimitNs);
}

extern "C" int fa_selftest_bwd_timeout(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                       const void *dout, void *dq, void *dk, void *dv, float *delta, int B, int H,
                                       int Sq, int Sk, int D, float scale, int causal, unsigned long long timeout_ns,
                                       void *stream) {
    if (timeout_ns > kWaitLimitNs) return FA_ERR_BAD_SHAPE;
    return bwd_checked(q, k, v, o, lse, dout, dq, dk, dv, delta, B, H, Sq, Sk, D, scale, causal, stream, timeout_ns);
}

// --------------------------------------------------- the paged 8-bit cache
namespace {

struct Span {
    const void *ptr;
    size_t bytes;
};

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// Whether an output overlaps an input or another output.
template <int NO, int NI>
bool any_alias(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int a = 0; a < NO; ++a) {
        if (!outs[a].ptr) continue;
        for (int b = 0; b < NI; ++b)
            if (ins[b].ptr && overlaps(outs[a].ptr, outs[a].bytes, ins[b].ptr, ins[b].bytes)) return true;
        for (int b = a + 1; b < NO; ++b)
            if (outs[b].ptr && overlaps(outs[a].ptr, outs[a].bytes, outs[b].ptr, outs[b].bytes)) return true;
    }
    return false;
}

// log2 of the page size, or -1.
int page_log2_of(int page_size) {
    return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

// Tokens, free pages and chosen pages of a call: kernels count them in int, in steps
// of up to 2^18 past the end.
constexpr int kMostCounted = 1 << 30;

// What the cache's entry points share; FA_OK when the sizes are in range.
int check_cache(int B, int T, int Hkv, int D, int max_pages, int num_pages, int page_size) {
    if (B < 1 || B > fa::kMaxSequences || T < 1 || T > kMostCounted || Hkv < 1 || Hkv > 1024 || max_pages < 1 || num_pages < 1)
        return FA_ERR_BAD_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED_D;
    if (page_log2_of(page_size) < 0) return FA_ERR_BAD_PAGE;
    if ((long long)num_pages * Hkv > 0x7fffffffll || (long long)num_pages * page_size > 0x7fffffffll || (long long)max_pages * page_size > 0x7fffffffll)
        return FA_ERR_BAD_SHAPE;
    return FA_OK;
}

// The stride between tokens of H heads of D elements each.
bool stride_ok(long long stride, int H, int D) {
    return stride >= (long long)H * D && stride % 8 == 0 && stride < (1ll << 40);
}

size_t strided_bytes(int T, long long stride, int H, int D) {
    return ((size_t)(T - 1) * (size_t)stride + (size_t)H * D) * 2;
}

}  // namespace

static int plan_checked(const int *cached_lens, const int *new_lens, const int *free_pages, const int *free_count,
                        int *block_table, int *cu_q, int *seq_lens, int *slot_map, int *positions, int *free_left, int B,
                        int T, int max_pages, int num_free, int num_pages, int page_size, void *stream) {
    const void *ptrs[9] = {cached_lens, new_lens, free_pages, free_count, block_table, cu_q, seq_lens, slot_map, free_left};
    for (const void *ptr : ptrs)
        if (!ptr) return FA_ERR_NULLPTR;
    for (const void *ptr : ptrs)
        if (!aligned4(ptr)) return FA_ERR_MISALIGNED;
    if (!aligned4(positions)) return FA_ERR_MISALIGNED;
    if (num_free < 1 || num_free > kMostCounted) return FA_ERR_BAD_SHAPE;
    const int st = check_cache(B, T, 1, 64, max_pages, num_pages, page_size);
    if (st != FA_OK) return st;
    const Span outs[6] = {{block_table, (size_t)B * max_pages * 4}, {cu_q, ((size_t)B + 1) * 4}, {seq_lens, (size_t)B * 4},
                          {slot_map, (size_t)T * 4}, {free_left, 4}, {positions, (size_t)T * 4}};
    const Span ins[4] = {{cached_lens, (size_t)B * 4}, {new_lens, (size_t)B * 4}, {free_pages, (size_t)num_free * 4}, {free_count, 4}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    fa::PlanParams p;
    p.cached = cached_lens;
    p.fresh = new_lens;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.table = block_table;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.slots = slot_map;
    p.positions = positions;
    p.free_left = free_left;
    p.B = B;
    p.T = T;
    p.max_pages = max_pages;
    p.num_free = num_free;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    const cudaError_t e = fa::launch_kv_plan(p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

extern "C" int fa_kv_plan(const int *cached_lens, const int *new_lens, const int *free_pages, const int *free_count,
                          int *block_table, int *cu_q, int *seq_lens, int *slot_map, int *free_left, int B, int T,
                          int max_pages, int num_free, int num_pages, int page_size, void *stream) {
    return plan_checked(cached_lens, new_lens, free_pages, free_count, block_table, cu_q, seq_lens, slot_map, nullptr, free_left, B, T,
                        max_pages, num_free, num_pages, page_size, stream);
}

extern "C" int fa_kv_plan_positions(const int *cached_lens, const int *new_lens, const int *free_pages,
                                    const int *free_count, int *block_table, int *cu_q, int *seq_lens, int *slot_map,
                                    int *positions, int *free_left, int B, int T, int max_pages, int num_free,
                                    int num_pages, int page_size, void *stream) {
    if (!positions) return FA_ERR_NULLPTR;
    return plan_checked(cached_lens, new_lens, free_pages, free_count, block_table, cu_q, seq_lens, slot_map, positions, free_left, B,
                        T, max_pages, num_free, num_pages, page_size, stream);
}

extern "C" int fa_kv_append(const void *k, const void *v, const int *slot_map, void *k_pages, void *v_pages,
                            float *k_scale, float *v_scale, signed char *k_mean, float *k_mean_scale, int T, int Hkv,
                            int D, long long k_stride, long long v_stride, int num_pages, int page_size,
                            void *stream) {
    if (!k || !v || !slot_map || !k_pages || !v_pages || !k_scale || !v_scale || (!k_mean != !k_mean_scale))
        return FA_ERR_NULLPTR;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_mean) ||
        !aligned4(slot_map) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(k_mean_scale))
        return FA_ERR_MISALIGNED;
    const int st = check_cache(1, T, Hkv, D, 1, num_pages, page_size);
    if (st != FA_OK) return st;
    if (!stride_ok(k_stride, Hkv, D) || !stride_ok(v_stride, Hkv, D)) return FA_ERR_BAD_SHAPE;
    const size_t heads = (size_t)num_pages * Hkv, codes = heads * page_size * D;
    const Span outs[6] = {{k_pages, codes}, {v_pages, codes}, {k_scale, heads * 4}, {v_scale, heads * 4},
                          {k_mean, heads * D}, {k_mean_scale, heads * 4}};
    const Span ins[3] = {{k, strided_bytes(T, k_stride, Hkv, D)}, {v, strided_bytes(T, v_stride, Hkv, D)},
                         {slot_map, (size_t)T * 4}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    fa::AppendParams p{};
    p.x[0] = k;
    p.x[1] = v;
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.slots = slot_map;
    p.pages[0] = static_cast<uint8_t *>(k_pages);
    p.pages[1] = static_cast<uint8_t *>(v_pages);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.mean = reinterpret_cast<int8_t *>(k_mean);
    p.mean_scale = k_mean_scale;
    p.T = T;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    const cudaError_t e = fa::launch_kv_append(D, p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

// ------------------------------------------------------------- rotary positions
namespace {

// A tensor [B, H, S, D] of bf16 with strides (elements) between sequences, tokens and
// heads; its elements within a head are contiguous.
struct Strided {
    const void *ptr;
    long long stride[3];
    int B, S, H, D;

    uintptr_t begin() const { return (uintptr_t)ptr; }
    uintptr_t end() const {
        return begin() + 2 * (size_t)((B - 1) * stride[0] + (S - 1) * stride[1] + (H - 1) * stride[2] + D);
    }
    bool strides_ok() const {
        const int n[3] = {B, S, H};
        double past = D;  // an address counts bytes in 63 bits
        for (int d = 0; d < 3; ++d) {
            if (stride[d] < 0 || stride[d] % 8 != 0 || stride[d] >= (1ll << 40)) return false;
            past += (double)stride[d] * (n[d] - 1);
        }
        return past < 0x1p60;
    }
    // Whether no two of its elements are the same memory: each dimension, in the order
    // of their strides, steps past all of the smaller ones.
    bool distinct() const {
        int n[3] = {B, S, H}, order[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (stride[order[j]] < stride[order[i]]) {
                    const int x = order[i];
                    order[i] = order[j];
                    order[j] = x;
                }
        long long past = D;
        for (const int d : order) {
            if (n[d] == 1) continue;
            if (stride[d] < past) return false;
            past += stride[d] * (n[d] - 1);
        }
        return true;
    }
    bool same(const Strided &o) const {
        return ptr == o.ptr && B == o.B && S == o.S && H == o.H && D == o.D && (B == 1 || stride[0] == o.stride[0]) &&
               (S == 1 || stride[1] == o.stride[1]) && (H == 1 || stride[2] == o.stride[2]);
    }
};

// Whether two tensors share memory.  Those whose spans do may still be columns of one
// fused tensor: with the same strides between tokens and between sequences, the latter
// a multiple of the former, each lies within its own part of every token's row.
bool shares(const Strided &a, const Strided &b) {
    if (a.end() <= b.begin() || b.end() <= a.begin()) return false;
    const int step = a.S > 1 ? 1 : 0;  // sequences of one token: their stride is the row's
    const long long row = a.stride[step];
    if (a.B != b.B || a.S != b.S || row <= 0 || b.stride[step] != row) return true;
    if (a.S > 1 && a.B > 1 && (a.stride[0] != b.stride[0] || a.stride[0] % row != 0)) return true;
    const long long na = (a.H - 1) * a.stride[2] + a.D, nb = (b.H - 1) * b.stride[2] + b.D;
    const long long bytes = (long long)(b.begin() - a.begin());  // (wraps around where b is lower)
    if (bytes % 2 != 0) return true;
    const long long at = ((bytes / 2) % row + row) % row;  // b's place in a's rows
    return at < na || at + nb > row;
}

// A rotated tensor and its output: the very same tensor, or no memory in common.
bool turned_in_place_or_apart(const Strided &x, const Strided &y) { return x.same(y) || !shares(x, y); }

int check_rotation(const unsigned long long *phases, const int *positions, int rot_dim, int D, int interleaved, float amplitude) {
    if (!phases) return FA_ERR_NULLPTR;
    if (((uintptr_t)phases & 7u) != 0 || !aligned4(positions)) return FA_ERR_MISALIGNED;
    if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > D || (interleaved != 0 && interleaved != 1)) return FA_ERR_BAD_SHAPE;
    if (!isfinite(amplitude) || !(amplitude > 0.f)) return FA_ERR_BAD_SCALE;
    return FA_OK;
}

int rope_checked(const void *q, const void *k, void *q_out, void *k_out, const int *positions, const unsigned long long *phases,
                 int B, int S, int Hq, int Hk, int D, int rot_dim, const long long *strides, long long positions_stride,
                 int interleaved, float amplitude, int inverse, void *stream) {
    if (!q || !q_out || !phases || !strides || (Hk > 0 && (!k || !k_out))) return FA_ERR_NULLPTR;
    if (!aligned16(q) || !aligned16(q_out) || (Hk > 0 && (!aligned16(k) || !aligned16(k_out)))) return FA_ERR_MISALIGNED;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED_D;
    if (B < 1 || S < 1 || (long long)B * S > kMostCounted || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535) return FA_ERR_BAD_SHAPE;
    const int st = check_rotation(phases, positions, rot_dim, D, interleaved, amplitude);
    if (st != FA_OK) return st;
    if (positions && (positions_stride < 0 || positions_stride >= (1ll << 31) || (positions_stride != 0 && positions_stride < S && B > 1)))
        return FA_ERR_BAD_SHAPE;
    Strided t[4];  // q, k, q_out, k_out
    const void *ptr[4] = {q, k, q_out, k_out};
    for (int i = 0; i < 4; ++i) {
        t[i] = Strided{ptr[i], {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]}, B, S, i % 2 ? Hk : Hq, D};
        if (i % 2 && Hk == 0) continue;
        if (!t[i].strides_ok() || (i >= 2 && !t[i].distinct())) return FA_ERR_BAD_SHAPE;
    }
    if (!turned_in_place_or_apart(t[0], t[2])) return FA_ERR_ALIAS;
    if (Hk > 0 && (!turned_in_place_or_apart(t[1], t[3]) || shares(t[0], t[3]) || shares(t[1], t[2]) || shares(t[2], t[3])))
        return FA_ERR_ALIAS;
    // the other inputs, which may lie in no gap of an output either
    const size_t np = positions ? ((size_t)(B - 1) * (size_t)positions_stride + (size_t)S) * 4 : 0;
    for (int i = 2; i < (Hk > 0 ? 4 : 3); ++i) {
        const size_t n = t[i].end() - t[i].begin();
        if ((positions && overlaps(t[i].ptr, n, positions, np)) || overlaps(t[i].ptr, n, phases, (size_t)rot_dim * 4)) return FA_ERR_ALIAS;
    }
    fa::RopeParams p{};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = ptr[i];
        p.y[i] = const_cast<void *>(ptr[i + 2]);
        for (int d = 0; d < 3; ++d) {
            p.x_stride[i][d] = strides[3 * i + d];
            p.y_stride[i][d] = strides[3 * (i + 2) + d];
        }
    }
    p.H[0] = Hq;
    p.H[1] = Hk;
    p.positions = positions;
    p.positions_stride = positions_stride;
    p.phases = phases;
    p.B = B;
    p.S = S;
    p.D = D;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.inverse = inverse;
    p.amplitude = amplitude;
    const cudaError_t e = fa::launch_rope(p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

}  // namespace

extern "C" int fa_rope(const void *q, const void *k, void *q_out, void *k_out, const int *positions,
                       const unsigned long long *phases, int B, int S, int Hq, int Hk, int D, int rot_dim,
                       const long long *strides, long long positions_stride, int interleaved, float amplitude,
                       void *stream) {
    return rope_checked(q, k, q_out, k_out, positions, phases, B, S, Hq, Hk, D, rot_dim, strides, positions_stride, interleaved,
                        amplitude, 0, stream);
}

extern "C" int fa_rope_bwd(const void *dq_out, const void *dk_out, void *dq, void *dk, const int *positions,
                           const unsigned long long *phases, int B, int S, int Hq, int Hk, int D, int rot_dim,
                           const long long *strides, long long positions_stride, int interleaved, float amplitude,
                           void *stream) {
    return rope_checked(dq_out, dk_out, dq, dk, positions, phases, B, S, Hq, Hk, D, rot_dim, strides, positions_stride, interleaved,
                        amplitude, 1, stream);
}

extern "C" int fa_rope_phases(unsigned long long *phases, float *amplitude, int rot_dim, double base, int scaling,
                              double factor, double span, double fast, double slow, const double *frequencies) {
    if (!phases || !amplitude) return FA_ERR_NULLPTR;
    if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > 128) return FA_ERR_BAD_SHAPE;
    if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_YARN) return FA_ERR_BAD_SHAPE;
    const double two_pi = 6.283185307179586476925;
    if (!frequencies && (!isfinite(base) || !(base > 1.0))) return FA_ERR_BAD_SCALE;
    if (scaling != FA_ROPE_PLAIN && (!isfinite(factor) || !(factor >= 1.0))) return FA_ERR_BAD_SCALE;
    if (scaling == FA_ROPE_NTK && frequencies) return FA_ERR_BAD_SHAPE;
    if (scaling == FA_ROPE_YARN && (!isfinite(span) || !(span >= 1.0) || !isfinite(fast) || !(slow > 0.0) || !(fast >= slow)))
        return FA_ERR_BAD_SCALE;
    if (scaling == FA_ROPE_YARN && frequencies) return FA_ERR_BAD_SHAPE;
    *amplitude = 1.f;
    double lo = 0.0, hi = 0.0;
    if (scaling == FA_ROPE_NTK) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    if (scaling == FA_ROPE_YARN) {
        // the pairs that make `fast` and `slow` turns over the span
        lo = floor(rot_dim * log(span / (fast * two_pi)) / (2.0 * log(base)));
        hi = ceil(rot_dim * log(span / (slow * two_pi)) / (2.0 * log(base)));
        lo = lo > 0.0 ? lo : 0.0;
        hi = hi < rot_dim - 1 ? hi : rot_dim - 1;
        *amplitude = (float)(0.1 * log(factor) + 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = frequencies ? frequencies[i] : pow(base, -2.0 * i / rot_dim);
        if (!isfinite(f)) return FA_ERR_BAD_SCALE;
        if (scaling == FA_ROPE_LINEAR) f /= factor;
        if (scaling == FA_ROPE_YARN) {
            const double width = hi - lo > 0.001 ? hi - lo : 0.001;
            const double ramp = fmin(1.0, fmax(0.0, (i - lo) / width));
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        double turns = f / two_pi;
        turns -= floor(turns);  // in [0, 1], and 1 is no turn at all
        phases[i] = turns < 1.0 ? (unsigned long long)(turns * 18446744073709551616.0) : 0ull;
    }
    return FA_OK;
}

extern "C" int fa_kv_append_rope(const void *k, const void *v, const int *positions, const unsigned long long *phases,
                                 const int *slot_map, void *k_pages, void *v_pages, float *k_scale, float *v_scale,
                                 signed char *k_mean, float *k_mean_scale, const void *q, void *q_out, int T, int Hkv,
                                 int Hq, int D, int rot_dim, int interleaved, float amplitude, long long k_stride,
                                 long long v_stride, long long q_stride, long long q_out_stride, int num_pages,
                                 int page_size, void *stream) {
    if (!k || !v || !positions || !phases || !slot_map || !k_pages || !v_pages || !k_scale || !v_scale || (!k_mean != !k_mean_scale) ||
        (!q != !q_out))
        return FA_ERR_NULLPTR;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_mean) || !aligned16(q) ||
        !aligned16(q_out) || !aligned4(slot_map) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(k_mean_scale))
        return FA_ERR_MISALIGNED;
    int st = check_cache(1, T, Hkv, D, 1, num_pages, page_size);
    if (st != FA_OK) return st;
    st = check_rotation(phases, positions, rot_dim, D, interleaved, amplitude);
    if (st != FA_OK) return st;
    if (!stride_ok(k_stride, Hkv, D) || !stride_ok(v_stride, Hkv, D)) return FA_ERR_BAD_SHAPE;
    if (q && (Hq < 1 || Hq > 65535 || Hq % Hkv != 0 || !stride_ok(q_stride, Hq, D) || !stride_ok(q_out_stride, Hq, D))) return FA_ERR_BAD_SHAPE;
    const size_t heads = (size_t)num_pages * Hkv, codes = heads * page_size * D;
    const size_t k_bytes = strided_bytes(T, k_stride, Hkv, D), v_bytes = strided_bytes(T, v_stride, Hkv, D);
    const size_t q_bytes = q ? strided_bytes(T, q_stride, Hq, D) : 0, q_out_bytes = q ? strided_bytes(T, q_out_stride, Hq, D) : 0;
    const Span outs[6] = {{k_pages, codes}, {v_pages, codes}, {k_scale, heads * 4}, {v_scale, heads * 4},
                          {k_mean, heads * D}, {k_mean_scale, heads * 4}};
    const Span ins[7] = {{k, k_bytes}, {v, v_bytes}, {slot_map, (size_t)T * 4}, {positions, (size_t)T * 4}, {phases, (size_t)rot_dim * 4},
                         {q, q_bytes}, {q_out, q_out_bytes}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    if (q) {  // rotated queries may lie in the same fused tensor
        const Strided a{k, {0, k_stride, D}, 1, T, Hkv, D}, b{v, {0, v_stride, D}, 1, T, Hkv, D};
        const Strided x{q, {0, q_stride, D}, 1, T, Hq, D}, y{q_out, {0, q_out_stride, D}, 1, T, Hq, D};
        if (!x.strides_ok() || !y.strides_ok() || !a.strides_ok() || !b.strides_ok()) return FA_ERR_BAD_SHAPE;
        if (!turned_in_place_or_apart(x, y) || shares(a, y) || shares(b, y)) return FA_ERR_ALIAS;
        for (int i = 2; i < 5; ++i)
            if (overlaps(q_out, q_out_bytes, ins[i].ptr, ins[i].bytes)) return FA_ERR_ALIAS;
    }
    fa::AppendParams p{};
    p.x[0] = k;
    p.x[1] = v;
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.slots = slot_map;
    p.pages[0] = static_cast<uint8_t *>(k_pages);
    p.pages[1] = static_cast<uint8_t *>(v_pages);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.mean = reinterpret_cast<int8_t *>(k_mean);
    p.mean_scale = k_mean_scale;
    p.T = T;
    p.Hkv = Hkv;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.amplitude = amplitude;
    p.positions = positions;
    p.phases = phases;
    p.q = q;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.G = q ? Hq / Hkv : 0;
    const cudaError_t e = fa::launch_kv_append(D, p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

extern "C" int fa_page_select(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                              const signed char *k_mean, const float *k_mean_scale, int *sel, int *sel_count, int B,
                              int T, int Hq, int Hkv, int D, long long q_stride, int max_pages, int num_pages,
                              int page_size, int top_k, int keep_first, int keep_last, void *stream) {
    if (!q || !cu_q || !seq_lens || !block_table || !k_mean || !k_mean_scale || !sel || !sel_count)
        return FA_ERR_NULLPTR;
    const void *ints[6] = {cu_q, seq_lens, block_table, k_mean_scale, sel, sel_count};
    for (const void *ptr : ints)
        if (!aligned4(ptr)) return FA_ERR_MISALIGNED;
    if (!aligned16(q) || !aligned16(k_mean)) return FA_ERR_MISALIGNED;
    const int st = check_cache(B, T, Hkv, D, max_pages, num_pages, page_size);
    if (st != FA_OK) return st;
    if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0 || !stride_ok(q_stride, Hq, D) || max_pages > fa::kSelectMaxPages ||
        (long long)T * Hq > 0x7fffffff || top_k < 1 || top_k > kMostCounted || keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > top_k)
        return FA_ERR_BAD_SHAPE;
    const Span outs[2] = {{sel, (size_t)B * Hkv * top_k * 4}, {sel_count, (size_t)B * Hkv * 4}};
    const Span ins[6] = {{q, strided_bytes(T, q_stride, Hq, D)}, {cu_q, ((size_t)B + 1) * 4}, {seq_lens, (size_t)B * 4},
                         {block_table, (size_t)B * max_pages * 4}, {k_mean, (size_t)num_pages * Hkv * D},
                         {k_mean_scale, (size_t)num_pages * Hkv * 4}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    fa::SelectParams p;
    p.q = q;
    p.q_stride = q_stride;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.table = block_table;
    p.mean = reinterpret_cast<const int8_t *>(k_mean);
    p.mean_scale = k_mean_scale;
    p.sel = sel;
    p.sel_count = sel_count;
    p.B = B;
    p.T = T;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    p.top_k = top_k;
    p.keep_first = keep_first;
    p.keep_last = keep_last;
    const cudaError_t e = fa::launch_page_select(D, p, (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

static bool paged_shape_ok(int B, int T, int Hq, int Hkv, int D) {
    return B >= 1 && B <= fa::kMaxSequences && T >= 1 && T <= kMostCounted && Hkv >= 1 && Hkv <= 1024 && Hq >= 1 && Hq <= 65535 &&
           Hq % Hkv == 0 && (long long)T * Hq <= 0x7fffffff && (D == 64 || D == 128);
}

extern "C" size_t fa_fwd_paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    if (!paged_shape_ok(B, T, Hq, Hkv, D)) return 0;
    return fa::paged_workspace_bytes(B, T, Hq, Hkv, D, sm_count());
}

extern "C" int fa_fwd_paged(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                            const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                            const int *sel, const int *sel_count, void *o, float *lse, int B, int T, int Hq, int Hkv,
                            int D, float scale, long long q_stride, int max_pages, int num_pages, int page_size,
                            int sel_width, void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !cu_q || !seq_lens || !block_table || !k_pages || !v_pages || !k_scale || !v_scale || !o || !lse ||
        (!sel != !sel_count))
        return FA_ERR_NULLPTR;
    const void *ints[8] = {cu_q, seq_lens, block_table, k_scale, v_scale, sel, sel_count, lse};
    for (const void *ptr : ints)
        if (!aligned4(ptr)) return FA_ERR_MISALIGNED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o)) return FA_ERR_MISALIGNED;
    const int st = check_cache(B, T, Hkv, D, max_pages, num_pages, page_size);
    if (st != FA_OK) return st;
    if (!paged_shape_ok(B, T, Hq, Hkv, D) || !stride_ok(q_stride, Hq, D) || (sel && sel_width < 1)) return FA_ERR_BAD_SHAPE;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!isfinite(scale) || !(scale > 0.f) || !isfinite(scale_log2)) return FA_ERR_BAD_SCALE;
    const size_t need = fa::paged_workspace_bytes(B, T, Hq, Hkv, D, sm_count());
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t heads = (size_t)num_pages * Hkv, codes = heads * page_size * D;
    if (heads * page_size > 0xffffffffull) return FA_ERR_BAD_SHAPE;  // rows of a cache: more than memory holds
    const Span outs[3] = {{o, (size_t)T * Hq * D * 2}, {lse, (size_t)T * Hq * 4}, {workspace, need}};
    const Span ins[10] = {{q, strided_bytes(T, q_stride, Hq, D)}, {cu_q, ((size_t)B + 1) * 4}, {seq_lens, (size_t)B * 4},
                          {block_table, (size_t)B * max_pages * 4}, {k_pages, codes}, {v_pages, codes},
                          {k_scale, heads * 4}, {v_scale, heads * 4}, {sel, (size_t)B * Hkv * (sel ? sel_width : 0) * 4},
                          {sel_count, (size_t)B * Hkv * 4}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    fa::PagedParams p;
    p.q = q;
    p.q_stride = q_stride;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.table = block_table;
    p.k_pages = static_cast<const uint8_t *>(k_pages);
    p.v_pages = static_cast<const uint8_t *>(v_pages);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.sel = sel;
    p.sel_count = sel_count;
    p.o = o;
    p.lse = lse;
    p.ws = static_cast<float *>(workspace);
    p.B = B;
    p.T = T;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    p.sel_width = sel ? sel_width : 0;
    p.scale_log2 = scale_log2;
    if (!fa::paged_fits(D, p)) return FA_ERR_BAD_SHAPE;
    const cudaError_t e = fa::launch_fwd_paged(D, p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

extern "C" size_t fa_fwd_paged_chunk_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    if (!paged_shape_ok(B, T, Hq, Hkv, D)) return 0;
    return fa::paged_chunk_workspace_bytes(D, sm_count());
}

static int chunk_checked(const void *q, const int *cu_q, const int *seq_lens, const int *block_table, const void *k_pages,
                         const void *v_pages, const float *k_scale, const float *v_scale, void *o, float *lse, int B, int T, int Hq,
                         int Hkv, int D, float scale, long long q_stride, int max_pages, int num_pages, int page_size,
                         void *workspace, size_t workspace_bytes, unsigned long long timeout_ns, void *stream) {
    if (!q || !cu_q || !seq_lens || !block_table || !k_pages || !v_pages || !k_scale || !v_scale || !o || !lse) return FA_ERR_NULLPTR;
    const void *ints[6] = {cu_q, seq_lens, block_table, k_scale, v_scale, lse};
    for (const void *ptr : ints)
        if (!aligned4(ptr)) return FA_ERR_MISALIGNED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o)) return FA_ERR_MISALIGNED;
    const int st = check_cache(B, T, Hkv, D, max_pages, num_pages, page_size);
    if (st != FA_OK) return st;
    if (!paged_shape_ok(B, T, Hq, Hkv, D) || !stride_ok(q_stride, Hq, D)) return FA_ERR_BAD_SHAPE;
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!isfinite(scale) || !(scale > 0.f) || !isfinite(scale_log2)) return FA_ERR_BAD_SCALE;
    const size_t need = fa::paged_chunk_workspace_bytes(D, sm_count());
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return FA_ERR_WORKSPACE;
    const size_t heads = (size_t)num_pages * Hkv, codes = heads * page_size * D;
    if (heads * page_size > 0xffffffffull) return FA_ERR_BAD_SHAPE;  // rows of a cache: more than memory holds
    if ((long long)max_pages * page_size > 0x7fffffffll - 1024) return FA_ERR_BAD_SHAPE;  // a length, a tile and an item's fixed cost are one int
    const Span outs[3] = {{o, (size_t)T * Hq * D * 2}, {lse, (size_t)T * Hq * 4}, {workspace, need}};
    const Span ins[8] = {{q, strided_bytes(T, q_stride, Hq, D)}, {cu_q, ((size_t)B + 1) * 4}, {seq_lens, (size_t)B * 4},
                         {block_table, (size_t)B * max_pages * 4}, {k_pages, codes}, {v_pages, codes},
                         {k_scale, heads * 4}, {v_scale, heads * 4}};
    if (any_alias(outs, ins)) return FA_ERR_ALIAS;
    fa::ChunkParams p{};
    p.q = q;
    p.q_stride = q_stride;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.table = block_table;
    p.k_pages = static_cast<const uint8_t *>(k_pages);
    p.v_pages = static_cast<const uint8_t *>(v_pages);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.o = o;
    p.lse = lse;
    p.ws = static_cast<float *>(workspace);
    p.B = B;
    p.T = T;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_log2 = page_log2_of(page_size);
    p.scale_log2 = scale_log2;
    p.limit_us = (uint32_t)(timeout_ns / 1000);
    const cudaError_t e = fa::launch_fwd_paged_chunk(D, p, sm_count(), (cudaStream_t)stream);
    return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

extern "C" int fa_fwd_paged_chunk(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                                  const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                                  void *o, float *lse, int B, int T, int Hq, int Hkv, int D, float scale,
                                  long long q_stride, int max_pages, int num_pages, int page_size, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    return chunk_checked(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o, lse, B, T, Hq, Hkv, D, scale, q_stride,
                         max_pages, num_pages, page_size, workspace, workspace_bytes, kWaitLimitNs, stream);
}

extern "C" int fa_selftest_paged_chunk_timeout(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                                               const void *k_pages, const void *v_pages, const float *k_scale,
                                               const float *v_scale, void *o, float *lse, int B, int T, int Hq, int Hkv,
                                               int D, float scale, long long q_stride, int max_pages, int num_pages,
                                               int page_size, void *workspace, size_t workspace_bytes,
                                               unsigned long long timeout_ns, void *stream) {
    if (timeout_ns > kWaitLimitNs) return FA_ERR_BAD_SHAPE;
    return chunk_checked(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o, lse, B, T, Hq, Hkv, D, scale, q_stride,
                         max_pages, num_pages, page_size, workspace, workspace_bytes, timeout_ns, stream);
}

extern "C" int fa_device_status(void *stream) {
    int v = 0, w = 0, x = 0;
    cudaError_t e = fa::status_read_and_clear(&v, (cudaStream_t)stream);
    if (e == cudaSuccess) e = fa::splitkv_status_read_and_clear(&w);
    if (e == cudaSuccess) e = fa::bwd_status_read_and_clear(&x);
    int cache[5] = {0, 0, 0, 0, 0};  // the paged cache's kernels
    if (e == cudaSuccess) e = fa::kv_cache_status_read_and_clear(&cache[0]);
    if (e == cudaSuccess) e = fa::page_select_status_read_and_clear(&cache[1]);
    if (e == cudaSuccess) e = fa::paged_status_read_and_clear(&cache[2]);
    if (e == cudaSuccess) e = fa::paged_chunk_status_read_and_clear(&cache[3]);
    if (e == cudaSuccess) e = fa::kv_append_rope_status_read_and_clear(&cache[4]);
    if (e != cudaSuccess) return fail_cuda(e);
    for (int c : cache)
        if (x == FA_OK) x = c;
    return v != FA_OK ? v : (w != FA_OK ? w : x);
}

extern "C" int fa_selftest_bounded_wait(int timeout_us, void *stream) {
    if (timeout_us < 1 || timeout_us > 1000000) return FA_ERR_BAD_SHAPE;
    const cudaError_t e = fa::launch_wait_selftest((unsigned long long)timeout_us * 1000ull, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    return FA_OK;
}

extern "C" int fa_selftest_fwd_timeout(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                                       int H, int Sq, int Sk, int D, float scale, int causal,
                                       unsigned long long timeout_ns, void *stream) {
    const int st = check_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale);
    if (st != FA_OK) return st;
    if (causal != 0 && causal != 1) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (causal && Sq != Sk) return FA_ERR_UNSUPPORTED_CAUSAL;
    if (timeout_ns > kWaitLimitNs) return FA_ERR_BAD_SHAPE;
    return launch_checked(q, k, v, o, lse, B, H, Sq, Sk, D, scale, -1, causal ? 0 : -1, stream, timeout_ns);
}
