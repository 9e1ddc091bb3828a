// fa_paged.h -- declarations of the paged 8-bit cache's kernels, shared by
// the C-ABI layer and their translation units.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

constexpr int kMaxSequences = 8192;  // of a call; fa_kv_plan's sums of that many stay in shared memory

struct PlanParams {
    const int *cached, *fresh;   // [B] tokens in the cache, tokens of this step
    const int *free_pages, *free_count;
    int *table;                  // [B, max_pages]
    int *cu_q, *seq_lens, *slots, *free_left;
    int *positions;              // [T], or null
    int B, T, max_pages, num_free, num_pages, page_log2;
};
cudaError_t launch_kv_plan(const PlanParams &p, int num_sms, cudaStream_t stream);

struct AppendParams {
    const void *x[2];            // k, v: bf16 [T, Hkv, D]
    long long stride[2];         // elements between tokens
    const int *slots;
    uint8_t *pages[2];           // k_pages, v_pages
    float *scale[2];
    int8_t *mean;                // null: no means are kept
    float *mean_scale;
    int T, Hkv, num_pages, page_log2;
    // fa_kv_append_rope (rot = 0: keys are not rotated)
    int rot, interleaved;        // elements of a head that are rotated; which make a pair
    float amplitude;
    const int *positions;        // [T]
    const unsigned long long *phases;  // [rot / 2]
    const void *q;               // bf16 [T, Hkv * G, D], or null: no queries
    void *q_out;
    long long q_stride, q_out_stride;
    int G;
};
cudaError_t launch_kv_append(int D, const AppendParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_append_rope(int D, const AppendParams &p, int num_sms, cudaStream_t stream);

struct SelectParams {
    const void *q;               // bf16 [T, Hq, D]
    long long q_stride;
    const int *cu_q, *seq_lens, *table;
    const int8_t *mean;
    const float *mean_scale;
    int *sel, *sel_count;
    int B, T, G, Hkv, max_pages, num_pages, page_log2;
    int top_k, keep_first, keep_last;
};
struct RopeParams {
    const void *x[2];            // queries, keys: bf16 [B, H, S, D] with any strides
    void *y[2];
    long long x_stride[2][3], y_stride[2][3];  // batch, token, head
    int H[2];                    // heads; keys may have none
    const int *positions;        // null: 0 .. S - 1
    long long positions_stride;  // between sequences
    const unsigned long long *phases;
    int B, S, D, rot, interleaved, inverse;
    float amplitude;
};
cudaError_t launch_rope(const RopeParams &p, int num_sms, cudaStream_t stream);

constexpr int kSelectMaxPages = 49152;  // scores of one (sequence, head) stay in shared memory
cudaError_t launch_page_select(int D, const SelectParams &p, cudaStream_t stream);

struct PagedParams {
    const void *q;               // bf16 [T, Hq, D]
    long long q_stride;
    const int *cu_q, *seq_lens, *table;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int *sel, *sel_count;  // null: every page
    void *o;                     // bf16 [T, Hq, D]
    float *lse;                  // fp32 [T, Hq]
    float *ws;
    int B, T, G, Hkv, max_pages, num_pages, page_log2, sel_width;
    int max_len;                 // tokens that a table row holds (set by the launch)
    float scale_log2;            // scale * log2(e)
};
// Whether the work of these sizes, at most, can be laid out in 32-bit places.
bool paged_fits(int D, const PagedParams &p);
size_t paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int num_sms);
cudaError_t launch_fwd_paged(int D, const PagedParams &p, int num_sms, cudaStream_t stream);

struct ChunkParams {
    const void *q;               // bf16 [T, Hq, D]
    long long q_stride;
    const int *cu_q, *seq_lens, *table;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    void *o;                     // bf16 [T, Hq, D]
    float *lse;                  // fp32 [T, Hq]
    float *ws;
    int B, T, G, Hkv, max_pages, num_pages, page_log2;
    int max_len;                 // tokens that a table row holds (set by the launch)
    int item_keys;               // keys that an item sees more than the one before it, about (set by the launch)
    float scale_log2;            // scale * log2(e)
    uint32_t limit_us;           // bound of every on-chip wait
};
size_t paged_chunk_workspace_bytes(int D, int num_sms);
cudaError_t launch_fwd_paged_chunk(int D, ChunkParams p, int num_sms, cudaStream_t stream);

// Each translation unit's device status word: read it and reset it.
cudaError_t kv_cache_status_read_and_clear(int *out);
cudaError_t page_select_status_read_and_clear(int *out);
cudaError_t paged_status_read_and_clear(int *out);
cudaError_t paged_chunk_status_read_and_clear(int *out);
cudaError_t kv_append_rope_status_read_and_clear(int *out);

// A launch whose blocks may be made ready while the kernel before it in the stream
// ends: every kernel of the paged cache begins by waiting for the one before it to have
// ended and its writes to be seen (grid_wait).  Back to back calls of fa_kv_plan: 5.1 us with
// plain launches, 3.1 us with these.  (None lets the next one in before its own end: blocks
// that wait take the place of blocks that work, 4.3 -> 7.1 us where there are many.)
// `cluster`: blocks of a cluster along x.
template <class... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

}  // namespace fa
