// qasa_launch.h -- kernel parameter blocks and launchers shared by the
// kernel translation units and the C entry points (host + device visible).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qasa.h"

namespace qasa {

struct AppendParams {
    void *k_pool;
    void *v_pool;
    void *bounds;
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *append_lens;
    const void *k_new;
    const void *v_new;
    int32_t *status;
    int num_phys, Hkv, P, max_pages, T;
    float *scales;       // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
};

struct RotatedParams {
    void *k_pool;
    void *v_pool;
    void *bounds;
    float *scales;       // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *append_lens;
    const float *table;  // [max_positions][2][rot / 2]
    const void *q;       // or NULL
    void *q_out;
    const void *k_new;
    const void *v_new;
    long long q_batch, q_token, k_batch, k_token, v_batch, v_token;   // strides in elements
    int32_t *status;
    int num_phys, Hkv, Hq, P, max_pages, T, max_positions, rot, interleaved;
    int kv_blocks;       // blocks in x of the KV role, the rest rotate q
    int q_span;          // batches of query heads that a warp rotates
    int sms;             // SMs of the device
    // positions given by the caller (NULL: those of the slots)
    const int32_t *positions;
    long long pos_axis, pos_batch;   // strides in elements
    int num_axes;
    uint32_t pair_axes[4];           // axis of each channel pair, two bits each
};

struct WindowParams {
    const void *q;
    void *out;
    const void *k_pool;
    const void *v_pool;
    const float *scales; // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
    const int32_t *q_lens;
    const int32_t *block_table;
    const int32_t *seq_lens;
    int32_t *status;
    int B, T, Hq, Hkv, G, P, max_pages, num_phys;
    int window, sinks;
    float scale_log2;
    int cluster;         // CTAs that share a unit (row tile of a sequence and KV head)
    int row_tiles;       // row tiles (pairs of them in the prompt kernel) of the longest sequence
    int sms;             // prompt kernel: SMs of the device
    long long most_tiles;   // prompt kernel: the most 16-token tiles that a CTA's rows see
    int b0;              // prompt kernel: first sequence of the launch, which has B of them
    int ws_pages;        // E4M3, prompt kernel: pages per sequence in the workspace
    unsigned long long wait_limit_ns;    // prompt kernel: waits on other warps
    unsigned long long drain_limit_ns;   // waits for the CTA's own copies and products (never shortened)
    // trees of drafted tokens: [batch][T][mask_words], bit j of row t: query t sees the drafted token j
    const int32_t *mask;
    long long mask_batch;                // words from one sequence's mask to the next (0: all share one)
    int mask_words;
};

struct TreeParams {
    WindowParams w;
    int whole_units;     // a CTA takes whole units: nothing to join
    int4 *cuts;          // [ctas] the unit whose first piece the CTA has (sequence, KV head, token; x < 0: none), last CTA
    float2 *part_ml;     // [2 ctas][rows] maximum (log2 units) and sum of weights
    float4 *part_o;      // [2 ctas][d / 4][rows]
};
// Byte offsets in a workspace (cuts lie first), and its size.
struct TreeWorkspace { size_t ml, o, bytes; };

struct KeepParams {
    void *k_pool;
    void *v_pool;
    void *bounds;
    float *scales;       // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *starts;
    const int32_t *keep; // [batch][M]
    const int32_t *keep_lens;
    int32_t *lens_out;
    int32_t *status;
    int num_phys, Hkv, P, max_pages, M;
    int cluster;         // CTAs that share a sequence's K or V of a KV head
};

struct PageCopyParams {
    void *k_pool;
    void *v_pool;
    void *bounds;
    float *scales;       // FP8 KV, else NULL
    int32_t *status;
    int num_phys, Hkv, P, row_chunks;    // 16-byte chunks of a row
    int pieces;          // blocks per page
    // copies
    const int32_t *src_pages, *dst_pages;
    // forks
    const int32_t *block_table, *seq_lens, *parents, *new_pages;
    int32_t *table_out, *lens_out;
    int max_pages, batch;
};

struct TreeMaskParams {
    const int32_t *parents;
    const int32_t *lens;
    int32_t *mask;
    int32_t *depths;
    int32_t *status;
    int T, words;
};

struct SelectParams {
    const void *bounds;
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *budget;
    const void *q;
    int32_t *selected;
    float *scores_out;
    int32_t *counters;       // [units] the attention kernel's page tickets, cleared here
    int32_t *status;
    int B, num_phys, Hkv, P, G, Hq, max_pages, max_budget;
    const float *scales;   // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
    unsigned long long *trace;   // diagnostics: [QASA_TRACE_MAX_CTAS][QASA_TRACE_SELECT_EVENTS] or NULL
};

struct AttnParams {
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *budget;
    int32_t *selected;       // read; written too by the single-launch kernel
    const void *q;
    void *out;
    float *part_o;     // [(units + C) * G * D]
    float *part_ml;    // [(units + C) * G * 2]  (running max in log2 units, sum of weights)
    int32_t *counters; // [units]
    int32_t *status;
    int B, Hkv, G, Hq, max_pages, max_budget, num_phys;
    float scale_log2;
    int dense;
    int unit_weight;   // page-equivalents a unit adds to a CTA range's work (ranges balance pages + this per unit)
    int one_box;       // 2: one box per page holding its K and V tiles (kmap only);
                       // 1: one 3-D TMA box per K/V tile; 0: one 2-D box per 128 bytes of head dim
    int stages;        // ring depth, a multiple of `consumers`
    int consumers;     // consumer warps that take pages (<= the compiled count)
    unsigned long long wait_limit_ns;    // waits on other warps, CTAs or flags
    unsigned long long drain_limit_ns;   // waits for this CTA's own copies in flight (never shortened)
    // single-launch decode only: the selection inputs and outputs
    const void *bounds;
    float *scores_out;
    int32_t *ready;    // [units] 1 once a unit's kept ids are published (zero at launch)
    const float *scales;   // FP8 KV: [num_phys][Hkv][4] (amax K, amax V, -, -)
    unsigned long long *trace;   // diagnostics: [QASA_TRACE_MAX_CTAS][QASA_TRACE_ATTN_EVENTS] or NULL
};

struct MassParams {
    const void *k_pool;
    const int32_t *block_table;
    const int32_t *seq_lens;
    const void *q;
    float *mass;       // [B][Hkv][max_pages]
    int32_t *status;
    int num_phys, Hkv, P, G, Hq, max_pages;
    float scale_log2;
};

struct HitParams {
    const float *mass;        // [B][Hkv][max_pages]
    const int32_t *seq_lens;
    const int32_t *budget;
    const int32_t *selected;  // [B][Hkv][max_budget]
    int32_t *hits;            // [B][Hkv]
    float *covered;           // [B][Hkv]
    float *best;              // [B][Hkv]
    int32_t *status;
    int Hkv, P, max_pages, max_budget;
};

struct RebuildParams {
    const void *k_pool;
    void *bounds;
    const int32_t *block_table;
    const int32_t *seq_lens;
    int32_t *status;
    int num_phys, Hkv, P, max_pages;
};

cudaError_t launch_append(qasa_dtype dt, int D, const AppendParams &p, int batch, cudaStream_t stream);
cudaError_t launch_append_rotated(qasa_dtype dt, int D, const RotatedParams &p, int batch, cudaStream_t stream);
// Windowed attention for few query rows per KV head; window_row_tiles: the units
// per (sequence, KV head) that it makes of `rows` rows.
int window_row_tiles(qasa_dtype dt, int rows);
cudaError_t launch_window_rows(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream);
// Trees of drafted tokens (p.mask).
cudaError_t launch_tree_masks(const TreeMaskParams &p, int batch, cudaStream_t stream);
// 16-bit and E4M3 caches, many rows: q, k, v as for launch_window_prompt (k, v not read for E4M3 pages).
// wide: units of two row tiles.  ctas: at most one per SM.
TreeWorkspace tree_workspace(int D, bool wide, int ctas);
cudaError_t launch_tree(qasa_dtype dt, int D, bool wide, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                        const TreeParams &p, int ctas, cudaStream_t stream);
cudaError_t launch_tree_rows(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream);
cudaError_t launch_keep(qasa_dtype dt, int D, const KeepParams &p, int batch, cudaStream_t stream);
int page_pieces(const PageCopyParams &p);
cudaError_t launch_copy_pages(const PageCopyParams &p, int pairs, cudaStream_t stream);
cudaError_t launch_fork(const PageCopyParams &p, int children, cudaStream_t stream);
// The same for many: 16-bit and E4M3 caches.  q: [batch * tokens][heads][d] in boxes of
// 64 channels, G heads and 128 / G tokens; k, v: pool rows (E4M3: the rows that
// launch_unpack_codes has written) in boxes of 64 channels and a page's rows; 128-byte
// swizzle.
cudaError_t launch_unpack_codes(int D, const WindowParams &p, void *keys, void *values, cudaStream_t stream);
cudaError_t launch_window_prompt(qasa_dtype dt, int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                 const WindowParams &p, cudaStream_t stream);
cudaError_t launch_select(qasa_dtype dt, int D, const SelectParams &p, int units, cudaStream_t stream);
cudaError_t launch_attention(qasa_dtype dt, int D, int P, const CUtensorMap &km, const CUtensorMap &vm,
                             const AttnParams &p, int grid, size_t smem_budget, bool pdl,
                             cudaStream_t stream);
// One launch for the whole decode step (scoring, selection, attention);
// cooperative, grid = one CTA per SM.
cudaError_t launch_fused_decode(qasa_dtype dt, int D, int P, const CUtensorMap &km, const CUtensorMap &vm,
                                const AttnParams &p, int grid, size_t smem_budget, cudaStream_t stream);

cudaError_t launch_rebuild_bounds(qasa_dtype dt, int D, const RebuildParams &p, int batch,
                                  cudaStream_t stream);
cudaError_t launch_page_mass(qasa_dtype dt, int D, const MassParams &p, int units, cudaStream_t stream);
cudaError_t launch_page_hit(const HitParams &p, int units, cudaStream_t stream);

}  // namespace qasa
