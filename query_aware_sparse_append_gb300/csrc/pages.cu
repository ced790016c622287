// pages.cu -- whole pages copied inside the pools, and sequences forked: children
// share their parent's full pages and get a copy of its part-filled one.
//
// Nothing is computed: both are bound by the bytes, each read and written once.  A
// page is two contiguous tiles (all KV heads of K, then of V), its boxes and, E4M3,
// its scales; a block takes a fixed number of its 16-byte chunks, so that blocks are
// alike whatever the page's size, and every thread has its loads under way at once.
// The chain is id -> chunk -> store; many small blocks per SM overlap it.  16384 pages of
// 32 KB, f16: 170 us, 6.7 TB/s, the copy rate; 192 part-filled pages for 256 children, 25 MB
// with their rows, 7.9 us; a few pages 2.3 us.
#include "qasa_device.cuh"
#include "qasa_launch.h"

namespace qasa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                        // chunks of a thread under way
constexpr int kPiece = kThreads * kUnroll;        // chunks of a block: 16 KB

// 16-byte chunks of a page: K tile, V tile, boxes, scales.
struct PageChunks {
    int tile, box, scale;
    __host__ __device__ int all() const { return 2 * tile + box + scale; }
};

__host__ __device__ inline PageChunks page_chunks(const PageCopyParams &p) {
    return {p.Hkv * p.P * p.row_chunks, p.Hkv * 2 * p.row_chunks, p.scales ? p.Hkv : 0};
}

__device__ __forceinline__ uint4 *chunk_at(const PageCopyParams &p, const PageChunks &n, int page, int x) {
    if (x < n.tile) return static_cast<uint4 *>(p.k_pool) + (size_t)page * n.tile + x;
    x -= n.tile;
    if (x < n.tile) return static_cast<uint4 *>(p.v_pool) + (size_t)page * n.tile + x;
    x -= n.tile;
    if (x < n.box) return static_cast<uint4 *>(p.bounds) + (size_t)page * n.box + x;
    return reinterpret_cast<uint4 *>(p.scales) + (size_t)page * n.scale + (x - n.box);
}

// `piece` of the page's chunks; rows < 0: all of them, else slots below `rows`.
__device__ __forceinline__ void copy_piece(const PageCopyParams &p, int src, int dst, int piece, int rows) {
    const PageChunks n = page_chunks(p);
    const int part = rows < 0 ? n.tile : p.Hkv * rows * p.row_chunks;       // chunks of a tile to copy
    const int count = 2 * part + n.box + n.scale;
    uint4 v[kUnroll];
    int at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        int x = piece * kPiece + u * kThreads + threadIdx.x;
        at[u] = -1;
        if (x >= count) continue;
        if (rows >= 0) {                          // the chunk's place in the whole page
            if (x < 2 * part) {
                const int v_tile = x >= part, y = x - v_tile * part, head = rows * p.row_chunks;
                x = v_tile * n.tile + y / head * (p.P * p.row_chunks) + y % head;
            } else {
                x += 2 * (n.tile - part);
            }
        }
        at[u] = x;
        v[u] = *chunk_at(p, n, src, x);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (at[u] >= 0) *chunk_at(p, n, dst, at[u]) = v[u];
}

__device__ __forceinline__ bool in_pool(const PageCopyParams &p, int page) { return page >= 0 && page < p.num_phys; }

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(PageCopyParams p) {
    const int pair = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
    const int src = p.src_pages[pair], dst = p.dst_pages[pair];
    if (!in_pool(p, src) || !in_pool(p, dst)) {
        if (piece == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
        return;
    }
    if (src != dst) copy_piece(p, src, dst, piece, -1);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(PageCopyParams p) {
    const int child = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
    const bool report = piece == 0 && threadIdx.x == 0 && p.status;
    const int parent = p.parents[child];
    if (parent < 0 || parent >= p.batch) {
        if (report) atomicOr(p.status, QASA_DEVERR_PARENT);
        return;
    }
    const int L = valid_len(p.seq_lens[parent], p.max_pages, p.P, report ? p.status : nullptr);
    const int full = L / p.P, rows = L % p.P;
    const int32_t *from = p.block_table + (size_t)parent * p.max_pages;
    int32_t *to = p.table_out + (size_t)child * p.max_pages;
    int src = -1, dst = -1;
    if (rows > 0) {
        src = from[full];
        dst = p.new_pages[child];
        if (dst < 0) dst = src;                   // the parent's own page is taken over
        if (!in_pool(p, src) || !in_pool(p, dst)) {
            if (report) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
            return;
        }
    }
    for (int i = piece * kThreads + threadIdx.x; i < full + (rows > 0); i += p.pieces * kThreads)
        to[i] = i < full ? from[i] : dst;
    if (p.lens_out && piece == 0 && threadIdx.x == 0) p.lens_out[child] = L;
    if (src != dst) copy_piece(p, src, dst, piece, rows);
}

}  // namespace

// Blocks per page, each of kPiece chunks.
int page_pieces(const PageCopyParams &p) { return (page_chunks(p).all() + kPiece - 1) / kPiece; }

cudaError_t launch_copy_pages(const PageCopyParams &p, int pairs, cudaStream_t stream) {
    copy_pages_kernel<<<(unsigned)((long long)pairs * p.pieces), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fork(const PageCopyParams &p, int children, cudaStream_t stream) {
    fork_kernel<<<(unsigned)((long long)children * p.pieces), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace qasa
