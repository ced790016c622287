// window.cuh -- rules and helpers shared by the windowed-attention kernels.
#pragma once

#include "qasa_device.cuh"
#include "qasa_launch.h"

namespace qasa {

// Keys come in tiles of 16 tokens, the smaller page size: a tile never leaves
// its page, whatever that is.
constexpr int kTile = 16;

// Length of sequence b, its count of new tokens and the position of the first
// of them (negative where there are more queries than tokens).
struct QuerySpan { int len, n, first; };

__device__ __forceinline__ QuerySpan query_span(const WindowParams &p, int b, bool report) {
    QuerySpan s;
    int32_t *status = report ? p.status : nullptr;
    s.len = valid_len(p.seq_lens[b], p.max_pages, p.P, status);
    s.n = p.q_lens ? p.q_lens[b] : p.T;
    if (s.n < 0 || s.n > p.T) {
        if (status) atomicOr(status, QASA_DEVERR_APPEND);
        s.n = s.n < 0 ? 0 : p.T;
    }
    s.first = s.len - s.n;
    return s;
}

// The tiles that some query at a position in [first, last] can see: the tiles of
// the sinks that lie before the window of the first query, then the tiles from
// that window's start to `last`.
struct VisibleTiles {
    int lo, hi;          // tokens [lo, hi] are in somebody's window
    int head, body0;     // sink tiles 0 .. head, then tiles body0 ..
    int count;
    __device__ __forceinline__ int tile(int k) const { return k < head ? k : body0 + k - head; }
};

__device__ __forceinline__ VisibleTiles visible_tiles(int first, int last, int window, int sinks) {
    VisibleTiles v;
    v.hi = last;
    v.lo = first - window + 1 > 0 ? first - window + 1 : 0;
    v.body0 = v.lo / kTile;
    const int before = sinks < v.lo ? sinks : v.lo;
    v.head = min((before + kTile - 1) / kTile, v.body0);
    v.count = last < 0 ? 0 : v.head + last / kTile - v.body0 + 1;
    return v;
}

// Whether the query at position i sees token j.
__device__ __forceinline__ bool sees(int i, int j, int window, int sinks) {
    return j <= i && (j < sinks || j > i - window);
}

// Weights are exp2(score - m) with m this far below the largest score (log2 units),
// which the sums and outputs carry too, so that it cancels.  fp16 weights of the
// largest scores are then 2^7, and only those 2^-21 times as large fall below its
// normal numbers, where a rounding is no longer relative: values under a large E4M3
// scale may still count for something there.  bf16 has fp32's range.
template <typename T> constexpr float kHeadroom = elem<T>::id == QASA_DTYPE_F16 ? 7.f : 0.f;
// Sum of the weights that one pass gives a row from which on it looks for its own
// maximum: every single weight is inside fp16 up to there.
constexpr float kMostWeight = 32768.f;

// First pool row (token slot) of tile `t` for KV head h, or -1 for a bad page.
__device__ __forceinline__ long long tile_row(const WindowParams &p, const int32_t *table, int t, int h, int &phys) {
    const int per_page = p.P / kTile;
    phys = table[t / per_page];
    if (phys < 0 || phys >= p.num_phys) {
        if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
        phys = -1;
        return -1;
    }
    return ((long long)phys * p.Hkv + h) * p.P + (t % per_page) * kTile;
}

// Four E4M3 codes as four halves, exactly.
__device__ __forceinline__ void codes_to_h(uint32_t c, uint32_t *h) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h[0]), "=r"(h[1]) : "r"(c));
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(const void *smem, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(smem)), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_v2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace qasa
