// keep.cu -- tokens that stay move together: the accepted path of a tree of drafted
// tokens, or any ascending list of a sequence's tokens, goes to consecutive positions
// behind a start; boxes and E4M3 scales follow.
//
// Token start + keep[i] goes to start + i.  The list ascends, so a token never moves up
// and what is written at a position is only ever read for positions at or before it:
// pages are taken in rounds, in order, every row of a round read into shared memory
// before any of it is written.  A round is as many pages as a cluster of CTAs holds,
// one warp to a page of a KV head's K or V, so a round costs one barrier and its rows
// are all under way at once.  Rounds need no barrier between them: a later round reads
// no position that an earlier one wrote.
//
// Long lists are bound by their rounds, each a chain list -> block table -> rows -> barrier
// -> rows written, under as many other clusters as there are units for (each row read and
// written once: 4096 of 16384 tokens of 8 sequences, bf16, 62 us, 4.4 TB/s, 3.4 CTAs per
// SM); an accepted path is one such chain (64 sequences, up to 6 of 32 tokens, E4M3: 5.9 us).
//
// The box is taken from all the tokens that the page then has, the earlier ones read
// again: tokens that were given up leave it.  An E4M3 page keeps its scale while the
// rows that come from other pages fit it; else it grows and the page's codes follow, in
// the fp32 steps of the appends.
#include "page_rows.cuh"
#include "qasa_launch.h"
#include "window.cuh"

namespace qasa {

namespace {

// Warps of a CTA and CTAs of a cluster: 4096 of 16384 tokens of 8 sequences, 8 KV heads,
// bf16, d = 128: 4 and 4 62 us, 8 and 2 63, 8 and 8 67, 4 and 8 72, 8 and 4 77, 16 and 8 95;
// 4 and 4 with the next round's rows fetched into a second buffer 82, with the halves of
// a row in units of their own 60.
constexpr int kMostWarps = 4;
constexpr int kMostCluster = 4;

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Magnitudes of four codes, which are in the order of their values; a NaN's, 0x7f, counts as
// zero: it takes no finite code beside it out of the largest one.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
    w &= 0x7f7f7f7fu;
    return w & ~(((w + 0x01010101u) >> 7 & 0x01010101u) * 0xffu);
}

// Length of the list that holds: `n` entries, or up to the first that does not ascend or
// lies at or past `end` (positions counted from the start).  All threads of the cluster,
// whose CTAs look at a part of the list each.
__device__ __forceinline__ int good_entries(const int32_t *keep, int n, int end, int rank, int cluster) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = n;
    __syncthreads();
    int mine = n;
#pragma unroll 4
    for (int i = rank * blockDim.x + threadIdx.x; i < n; i += cluster * blockDim.x) {
        const int at = __ldg(keep + i), before = i ? __ldg(keep + i - 1) : -1;
        if (at <= before || at >= end) mine = min(mine, i);
    }
    if (mine < n) atomicMin(&bad, mine);
    if (cluster == 1) {
        __syncthreads();
        return bad;
    }
    cluster_sync();
    int least = n;
    for (int k = 0; k < cluster; ++k) least = min(least, ld_cluster_s32(map_rank(&bad, k)));
    cluster_sync();                                // nobody leaves while its word is read
    return least;
}

// T: type of the pool's elements as chunks go (E4M3: codes).
template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(kMostWarps * 32) keep_kernel(KeepParams p) {
    constexpr int ROWB = D * (FP8 ? 1 : (int)sizeof(T));       // bytes of a row
    constexpr int LPR = FP8 ? ROWB / 16 : ROWB / 32;           // lanes of a row: 16 codes, or two 16-byte chunks
    constexpr int RPP = 32 / LPR;
    extern __shared__ __align__(128) unsigned char smem[];

    const int cluster = p.cluster, rank = blockIdx.x % cluster, unit = blockIdx.x / cluster;
    const int which = unit & 1, h = (unit >> 1) % p.Hkv, b = (unit >> 1) / p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const bool first = rank == 0 && h == 0 && which == 0 && threadIdx.x == 0;

    int32_t *status = first ? p.status : nullptr;
    const int L = valid_len(p.seq_lens[b], p.max_pages, p.P, status);
    int start = p.starts[b], n = p.keep_lens ? p.keep_lens[b] : p.M, err = 0;
    if (start < 0 || start > L) { err |= QASA_DEVERR_SEQ_LEN; start = start < 0 ? 0 : L; }
    if (n < 0 || n > p.M) { err |= QASA_DEVERR_APPEND; n = n < 0 ? 0 : p.M; }
    const int32_t *keep = p.keep + (size_t)b * p.M;
    const int good = good_entries(keep, n, L - start, rank, cluster);
    if (good < n) { err |= QASA_DEVERR_KEEP; n = good; }
    if (first) {
        if (err && p.status) atomicOr(p.status, err);
        if (p.lens_out) p.lens_out[b] = start + n;
    }
    const int end = start + n, page0 = start / p.P;
    const int pages = (end + p.P - 1) / p.P - page0;           // the start's page counts if it holds earlier tokens
    const int per_round = cluster * warps;
    const int32_t *table = p.block_table + (size_t)b * p.max_pages;
    unsigned char *pool = static_cast<unsigned char *>(which ? p.v_pool : p.k_pool);
    unsigned char *mine = smem + (size_t)warp * p.P * ROWB;

    // A warp's page of a round: its rows and where this lane's slot comes from and goes to.
    struct Place {
        int rows, src, dst, phys;                              // src, dst: pool rows; phys < 0: no page
        bool other;                                            // it comes from another page,
        float from, old;                                       // E4M3: of this amax; the page's own
    };
    auto look_up = [&](int at) {
        Place x{0, -1, -1, -1, false, 0.f, 0.f};
        if (at >= pages) return x;
        const int page = page0 + at, base = page * p.P, pos = base + lane;
        const int from = pos >= start && pos < end && lane < p.P ? start + __ldg(keep + pos - start) : pos;
        const int phys = table[page];
        if (phys < 0 || phys >= p.num_phys) {
            if (lane == 0 && p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
            return x;
        }
        x.phys = phys;
        x.rows = min(p.P, end - base);
        if (lane < x.rows) {
            x.dst = x.src = (phys * p.Hkv + h) * p.P + lane;
            const int fp = from / p.P;
            if (fp == page) {
                x.src = x.dst - lane + from % p.P;
            } else {
                const int sp = table[fp];
                x.other = sp >= 0 && sp < p.num_phys;
                if (!x.other && p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
                if (x.other) {
                    x.src = (sp * p.Hkv + h) * p.P + from % p.P;
                    if constexpr (FP8) x.from = p.scales[((size_t)sp * p.Hkv + h) * 4 + which];
                }
            }
        }
        if constexpr (FP8) x.old = p.scales[((size_t)phys * p.Hkv + h) * 4 + which];
        return x;
    };
    // every CTA of the cluster goes through the same rounds
    Place next = look_up(rank * warps + warp);
    for (int round = 0; round < pages; round += per_round) {
        const int at = round + rank * warps + warp;
        const int rows = next.rows, src = next.src, dst = next.dst, phys = next.phys;
        const bool other = next.other;
        const float amax_src = next.from, old = next.old;
        const int need = FP8 || !which ? 0 : max(start - (page0 + at) * p.P, 0);   // V: earlier rows stay as they are
        // all rows of the page under way, then everybody's
        for (int x0 = 0; x0 < rows * (ROWB / 16); x0 += 32) {
            const int r = (x0 + lane) / (ROWB / 16), c = (x0 + lane) % (ROWB / 16);
            const int from = __shfl_sync(0xffffffffu, src, r & 31);
            if (r >= need && r < rows) copy_async16(smem_u32(mine + r * ROWB + c * 16), pool + (size_t)from * ROWB + c * 16);
        }
        // the next round's places meanwhile; its scales are those of pages that no round before has written
        next = look_up(at + per_round);
        copy_async_wait();
        if (cluster > 1) cluster_sync(); else __syncthreads();
        __syncwarp();

        if constexpr (FP8) {
            const int c = lane % LPR;
            float top = 0.f;
            for (int r0 = 0; r0 < rows; r0 += RPP) {           // the largest |value| that comes from other pages
                const int r = r0 + lane / LPR;
                const float s = fp8_scale(__shfl_sync(0xffffffffu, amax_src, r & 31));
                const bool comes = __shfl_sync(0xffffffffu, (int)other, r & 31) != 0 && r < rows;
                if (comes) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(mine + r * ROWB + c * 16);
                    uint32_t m = __vmaxu4(__vmaxu4(magnitudes(w.x), magnitudes(w.y)), __vmaxu4(magnitudes(w.z), magnitudes(w.w)));
                    m = __vmaxu4(m, m >> 16);
                    m = max(m & 0xffu, m >> 8 & 0xffu);
                    top = fmaxf(top, __fmul_rn(e4m3_to_f(m), s));
                }
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float amax = fmaxf(old, top);
            const bool grown = amax > old;
            Box<__half> box;
            box.clear();
            for (int r0 = 0; r0 < rows; r0 += RPP) {
                const int r = r0 + lane / LPR;
                const float a = __shfl_sync(0xffffffffu, amax_src, r & 31);
                const bool comes = __shfl_sync(0xffffffffu, (int)other, r & 31) != 0;
                const int from = __shfl_sync(0xffffffffu, src, r & 31), to = __shfl_sync(0xffffffffu, dst, r & 31);
                if (r >= rows) continue;
                uint4 w = *reinterpret_cast<const uint4 *>(mine + r * ROWB + c * 16);
                if (comes || grown) {
                    const float was = comes ? a : old, by = __fdiv_rn(was, amax);
                    const uint2 lo = recode8(make_uint2(w.x, w.y), by, was, amax), hi = recode8(make_uint2(w.z, w.w), by, was, amax);
                    w = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
                if (comes || grown || from != to) *reinterpret_cast<uint4 *>(pool + (size_t)to * ROWB + c * 16) = w;
                if (!which) box.fold(codes_to_halves(make_uint2(w.x, w.y)), codes_to_halves(make_uint2(w.z, w.w)));
            }
            if (rows > 0 && grown && lane == 0) p.scales[((size_t)phys * p.Hkv + h) * 4 + which] = amax;
            if (!which) {
                box.template join<LPR>();
                if (rows > 0 && lane < LPR) {
                    unsigned char *row = static_cast<unsigned char *>(p.bounds) + ((size_t)phys * p.Hkv + h) * 2 * ROWB + c * 16;
                    const uint2 l0 = halves_to_codes(box.lo), l1 = halves_to_codes(box.lo + 4);
                    const uint2 h0 = halves_to_codes(box.hi), h1 = halves_to_codes(box.hi + 4);
                    *reinterpret_cast<uint4 *>(row) = make_uint4(l0.x, l0.y, l1.x, l1.y);
                    *reinterpret_cast<uint4 *>(row + ROWB) = make_uint4(h0.x, h0.y, h1.x, h1.y);
                }
            }
        } else {
            const int c = lane % LPR * 32;
            Box<T> box;
            box.clear();
            for (int r0 = need / RPP * RPP; r0 < rows; r0 += RPP) {
                const int r = r0 + lane / LPR;
                const int from = __shfl_sync(0xffffffffu, src, r & 31), to = __shfl_sync(0xffffffffu, dst, r & 31);
                if (r >= rows || r < need) continue;
                const uint4 a = *reinterpret_cast<const uint4 *>(mine + r * ROWB + c);
                const uint4 e = *reinterpret_cast<const uint4 *>(mine + r * ROWB + c + 16);
                if (from != to) {
                    uint4 *out = reinterpret_cast<uint4 *>(pool + (size_t)to * ROWB + c);
                    out[0] = a;
                    out[1] = e;
                }
                if (!which) box.fold(a, e);
            }
            if (!which) {
                box.template join<LPR>();
                if (rows > 0 && lane < LPR) {
                    unsigned char *row = static_cast<unsigned char *>(p.bounds) + ((size_t)phys * p.Hkv + h) * 2 * ROWB + c;
                    uint4 *lo = reinterpret_cast<uint4 *>(row), *hi = reinterpret_cast<uint4 *>(row + ROWB);
                    lo[0] = make_uint4(box.lo[0], box.lo[1], box.lo[2], box.lo[3]);
                    lo[1] = make_uint4(box.lo[4], box.lo[5], box.lo[6], box.lo[7]);
                    hi[0] = make_uint4(box.hi[0], box.hi[1], box.hi[2], box.hi[3]);
                    hi[1] = make_uint4(box.hi[4], box.hi[5], box.hi[6], box.hi[7]);
                }
            }
        }
        __syncwarp();                                          // the next round's copies come over this one's rows
    }
}

template <typename T, int D, bool FP8>
cudaError_t launch_t(KeepParams p, int batch, cudaStream_t stream) {
    const int most = (p.M + p.P - 2) / p.P + 1;                // pages that M tokens touch
    const int warps = most < kMostWarps ? most : kMostWarps;
    const int fill = (most + warps - 1) / warps;
    p.cluster = fill < kMostCluster ? fill : kMostCluster;
    const size_t smem = (size_t)warps * p.P * D * (FP8 ? 1 : sizeof(T));
    const long long grid = 2LL * batch * p.Hkv * p.cluster;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kernel = keep_kernel<T, D, FP8>;
    if (smem + 64 > 48 << 10) {                                // and the static word
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_keep(qasa_dtype dt, int D, const KeepParams &p, int batch, cudaStream_t stream) {
    switch (dt) {
    case QASA_DTYPE_E4M3:
        return D == 64 ? launch_t<__half, 64, true>(p, batch, stream) : launch_t<__half, 128, true>(p, batch, stream);
    case QASA_DTYPE_F32:
        return D == 64 ? launch_t<float, 64, false>(p, batch, stream) : launch_t<float, 128, false>(p, batch, stream);
    case QASA_DTYPE_F16:
        return D == 64 ? launch_t<__half, 64, false>(p, batch, stream) : launch_t<__half, 128, false>(p, batch, stream);
    default:
        return D == 64 ? launch_t<__nv_bfloat16, 64, false>(p, batch, stream)
                       : launch_t<__nv_bfloat16, 128, false>(p, batch, stream);
    }
}

}  // namespace qasa
