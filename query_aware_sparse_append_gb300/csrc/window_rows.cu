// window_rows.cu -- windowed attention for few query rows (tokens x heads of the
// group) per KV head: the decode step and, up to 16 rows, drafted tokens; E4M3 up to
// 128 rows, as their pages need no unpacking here; every fp32 call.
//
//   out(i) = sum_j softmax_j(scale q_i . k_j) v_j  over  j <= i, j < sinks or j > i - window
//
// What bounds it: the visible keys and values are read once from HBM and meet at
// most 16 query rows, so it is a stream of pages with a few operations per byte;
// with few sequences it is the chain of dependent loads (length, block table,
// page) and the joins.
//
// Split: the rows (token, query head of the group) of a sequence and KV head form
// row tiles of 16 (8 where no more exist); a row tile is a unit, worked on by a
// cluster of 1 to 8 CTAs.  The unit's 16-token tiles go round the warps of the
// cluster, each warp keeping its own running maximum, sum and output, so nothing
// waits inside the loop.  At the end the warps of a CTA are joined through its
// shared memory and the CTAs through distributed shared memory: no workspace, no
// counters, one launch, and always in the same order.
//
// Each warp has a ring of its own, filled by asynchronous 16-byte copies that hold
// no registers: keys, values and the next keys are under way while it computes, and
// four CTAs of four warps fit an SM, 128 KB and more in flight there (loads straight
// into registers left two CTAs, 43 % of the copy rate).  Chunks go from the ring
// into the fragments of m16n8k16 products as they are, tokens and channels as the 16
// rows and the query rows as the 8 columns (the other way round half of every product
// is empty at a group of 8).  A lane's 16-byte chunk of a key row is read as the pairs
// of k-steps; q's fragments take the same channel order, and the sum over channels
// does not care about it.  Values need pairs of tokens per channel: a lane takes the
// same channels of two neighbouring rows and interleaves the halves with byte
// permutes.  As in the prompt kernel a step's maximum is sought only where its
// weights grow large.
//
// TREE: the queries are a tree of drafted tokens; only which tokens they see differs.
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kMaxCluster = 8;

// Joins the partial states of a unit and writes its rows.  Every warp of the CTA
// has left ROWS rows of o[D] and (m, l) in shared memory: m the running maximum
// in log2 units (-inf where the warp saw nothing), l the sum of weights: 0 where it
// saw nothing, NaN of a query that has one, whose scores no maximum takes up.
template <typename T, int D, int ROWS, int W>
__device__ __forceinline__ void join_and_write(const WindowParams &p, float *part_o, float2 *part_ml, int cluster,
                                               int row0, int rows, int b, int h) {
    constexpr int CH = D / 4;                        // float4 chunks of a row
    __syncthreads();
    // the CTA's warps: slot 0 takes the joined state
    float2 *sum_ml = part_ml + W * ROWS;
    for (int x = threadIdx.x; x < ROWS * CH; x += W * 32) {
        const int r = x / CH, c = x % CH;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, part_ml[w * ROWS + r].x);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 ml = part_ml[w * ROWS + r];
            if (ml.y == 0.f) continue;
            const float f = exp2f(ml.x - m);
            const float4 v = reinterpret_cast<const float4 *>(part_o + ((size_t)w * ROWS + r) * D)[c];
            l = fmaf(f, ml.y, l);
            o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
        }
        reinterpret_cast<float4 *>(part_o + (size_t)r * D)[c] = o;   // only this thread read chunk (r, c)
        if (c == 0) sum_ml[r] = make_float2(m, l);
    }
    if (cluster > 1) cluster_sync(); else __syncthreads();
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    for (int x = rank * (W * 32) + threadIdx.x; x < rows * CH; x += cluster * W * 32) {
        const int r = x / CH, c = x % CH;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        if (cluster == 1) {
            o = reinterpret_cast<const float4 *>(part_o + (size_t)r * D)[c];
            l = sum_ml[r].y;
        } else {
            float2 ml[kMaxCluster];
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < cluster) {
                    ml[k] = ld_cluster_v2(map_rank(sum_ml + r, k));
                    m = fmaxf(m, ml[k].x);
                }
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < cluster && ml[k].y != 0.f) {
                    const float4 v = ld_cluster_v4(map_rank(part_o + (size_t)r * D + 4 * c, k));
                    const float f = exp2f(ml[k].x - m);
                    l = fmaf(f, ml[k].y, l);
                    o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
                    o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
                }
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing is zero
        const int row = row0 + r, t = row / p.G, g = row % p.G;
        T *dst = static_cast<T *>(p.out) + (((size_t)b * p.T + t) * p.Hq + h * p.G + g) * D + 4 * c;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(mma16816<T>::pack2(o.x * inv, o.y * inv),
                                                         mma16816<T>::pack2(o.z * inv, o.w * inv));
        }
    }
    if (cluster > 1) cluster_sync();                 // nobody leaves while its state is read
}

template <int D, int ROWS, int W>
constexpr size_t rows_smem() { return (size_t)W * ROWS * D * 4 + (size_t)(W + 1) * ROWS * 8; }

// ------------------------------------------------------- 16-bit and E4M3 pages

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

constexpr int kSlots = 3;                      // copies under way per warp: keys, values, the next keys

// What a warp takes at once: `TPS` tiles, so that a copy is 4 KB (2 KB: E4M3, d 64).
template <bool FP8, int D> struct Step {
    static constexpr int ROWB = D * (FP8 ? 1 : 2);         // bytes of a row
    static constexpr int TPS = ROWB == 256 ? 1 : 2;
    static constexpr int BYTES = TPS * kTile * ROWB;
    static constexpr int KC = ROWB / 64;                   // 16-byte chunks of a key row per lane
    static constexpr bool V8 = ROWB == 64;                 // a lane's share of a value row is 8 bytes
    static constexpr int VC = V8 ? 1 : ROWB / 128;         // chunks of a value row per lane
};

template <bool FP8, int D, int ROWS, int W>
constexpr size_t step_smem() {
    constexpr size_t ring = (size_t)W * kSlots * Step<FP8, D>::BYTES;
    constexpr size_t most = ring > rows_smem<D, ROWS, W>() ? ring : rows_smem<D, ROWS, W>();
    static_assert(most <= 48 << 10, "no opt-in needed");
    return most;
}

// T: type of q and out; FP8: pages of E4M3 codes (T is __half).
template <typename T, bool FP8, int D, int ROWS, int W, bool TREE>
__global__ void __launch_bounds__(W * 32, ROWS == 8 ? 4 : 3) window_rows_kernel(WindowParams p) {
    using R = Step<FP8, D>;
    constexpr int NH = ROWS / 8;              // query rows are the products' columns, 8 at a time
    constexpr int KS = D / 16;                // k-steps of the scores
    constexpr int VCH = D / 8 / R::VC;        // channels of a value chunk (8 or 16)
    constexpr int TPS = R::TPS, ROWB = R::ROWB;

    extern __shared__ __align__(128) unsigned char smem[];
    float *part_o = reinterpret_cast<float *>(smem);
    float2 *part_ml = reinterpret_cast<float2 *>(smem + (size_t)W * ROWS * D * 4);

    const int cluster = p.cluster;
    const int unit = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int h = unit % p.Hkv, rt = unit / p.Hkv % p.row_tiles, b = unit / p.Hkv / p.row_tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const QuerySpan s = query_span(p, b, h == 0 && rt == 0 && rank == 0 && threadIdx.x == 0);
    const int row0 = rt * ROWS;
    const int rows = min(ROWS, s.n * p.G - row0);
    if (rows <= 0) return;                    // the same for the whole cluster
    const int t0 = row0 / p.G, t1 = (row0 + rows - 1) / p.G;
    // a tree's queries may be at any depth and see any drafted token
    const VisibleTiles vis = TREE ? visible_tiles(s.first, s.len - 1, p.window, p.sinks)
                                  : visible_tiles(s.first + t0, s.first + t1, p.window, p.sinks);
    const int32_t *table = p.block_table + (size_t)b * p.max_pages;

    // This warp's tiles are number wg, wg + stride, ... of the visible ones.  Lane x
    // holds the pool row (and scales) of tile from + x, and those of the 32 after.
    const int stride = cluster * W, wg = rank * W + warp;
    const int mine = vis.count > wg ? (vis.count - wg + stride - 1) / stride : 0;
    const int steps = (mine + TPS - 1) / TPS;
    struct Place { int row; float ks, vs; };
    auto look_up = [&](int x) {
        Place a{-1, 0.f, 0.f};
        if (x < mine) {
            int phys;
            a.row = (int)tile_row(p, table, vis.tile(wg + x * stride), h, phys);      // below 2^31: checked on the host
            if (FP8 && phys >= 0) {
                const float2 amax = __ldg(reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + h) * 4));
                a.ks = fp8_scale(amax.x);
                a.vs = fp8_scale(amax.y);
            }
        }
        return a;
    };
    Place here = look_up(lane), there = look_up(32 + lane);
    int from = 0;                              // `here` is tiles [from, from + 32)

    const int g4 = lane >> 2, q4 = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * kSlots * R::BYTES;
    const unsigned char *pools[2] = {static_cast<const unsigned char *>(p.k_pool), static_cast<const unsigned char *>(p.v_pool)};
    // Copy number c: keys (even) or values (odd) of step c / 2.  Chunks are spread so
    // that the eight lanes of a shared-memory phase, which read two key rows or four
    // value rows, meet different banks.
    auto fetch = [&](int c, int slot) {
        const int step = c >> 1, v = c & 1;
        if (step < steps) {
            const uint32_t dst = ring + slot * R::BYTES;
#pragma unroll
            for (int t = 0; t < TPS; ++t) {
                const int x = step * TPS + t - from;              // at most one step past `here`
                const int row = x < 32 ? __shfl_sync(0xffffffffu, here.row, x) : __shfl_sync(0xffffffffu, there.row, x - 32);
                if (row < 0) continue;
                const unsigned char *src = pools[v] + (size_t)row * ROWB + lane * 16;
#pragma unroll
                for (int it = 0; it < kTile * ROWB / 512; ++it) {
                    const int id = it * 32 + lane, r = id / (ROWB / 16), ch = id % (ROWB / 16);
                    const int f = ROWB == 64 ? 0 : v ? (r & 6) : (r & 1) << 2;
                    copy16(dst + t * kTile * ROWB + r * ROWB + ((ch ^ f) << 4), src + it * 512);
                }
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int c = 0; c < kSlots; ++c) fetch(c, c);

    // q fragments: query row 8 x + g4, channels in the order of the key chunks
    uint32_t qb[NH][KS][2];
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        const int r = 8 * x + g4;
        const bool live = r < rows;
        const int t = (row0 + (live ? r : 0)) / p.G, g = (row0 + (live ? r : 0)) % p.G;
        const T *row = static_cast<const T *>(p.q) + (((size_t)b * p.T + t) * p.Hq + h * p.G + g) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            // 8 channels: four k-step halves.  Key chunks have 8 (16-bit) or 16 (E4M3) channels.
            const int c = FP8 ? (q4 + 4 * (j / 2)) * 16 + 8 * (j & 1) : (q4 + 4 * j) * 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = ld_global_nc_v4(row + c);
            qb[x][2 * j][0] = w.x;
            qb[x][2 * j][1] = w.y;
            qb[x][2 * j + 1][0] = w.z;
            qb[x][2 * j + 1][1] = w.w;
        }
    }
    // a lane's scores and outputs belong to query rows 8 x + 2 q4 and the one after
    int pos[NH][2];
    const uint32_t *mask[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = (row0 + min(8 * x + 2 * q4 + e, rows - 1)) / p.G;
            if constexpr (TREE) mask[x][e] = tree_row(p, b, t);
            pos[x][e] = s.first + (TREE ? tree_depth(p, mask[x][e], s.n) : t);
        }

    // o[c][u]: channels 2 u (elements 0, 1) and 2 u + 1 (2, 3) of this lane's chunk c
    float o[R::VC][VCH / 2][NH][4];
#pragma unroll
    for (int c = 0; c < R::VC; ++c)
#pragma unroll
        for (int u = 0; u < VCH / 2; ++u)
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][u][x][e] = 0.f;
    auto scale_o = [&](int x, float f0, float f1) {
#pragma unroll
        for (int c = 0; c < R::VC; ++c)
#pragma unroll
            for (int u = 0; u < VCH / 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][u][x][e] *= (e & 1) ? f1 : f0;
    };
    float m[NH][2], l[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x) { m[x][0] = m[x][1] = -INFINITY; l[x][0] = l[x][1] = 0.f; }
    bool unset = true;                        // some row has seen nothing yet
    float vref = 0.f, inv_vref = 0.f;         // E4M3: o is in units of the largest V scale so far

    int slot = 0;
    for (int i = 0; i < steps; ++i) {
        if (i * TPS - from >= 32) {
            here = there;
            from += 32;
            there = look_up(from + 32 + lane);
        }
        int tok0[TPS];                        // first token of each tile
        bool good[TPS];                       // the tile was brought
        bool inside = true;                   // every row sees every token
#pragma unroll
        for (int t = 0; t < TPS; ++t) {
            const int x = i * TPS + t;
            tok0[t] = vis.tile(wg + x * stride) * kTile;
            good[t] = __shfl_sync(0xffffffffu, here.row, x - from) >= 0 && x < mine;
            inside = inside && good[t] && tok0[t] + kTile - 1 <= (TREE ? s.first - 1 : s.first + t0) &&
                     (tok0[t] + kTile <= p.sinks || tok0[t] > (TREE ? s.len - 1 : s.first + t1) - p.window);
        }

        // scores: tokens g4 (elements 0, 1) and g4 + 8 (2, 3) of a tile
        copy_wait<kSlots - 1>();
        __syncwarp();
        float sc[TPS][NH][4];
        uint32_t at = ring + slot * R::BYTES + g4 * ROWB;
#pragma unroll
        for (int t = 0; t < TPS; ++t) {
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][x][e] = 0.f;
#pragma unroll
            for (int j = 0; j < R::KC; ++j) {
                const int f = ROWB == 64 ? 0 : (g4 & 1) << 2;
                const uint32_t chunk = at + t * kTile * ROWB + (((q4 + 4 * j) ^ f) << 4);
                const uint4 c0 = lds16(chunk), c1 = lds16(chunk + 8 * ROWB);
                constexpr int KW = FP8 ? 8 : 4;
                uint32_t w0[KW], w1[KW];
                if constexpr (FP8) {
                    codes_to_h(c0.x, w0); codes_to_h(c0.y, w0 + 2); codes_to_h(c0.z, w0 + 4); codes_to_h(c0.w, w0 + 6);
                    codes_to_h(c1.x, w1); codes_to_h(c1.y, w1 + 2); codes_to_h(c1.z, w1 + 4); codes_to_h(c1.w, w1 + 6);
                } else {
                    w0[0] = c0.x; w0[1] = c0.y; w0[2] = c0.z; w0[3] = c0.w;
                    w1[0] = c1.x; w1[1] = c1.y; w1[2] = c1.z; w1[3] = c1.w;
                }
#pragma unroll
                for (int k = 0; k < KW / 2; ++k) {
                    const uint32_t a[4] = {w0[2 * k], w1[2 * k], w0[2 * k + 1], w1[2 * k + 1]};
#pragma unroll
                    for (int x = 0; x < NH; ++x)
                        mma16816<T>::run(sc[t][x], a, qb[x][KW / 2 * j + k][0], qb[x][KW / 2 * j + k][1]);
                }
            }
        }
        __syncwarp();
        fetch(2 * i + kSlots, slot);
        if (++slot == kSlots) slot = 0;

        // weights
        float vs[TPS];
#pragma unroll
        for (int t = 0; t < TPS; ++t) {
            float to_log2 = p.scale_log2;
            if constexpr (FP8) to_log2 *= __shfl_sync(0xffffffffu, here.ks, i * TPS + t - from);
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][x][e] *= to_log2;
            vs[t] = 1.f;
        }
        if (!inside) {
#pragma unroll
            for (int t = 0; t < TPS; ++t)
#pragma unroll
                for (int x = 0; x < NH; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (TREE) {
                            if (!good[t] || !tree_sees(mask[x][e & 1], pos[x][e & 1], tok0[t] + 8 * (e >> 1) + g4, s.first, s.len,
                                                       p.window, p.sinks))
                                sc[t][x][e] = -INFINITY;
                        } else {
                            if (!good[t] || !sees(pos[x][e & 1], tok0[t] + 8 * (e >> 1) + g4, p.window, p.sinks))
                                sc[t][x][e] = -INFINITY;
                        }
                    }
        }
        if constexpr (FP8) {
            float top = 0.f;
#pragma unroll
            for (int t = 0; t < TPS; ++t) {
                vs[t] = __shfl_sync(0xffffffffu, here.vs, i * TPS + t - from);
                top = fmaxf(top, vs[t]);
            }
            if (top > vref) {
                const float g = vref / top;
#pragma unroll
                for (int x = 0; x < NH; ++x) scale_o(x, g, g);
                vref = top;
                inv_vref = 1.f / top;
            }
#pragma unroll
            for (int t = 0; t < TPS; ++t) vs[t] *= inv_vref;
        }
        uint32_t pb[TPS][NH][2];
        bool hidden[TPS][4];
        bool raise = unset;
        while (true) {
            if (raise) {                      // the step's own maximum
                bool none = false;
#pragma unroll
                for (int x = 0; x < NH; ++x) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = -INFINITY;
#pragma unroll
                        for (int t = 0; t < TPS; ++t) top = fmaxf(top, fmaxf(sc[t][x][e], sc[t][x][2 + e]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float m_new = fmaxf(m[x][e], top - kHeadroom<T>);
                        f[e] = m_new == -INFINITY ? 1.f : exp2_fast(m[x][e] - m_new);
                        m[x][e] = m_new;
                        l[x][e] *= f[e];
                        none = none || m_new == -INFINITY;
                    }
                    scale_o(x, f[0], f[1]);
                }
                unset = __any_sync(0xffffffffu, none);
            }
            float sum[NH][2];
            bool small = true;
#pragma unroll
            for (int x = 0; x < NH; ++x) {
                const float b0 = m[x][0] == -INFINITY ? 0.f : m[x][0], b1 = m[x][1] == -INFINITY ? 0.f : m[x][1];
                sum[x][0] = sum[x][1] = 0.f;
#pragma unroll
                for (int t = 0; t < TPS; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float w0 = exp2_fast(sc[t][x][2 * k] - b0), w1 = exp2_fast(sc[t][x][2 * k + 1] - b1);
                        sum[x][0] += w0;
                        sum[x][1] += w1;
                        if constexpr (FP8) { w0 *= vs[t]; w1 *= vs[t]; }
                        // weights in the values' 16-bit type: half a step each, while the sum keeps fp32
                        pb[t][x][k] = mma16816<T>::pack2(w0, w1);
                    }
                small = small && sum[x][0] <= kMostWeight && sum[x][1] <= kMostWeight;
            }
            if (raise || __all_sync(0xffffffffu, small)) {
#pragma unroll
                for (int x = 0; x < NH; ++x) { l[x][0] += sum[x][0]; l[x][1] += sum[x][1]; }
                break;
            }
            raise = true;
        }
        // from pairs of rows per token to pairs of tokens per row
#pragma unroll
        for (int t = 0; t < TPS; ++t)
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int k = 0; k < 2; ++k) pb[t][x][k] = movmatrix_trans(pb[t][x][k]);

        // output
        copy_wait<kSlots - 1>();
        __syncwarp();
        at = ring + slot * R::BYTES + 2 * q4 * ROWB;
#pragma unroll
        for (int t = 0; t < TPS; ++t) {
            if constexpr (TREE) {             // drafted tokens that none of these rows sees
                if (!inside) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int j = tok0[t] + 2 * q4 + (y & 1) + 8 * (y >> 1) - s.first;
                        bool any = j < 0 || j >= s.n;
                        for (int i = t0; i <= t1 && !any; ++i) any = __ldg(tree_row(p, b, i) + (j >> 5)) >> (j & 31) & 1u;
                        hidden[t][y] = !any;
                    }
                }
            }
            uint4 vr[4][R::VC];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = 2 * q4 + (y & 1) + 8 * (y >> 1);
                const uint32_t row = at + (t * kTile + (y & 1) + 8 * (y >> 1)) * ROWB;
#pragma unroll
                for (int c = 0; c < R::VC; ++c) {
                    if constexpr (R::V8) {
                        uint2 w;
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(row + g4 * 8));
                        vr[y][c] = make_uint4(w.x, w.y, 0, 0);
                    } else {
                        vr[y][c] = lds16(row + (((g4 + 8 * c) ^ (r & 6)) << 4));
                    }
                    if (!inside) {            // values that no row sees may be anything: 0 * NaN is not 0
                        const int j = tok0[t] + r;
                        if (!good[t] || j > vis.hi || (j < vis.lo && j >= p.sinks) || (TREE && hidden[t][y]))
                            vr[y][c] = make_uint4(0, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < R::VC; ++c)
#pragma unroll
                for (int d = 0; d < VCH / (FP8 ? 4 : 2); ++d) {        // 32-bit words of a chunk
                    uint32_t r[4][FP8 ? 2 : 1];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint4 &w = vr[y][c];
                        const uint32_t word = d == 0 ? w.x : d == 1 ? w.y : d == 2 ? w.z : w.w;
                        if constexpr (FP8) codes_to_h(word, r[y]);
                        else r[y][0] = word;
                    }
#pragma unroll
                    for (int z = 0; z < (FP8 ? 2 : 1); ++z) {
                        const uint32_t a[4] = {__byte_perm(r[0][z], r[1][z], 0x5410), __byte_perm(r[0][z], r[1][z], 0x7632),
                                               __byte_perm(r[2][z], r[3][z], 0x5410), __byte_perm(r[2][z], r[3][z], 0x7632)};
#pragma unroll
                        for (int x = 0; x < NH; ++x)
                            mma16816<T>::run(o[c][(FP8 ? 2 : 1) * d + z][x], a, pb[t][x][0], pb[t][x][1]);
                    }
                }
        }
        __syncwarp();
        fetch(2 * i + 1 + kSlots, slot);
        if (++slot == kSlots) slot = 0;
    }

    // this warp's state, over the rings: chunk c of this lane is channels
    // (8 c + g4) VCH ..
    copy_wait<0>();
    __syncthreads();
    const float unitv = FP8 ? vref : 1.f;
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[x][e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int r = 8 * x + 2 * q4 + e;
            float *dst = part_o + ((size_t)warp * ROWS + r) * D;
#pragma unroll
            for (int c = 0; c < R::VC; ++c)
#pragma unroll
                for (int u = 0; u < VCH / 2; u += 2)
                    *reinterpret_cast<float4 *>(dst + (8 * c + g4) * VCH + 2 * u) =
                        make_float4(o[c][u][x][e] * unitv, o[c][u][x][2 + e] * unitv, o[c][u + 1][x][e] * unitv,
                                    o[c][u + 1][x][2 + e] * unitv);
            if (g4 == 0) part_ml[warp * ROWS + r] = make_float2(m[x][e], sum);
        }
    join_and_write<T, D, ROWS, W>(p, part_o, part_ml, cluster, row0, rows, b, h);
}

// ------------------------------------------------------------------ fp32 pages

// The same split with fused multiply-adds: fp32 products have no tensor path that
// keeps their precision.  Four lanes share a key row (8 rows under way per warp);
// the ROWS scores of a row are summed over the four by a butterfly that leaves
// each lane ROWS / 4 of them (all of them for ROWS < 4); the values are read a
// whole row at a time, a lane owning D / 32 channels.
template <int D, int ROWS, int W, bool TREE>
__global__ void __launch_bounds__(W * 32) window_rows_f32_kernel(WindowParams p) {
    constexpr int KC = D / 16;                 // float4 chunks of a key row per lane
    constexpr int VN = D / 32;                 // channels per lane
    constexpr int PARTS = ROWS == 1 ? 2 : 1;   // halves of a tile under way at once, as registers allow
    extern __shared__ __align__(128) unsigned char smem[];
    float *part_o = reinterpret_cast<float *>(smem);
    float2 *part_ml = reinterpret_cast<float2 *>(smem + (size_t)W * ROWS * D * 4);
    __shared__ __align__(16) float qs[ROWS][D];
    __shared__ __align__(16) float ps[W][8][ROWS];

    const int cluster = p.cluster;
    const int unit = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int h = unit % p.Hkv, rt = unit / p.Hkv % p.row_tiles, b = unit / p.Hkv / p.row_tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const QuerySpan s = query_span(p, b, h == 0 && rt == 0 && rank == 0 && threadIdx.x == 0);
    const int row0 = rt * ROWS;
    const int rows = min(ROWS, s.n * p.G - row0);
    if (rows <= 0) return;
    const int t0 = row0 / p.G, t1 = (row0 + rows - 1) / p.G;
    const VisibleTiles vis = TREE ? visible_tiles(s.first, s.len - 1, p.window, p.sinks)
                                  : visible_tiles(s.first + t0, s.first + t1, p.window, p.sinks);
    const int32_t *table = p.block_table + (size_t)b * p.max_pages;
    __shared__ int depth[ROWS];               // TREE: depths of the rows
    if (TREE && threadIdx.x < rows) depth[threadIdx.x] = tree_depth(p, tree_row(p, b, (row0 + threadIdx.x) / p.G), s.n);

    for (int x = threadIdx.x; x < ROWS * D / 4; x += W * 32) {
        const int r = x / (D / 4), c = x % (D / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int t = (row0 + r) / p.G, g = (row0 + r) % p.G;
            v = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                 (((size_t)b * p.T + t) * p.Hq + h * p.G + g) * D)[c];
        }
        reinterpret_cast<float4 *>(qs[r])[c] = v;
    }
    __syncthreads();

    const int g4 = lane >> 2, q4 = lane & 3;
    float o[ROWS][VN], m[ROWS], l[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < VN; ++e) o[r][e] = 0.f;
    }
    const float *kpool = static_cast<const float *>(p.k_pool), *vpool = static_cast<const float *>(p.v_pool);
    const int stride = cluster * W;
    int k = rank * W + warp, phys;
    long long base = k < vis.count ? tile_row(p, table, vis.tile(k), h, phys) : -1;
    for (; k < vis.count; k += stride) {
        const int tile = vis.tile(k);
        const long long row = base;
        if (k + stride < vis.count) base = tile_row(p, table, vis.tile(k + stride), h, phys);
        if (row < 0) continue;
        float4 kc[PARTS][KC];
        float vv[PARTS][8][VN];
        auto load = [&](int part, int slot) {          // 8 tokens
            const float *krow = kpool + (size_t)(row + 8 * part + g4) * D + q4 * 4;
#pragma unroll
            for (int j = 0; j < KC; ++j) kc[slot][j] = __ldg(reinterpret_cast<const float4 *>(krow + j * 16));
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float *vrow = vpool + (size_t)(row + 8 * part + t) * D + lane * VN;
                const int j = tile * kTile + 8 * part + t;
                bool any = j <= vis.hi && (j >= vis.lo || j < p.sinks);         // seen by some row
                if (TREE && any && j >= s.first) {
                    any = false;
                    for (int i = t0; i <= t1; ++i)
                        any = any || (__ldg(tree_row(p, b, i) + ((j - s.first) >> 5)) >> ((j - s.first) & 31) & 1u);
                }
                if constexpr (VN == 4) {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(vrow));
                    vv[slot][t][0] = any ? x.x : 0.f; vv[slot][t][1] = any ? x.y : 0.f;
                    vv[slot][t][2] = any ? x.z : 0.f; vv[slot][t][3] = any ? x.w : 0.f;
                } else {
                    const float2 x = __ldg(reinterpret_cast<const float2 *>(vrow));
                    vv[slot][t][0] = any ? x.x : 0.f; vv[slot][t][1] = any ? x.y : 0.f;
                }
            }
        };
        if constexpr (PARTS == 2) { load(0, 0); load(1, 1); }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int tok0 = tile * kTile + 8 * part, slot = PARTS == 2 ? part : 0;
            if constexpr (PARTS == 1) load(part, 0);
            float sc[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    const float4 x = reinterpret_cast<const float4 *>(qs[r])[q4 + 4 * j];
                    a = fmaf(kc[slot][j].x, x.x, a); a = fmaf(kc[slot][j].y, x.y, a);
                    a = fmaf(kc[slot][j].z, x.z, a); a = fmaf(kc[slot][j].w, x.w, a);
                }
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                const int t = (row0 + min(r, rows - 1)) / p.G;
                const bool seen = TREE ? tree_sees(tree_row(p, b, t), s.first + depth[min(r, rows - 1)], tok0 + g4, s.first,
                                                   s.len, p.window, p.sinks)
                                       : sees(s.first + t, tok0 + g4, p.window, p.sinks);
                sc[r] = seen ? a * p.scale_log2 : -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float top = sc[r];
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float m_new = fmaxf(m[r], top);
                const float at = m_new == -INFINITY ? 0.f : m_new;
                const float f = exp2f(m[r] - at);
                m[r] = m_new;
                const float w = exp2f(sc[r] - at);
                l[r] = fmaf(l[r], f, w);            // this lane's token; summed over g4 at the end
#pragma unroll
                for (int e = 0; e < VN; ++e) o[r][e] *= f;
                if (q4 == 0) ps[warp][g4][r] = w;
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float w = ps[warp][t][r];
#pragma unroll
                    for (int e = 0; e < VN; ++e) o[r][e] = fmaf(w, vv[slot][t][e], o[r][e]);
                }
            __syncwarp();
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        float sum = l[r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        float *dst = part_o + ((size_t)warp * ROWS + r) * D + lane * VN;
#pragma unroll
        for (int e = 0; e < VN; ++e) dst[e] = o[r][e];
        if (lane == 0) part_ml[warp * ROWS + r] = make_float2(m[r], sum);
    }
    join_and_write<float, D, ROWS, W>(p, part_o, part_ml, cluster, row0, rows, b, h);
}

// ---------------------------------------------------------------------- launch

template <typename K>
cudaError_t launch_rows(K kernel, const WindowParams &p, long long units, int threads, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * p.cluster));
    cfg.blockDim = dim3(threads);
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

template <typename T, bool FP8, int D, bool TREE>
cudaError_t launch_16(WindowParams p, cudaStream_t stream) {
    const int rows = p.T * p.G;
    if (rows <= 8) {
        p.row_tiles = 1;
        return launch_rows(window_rows_kernel<T, FP8, D, 8, 4, TREE>, p, (long long)p.B * p.Hkv, 128, step_smem<FP8, D, 8, 4>(), stream);
    }
    p.row_tiles = (rows + 15) / 16;
    return launch_rows(window_rows_kernel<T, FP8, D, 16, 4, TREE>, p, (long long)p.B * p.Hkv * p.row_tiles, 128,
                       step_smem<FP8, D, 16, 4>(), stream);
}

template <int D, bool TREE>
cudaError_t launch_f32(WindowParams p, cudaStream_t stream) {
    const int rows = p.T * p.G;
    if (rows == 1) {
        p.row_tiles = 1;
        return launch_rows(window_rows_f32_kernel<D, 1, 4, TREE>, p, (long long)p.B * p.Hkv, 128, rows_smem<D, 1, 4>(), stream);
    }
    p.row_tiles = (rows + 7) / 8;
    return launch_rows(window_rows_f32_kernel<D, 8, 4, TREE>, p, (long long)p.B * p.Hkv * p.row_tiles, 128,
                       rows_smem<D, 8, 4>(), stream);
}

}  // namespace

// Row tiles of the largest sequence, as launch_window_rows cuts them.
int window_row_tiles(qasa_dtype dt, int rows) {
    const int per = dt == QASA_DTYPE_F32 ? (rows == 1 ? 1 : 8) : rows <= 8 ? 8 : 16;
    return (rows + per - 1) / per;
}

namespace {

template <bool TREE>
cudaError_t launch_any(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream) {
    switch (dt) {
    case QASA_DTYPE_F32: return D == 64 ? launch_f32<64, TREE>(p, stream) : launch_f32<128, TREE>(p, stream);
    case QASA_DTYPE_F16:
        return D == 64 ? launch_16<__half, false, 64, TREE>(p, stream) : launch_16<__half, false, 128, TREE>(p, stream);
    case QASA_DTYPE_BF16:
        return D == 64 ? launch_16<__nv_bfloat16, false, 64, TREE>(p, stream)
                       : launch_16<__nv_bfloat16, false, 128, TREE>(p, stream);
    default: return D == 64 ? launch_16<__half, true, 64, TREE>(p, stream) : launch_16<__half, true, 128, TREE>(p, stream);
    }
}

}  // namespace

cudaError_t launch_window_rows(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream) {
    return launch_any<false>(dt, D, p, stream);
}
cudaError_t launch_tree_rows(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream) {
    return launch_any<true>(dt, D, p, stream);
}

}  // namespace qasa
