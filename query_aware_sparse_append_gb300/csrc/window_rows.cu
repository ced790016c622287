// window_rows.cu -- windowed attention for few query rows per KV head: the
// decode step, and the verification of a few drafted tokens.
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
// A warp's tile never passes through shared memory: K and V come by 16-byte loads
// straight into the fragments of m16n8k16 products.  A lane's 16-byte chunk of a
// key row is read as the pairs of k-steps; q's fragments take the same channel
// order, and the sum over channels does not care about it.  Values need pairs of
// tokens per channel: a lane loads the same channels of two neighbouring rows and
// interleaves the halves with byte permutes.  The next tile's keys are under way
// while the softmax runs, the next values while the next scores are computed.
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kMaxCluster = 8;

// Joins the partial states of a unit and writes its rows.  Every warp of the CTA
// has left ROWS rows of o[D] and (m, l) in shared memory: m the running maximum
// in log2 units (-inf where the warp saw nothing), l the sum of weights.
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
            if (ml.x == -INFINITY) continue;
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
                if (k < cluster && ml[k].x != -INFINITY) {
                    const float4 v = ld_cluster_v4(map_rank(part_o + (size_t)r * D + 4 * c, k));
                    const float f = exp2f(ml[k].x - m);
                    l = fmaf(f, ml[k].y, l);
                    o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
                    o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
                }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;   // a row that sees nothing is zero
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

// K and V of a tile, straight from the pool.
template <bool FP8, int D> struct TileRegs {
    static constexpr int KC = FP8 ? D / 64 : D / 32;   // 16-byte chunks of a key row per lane
    static constexpr bool V8 = FP8 && D == 64;         // a lane's share of a value row is 8 bytes
    static constexpr int VC = FP8 ? 1 : D / 64;        // chunks of a value row per lane
};

// T: type of q and out; FP8: pages of E4M3 codes (T is __half).
template <typename T, bool FP8, int D, int ROWS, int W>
__global__ void __launch_bounds__(W * 32) window_rows_kernel(WindowParams p) {
    using R = TileRegs<FP8, D>;
    constexpr bool TWO = ROWS == 16;          // rows 8 .. 15 of the products exist
    constexpr int KS = D / 16;                // k-steps of the scores
    constexpr int NT = D / 8;                 // column tiles of the output
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int VCH = NT / R::VC;           // channels of a value chunk (8 or 16)

    extern __shared__ __align__(16) unsigned char smem[];
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
    const VisibleTiles vis = visible_tiles(s.first + t0, s.first + t1, p.window, p.sinks);

    const int g4 = lane >> 2, q4 = lane & 3;
    // q fragments: rows g4 and g4 + 8, channels in the order of the key chunks
    uint32_t qa[KS][TWO ? 4 : 2];
    int pos[TWO ? 2 : 1];                     // positions of this lane's rows
#pragma unroll
    for (int half = 0; half < (TWO ? 2 : 1); ++half) {
        const int r = g4 + 8 * half;
        const bool live = r < rows;
        const int t = (row0 + (live ? r : 0)) / p.G, g = (row0 + (live ? r : 0)) % p.G;
        pos[half] = s.first + t;
        const T *row = static_cast<const T *>(p.q) + (((size_t)b * p.T + t) * p.Hq + h * p.G + g) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            // 8 channels: four k-step halves.  Key chunks have 8 (16-bit) or 16 (E4M3) channels.
            const int c = FP8 ? (q4 + 4 * (j / 2)) * 16 + 8 * (j & 1) : (q4 + 4 * j) * 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = ld_global_nc_v4(row + c);
            qa[2 * j][half] = w.x;
            qa[2 * j][half + (TWO ? 2 : 1)] = w.y;
            qa[2 * j + 1][half] = w.z;
            qa[2 * j + 1][half + (TWO ? 2 : 1)] = w.w;
        }
    }

    float o[NT][TWO ? 4 : 2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < (TWO ? 4 : 2); ++e) o[n][e] = 0.f;
    float m[TWO ? 2 : 1], l[TWO ? 2 : 1];
#pragma unroll
    for (int x = 0; x < (TWO ? 2 : 1); ++x) { m[x] = -INFINITY; l[x] = 0.f; }
    float vref = 0.f;                         // E4M3: o is in units of the largest V scale so far

    const int32_t *table = p.block_table + (size_t)b * p.max_pages;
    const int stride = cluster * W;
    const int mine = vis.count > rank * W + warp ? (vis.count - (rank * W + warp) + stride - 1) / stride : 0;

    uint4 kr[2][R::KC];                       // key rows g4 and g4 + 8
    uint4 vr[4][R::VC];                       // value rows 2 q4, 2 q4 + 1, + 8 (E4M3, d 64: low halves)
    float ksc = 1.f, vsc = 1.f, ksc_next = 1.f, vsc_next = 1.f;

    // lane x holds the place of this warp's tile (batch + x)
    int batch = 0;
    long long row_x = -1;
    int phys_x = -1;
    auto look_up = [&](int from) {
        batch = from;
        row_x = -1;
        phys_x = -1;
        if (from + lane < mine)
            row_x = tile_row(p, table, vis.tile(rank * W + warp + (from + lane) * stride), h, phys_x);
    };
    const unsigned char *kpool = static_cast<const unsigned char *>(p.k_pool);
    const unsigned char *vpool = static_cast<const unsigned char *>(p.v_pool);
    auto load_k = [&](long long row) {
        if (row < 0) return;
        const unsigned char *base = kpool + (size_t)(row + g4) * D * ES + q4 * 16;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < R::KC; ++j) kr[x][j] = ld_global_nc_v4(base + x * 8 * D * ES + j * 64);
    };
    auto load_v = [&](long long row) {
        if (row < 0) return;
        const unsigned char *base = vpool + (size_t)(row + 2 * q4) * D * ES + g4 * (R::V8 ? 8 : 16);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < R::VC; ++j) {
                const unsigned char *a = base + ((x & 1) + 8 * (x >> 1)) * D * ES + j * 128;
                if constexpr (R::V8) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(a));
                    vr[x][j] = make_uint4(w.x, w.y, 0, 0);
                } else {
                    vr[x][j] = ld_global_nc_v4(a);
                }
            }
    };
    auto scales_of = [&](int phys, float &k, float &v) {
        if constexpr (FP8) {
            if (phys < 0) return;
            const float2 a = __ldg(reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + h) * 4));
            k = fp8_scale(a.x);
            v = fp8_scale(a.y);
        }
    };

    long long row = -1;
    if (mine > 0) {
        look_up(0);
        row = __shfl_sync(0xffffffffu, row_x, 0);
        scales_of(__shfl_sync(0xffffffffu, phys_x, 0), ksc, vsc);
        load_k(row);
        load_v(row);
    }
    for (int i = 0; i < mine; ++i) {
        // where the next tile is
        long long next = -1;
        if (i + 1 < mine) {
            if (i + 1 - batch == 32) look_up(i + 1);
            next = __shfl_sync(0xffffffffu, row_x, i + 1 - batch);
            scales_of(__shfl_sync(0xffffffffu, phys_x, i + 1 - batch), ksc_next, vsc_next);
        }
        const int tok0 = vis.tile(rank * W + warp + i * stride) * kTile;
        float sc[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[x][e] = 0.f;
        if (row >= 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    uint4 w;
                    if constexpr (FP8) {
                        const uint4 c = kr[x][j / 2];
                        w = (j & 1) ? make_uint4(e4m3x2_to_h2(c.z), e4m3x2_to_h2(c.z >> 16), e4m3x2_to_h2(c.w),
                                                 e4m3x2_to_h2(c.w >> 16))
                                    : make_uint4(e4m3x2_to_h2(c.x), e4m3x2_to_h2(c.x >> 16), e4m3x2_to_h2(c.y),
                                                 e4m3x2_to_h2(c.y >> 16));
                    } else {
                        w = kr[x][j];
                    }
                    uint32_t a[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[0] = qa[2 * j + k][0];
                        a[1] = TWO ? qa[2 * j + k][1] : 0u;
                        a[2] = qa[2 * j + k][TWO ? 2 : 1];
                        a[3] = TWO ? qa[2 * j + k][TWO ? 3 : 1] : 0u;
                        mma16816<T>::run(sc[x], a, k ? w.z : w.x, k ? w.w : w.y);
                    }
                }
        }
        load_k(next);

        if (row >= 0) {
            const float to_log2 = p.scale_log2 * ksc;
            // whole tile visible to every row of the unit?
            const bool inside = tok0 + kTile - 1 <= s.first + t0 &&
                                (tok0 + kTile <= p.sinks || tok0 > s.first + t1 - p.window);
            uint32_t pa[4] = {0u, 0u, 0u, 0u};
            float f[TWO ? 2 : 1];
            float vscale = 1.f;
            if constexpr (FP8) {
                if (vsc > vref) {
                    const float g = vref / vsc;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < (TWO ? 4 : 2); ++e) o[n][e] *= g;
                    vref = vsc;
                }
                vscale = vref > 0.f ? vsc / vref : 0.f;
            }
#pragma unroll
            for (int half = 0; half < (TWO ? 2 : 1); ++half) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = sc[e >> 1][2 * half + (e & 1)] * to_log2;
                    if (!inside && !sees(pos[half], tok0 + 8 * (e >> 1) + 2 * q4 + (e & 1), p.window, p.sinks))
                        v[e] = -INFINITY;
                }
                float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float m_new = fmaxf(m[half], top);
                const float base = m_new == -INFINITY ? 0.f : m_new;   // nothing seen yet: every weight is 0
                f[half] = exp2_fast(m[half] - base);
                m[half] = m_new;
                float w[4], sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) { w[e] = exp2_fast(v[e] - base); sum += w[e]; }
                l[half] = fmaf(l[half], f[half], sum);
                // weights in the values' 16-bit type: half a step each, while the sum keeps fp32
                pa[half] = mma16816<T>::pack2(w[0] * vscale, w[1] * vscale);
                pa[half + 2] = mma16816<T>::pack2(w[2] * vscale, w[3] * vscale);
            }
            bool same = f[0] == 1.f;
            if constexpr (TWO) same = same && f[1] == 1.f;
            if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= f[0];
                    o[n][1] *= f[0];
                    if constexpr (TWO) { o[n][2] *= f[1]; o[n][3] *= f[1]; }
                }
            }
            if (!inside) {   // values that no row sees may be anything: 0 * NaN is not 0
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = tok0 + 2 * q4 + (x & 1) + 8 * (x >> 1);
                    if (j > vis.hi || (j < vis.lo && j >= p.sinks))
#pragma unroll
                        for (int c = 0; c < R::VC; ++c) vr[x][c] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int c = 0; c < R::VC; ++c)
#pragma unroll
                for (int k = 0; k < VCH / 2; ++k) {
                    uint32_t r0, r1, r2, r3;
                    if constexpr (FP8) {
                        auto pick = [&](const uint4 &w) {
                            const uint32_t word = k / 2 == 0 ? w.x : k / 2 == 1 ? w.y : k / 2 == 2 ? w.z : w.w;
                            return e4m3x2_to_h2(k & 1 ? word >> 16 : word);
                        };
                        r0 = pick(vr[0][c]); r1 = pick(vr[1][c]); r2 = pick(vr[2][c]); r3 = pick(vr[3][c]);
                    } else {
                        auto pick = [&](const uint4 &w) { return k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w; };
                        r0 = pick(vr[0][c]); r1 = pick(vr[1][c]); r2 = pick(vr[2][c]); r3 = pick(vr[3][c]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t sel = e ? 0x7632u : 0x5410u;
                        float *acc = o[c * VCH + 2 * k + e];
                        float d[4] = {acc[0], acc[1], TWO ? acc[TWO ? 2 : 0] : 0.f, TWO ? acc[TWO ? 3 : 0] : 0.f};
                        mma16816<T>::run(d, pa, __byte_perm(r0, r1, sel), __byte_perm(r2, r3, sel));
                        acc[0] = d[0];
                        acc[1] = d[1];
                        if constexpr (TWO) { acc[2] = d[2]; acc[3] = d[3]; }
                    }
                }
        }
        load_v(next);
        row = next;
        ksc = ksc_next;
        vsc = vsc_next;
    }

    // this warp's state: column tile c * VCH + idx, columns 2 q4 and 2 q4 + 1, is
    // channel c * 8 VCH + VCH * column + idx
#pragma unroll
    for (int half = 0; half < (TWO ? 2 : 1); ++half) {
        float sum = l[half];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = g4 + 8 * half;
        float *dst = part_o + ((size_t)warp * ROWS + r) * D;
        const float unitv = FP8 ? vref : 1.f;
#pragma unroll
        for (int c = 0; c < R::VC; ++c)
#pragma unroll
            for (int col = 0; col < 2; ++col)
#pragma unroll
                for (int k = 0; k < VCH; k += 4)
                    *reinterpret_cast<float4 *>(dst + c * 8 * VCH + VCH * (2 * q4 + col) + k) =
                        make_float4(o[c * VCH + k][2 * half + col] * unitv, o[c * VCH + k + 1][2 * half + col] * unitv,
                                    o[c * VCH + k + 2][2 * half + col] * unitv,
                                    o[c * VCH + k + 3][2 * half + col] * unitv);
        if (q4 == 0) part_ml[warp * ROWS + r] = make_float2(m[half], sum);
    }
    join_and_write<T, D, ROWS, W>(p, part_o, part_ml, cluster, row0, rows, b, h);
}

// ------------------------------------------------------------------ fp32 pages

// The same split with fused multiply-adds: fp32 products have no tensor path that
// keeps their precision.  Four lanes share a key row (8 rows under way per warp);
// the ROWS scores of a row are summed over the four by a butterfly that leaves
// each lane ROWS / 4 of them (all of them for ROWS < 4); the values are read a
// whole row at a time, a lane owning D / 32 channels.
template <int D, int ROWS, int W>
__global__ void __launch_bounds__(W * 32) window_rows_f32_kernel(WindowParams p) {
    constexpr int KC = D / 16;                 // float4 chunks of a key row per lane
    constexpr int VN = D / 32;                 // channels per lane
    extern __shared__ __align__(16) unsigned char smem[];
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
    const VisibleTiles vis = visible_tiles(s.first + t0, s.first + t1, p.window, p.sinks);

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
    const int32_t *table = p.block_table + (size_t)b * p.max_pages;
    const float *kpool = static_cast<const float *>(p.k_pool), *vpool = static_cast<const float *>(p.v_pool);
    const int stride = cluster * W;
    for (int k = rank * W + warp; k < vis.count; k += stride) {
        const int tile = vis.tile(k);
        int phys;
        const long long base = tile_row(p, table, tile, h, phys);
        if (base < 0) continue;
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int tok0 = tile * kTile + 8 * part;
            const float *krow = kpool + (size_t)(base + 8 * part + g4) * D + q4 * 4;
            float4 kc[KC];
#pragma unroll
            for (int j = 0; j < KC; ++j) kc[j] = __ldg(reinterpret_cast<const float4 *>(krow + j * 16));
            float vv[8][VN];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float *vrow = vpool + (size_t)(base + 8 * part + t) * D + lane * VN;
                const int j = tok0 + t;
                const bool any = j <= vis.hi && (j >= vis.lo || j < p.sinks);   // seen by some row
                if constexpr (VN == 4) {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(vrow));
                    vv[t][0] = any ? x.x : 0.f; vv[t][1] = any ? x.y : 0.f;
                    vv[t][2] = any ? x.z : 0.f; vv[t][3] = any ? x.w : 0.f;
                } else {
                    const float2 x = __ldg(reinterpret_cast<const float2 *>(vrow));
                    vv[t][0] = any ? x.x : 0.f; vv[t][1] = any ? x.y : 0.f;
                }
            }
            float sc[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    const float4 x = reinterpret_cast<const float4 *>(qs[r])[q4 + 4 * j];
                    a = fmaf(kc[j].x, x.x, a); a = fmaf(kc[j].y, x.y, a);
                    a = fmaf(kc[j].z, x.z, a); a = fmaf(kc[j].w, x.w, a);
                }
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                const int t = (row0 + min(r, rows - 1)) / p.G;
                sc[r] = sees(s.first + t, tok0 + g4, p.window, p.sinks) ? a * p.scale_log2 : -INFINITY;
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
                    for (int e = 0; e < VN; ++e) o[r][e] = fmaf(w, vv[t][e], o[r][e]);
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
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, bool FP8, int D>
cudaError_t launch_16(WindowParams p, cudaStream_t stream) {
    const int rows = p.T * p.G;
    if (rows <= 8) {
        p.row_tiles = 1;
        return launch_rows(window_rows_kernel<T, FP8, D, 8, 4>, p, (long long)p.B * p.Hkv, 128, rows_smem<D, 8, 4>(), stream);
    }
    p.row_tiles = (rows + 15) / 16;
    return launch_rows(window_rows_kernel<T, FP8, D, 16, 4>, p, (long long)p.B * p.Hkv * p.row_tiles, 128,
                       rows_smem<D, 16, 4>(), stream);
}

template <int D>
cudaError_t launch_f32(WindowParams p, cudaStream_t stream) {
    const int rows = p.T * p.G;
    if (rows == 1) {
        p.row_tiles = 1;
        return launch_rows(window_rows_f32_kernel<D, 1, 4>, p, (long long)p.B * p.Hkv, 128, rows_smem<D, 1, 4>(), stream);
    }
    p.row_tiles = (rows + 7) / 8;
    return launch_rows(window_rows_f32_kernel<D, 8, 4>, p, (long long)p.B * p.Hkv * p.row_tiles, 128,
                       rows_smem<D, 8, 4>(), stream);
}

}  // namespace

// Row tiles of the largest sequence, as launch_window_rows cuts them.
int window_row_tiles(qasa_dtype dt, int rows) {
    const int per = dt == QASA_DTYPE_F32 ? (rows == 1 ? 1 : 8) : rows <= 8 ? 8 : 16;
    return (rows + per - 1) / per;
}

cudaError_t launch_window_rows(qasa_dtype dt, int D, const WindowParams &p, cudaStream_t stream) {
    switch (dt) {
    case QASA_DTYPE_F32: return D == 64 ? launch_f32<64>(p, stream) : launch_f32<128>(p, stream);
    case QASA_DTYPE_F16:
        return D == 64 ? launch_16<__half, false, 64>(p, stream) : launch_16<__half, false, 128>(p, stream);
    case QASA_DTYPE_BF16:
        return D == 64 ? launch_16<__nv_bfloat16, false, 64>(p, stream) : launch_16<__nv_bfloat16, false, 128>(p, stream);
    default: return D == 64 ? launch_16<__half, true, 64>(p, stream) : launch_16<__half, true, 128>(p, stream);
    }
}

}  // namespace qasa
