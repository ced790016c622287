// tree.cu -- attention of a tree of drafted tokens over the paged cache, on the
// fifth-generation tensor cores.
//
//   S = Q K^T,  P = exp2(scale S - m) over the tokens that the row sees,  O += P V,  out = O / sum P
//
// What bounds it: some tens of drafted tokens of a few query heads meet a long context,
// whose keys and values are read once.  Up to about 128 rows (tokens x heads of the group)
// per KV head that is HBM; with 256 rows the exponentials and the products take as long.
// With few sequences it is the number of SMs that the keys are spread over.
//
// Split: a unit is a block of rows of a (sequence, KV head); its key tiles are 128 tokens
// of its visible pages.  All units' tiles lie on one line, each unit with kUnitCost tiles
// more for its beginning and end, and every CTA, one per SM, takes an equal stretch:
// ragged lengths and any number of sequences fill the device alike.  A unit cut by a
// border of stretches leaves partial outputs in the workspace, which a second kernel,
// started beside the first one's end, joins in the order of the stretches: nothing
// depends on which CTA is faster.  A call of few tiles per unit takes whole units.
//
// Rows: as in the prompt kernel a row tile packs 128 (token, head) rows.  WIDE: a CTA has
// two row tiles and both go through every key tile.  Else a unit has one row tile, and
// two softmax groups take turns at the key tiles, each with its own scores, weights and
// output in tensor memory: the chain S -> softmax -> O of one overlaps that of the other
// whether there are rows for both or not.  The two outputs of a row lie in the same lane
// of tensor memory, so a thread of either group adds them up, half of the channels each.
//
// Warps: 0-7 two softmax groups, a thread a row; then one that issues the products, one
// that brings pages (TMA), one that watches over tiles: it zeroes hidden value rows and
// waits for tiles in the issuing thread's place; one that walks the CTA's stretch and tells
// the others its segments, some ahead; E4M3: four that turn codes into halves.  The ring of
// key and value tiles runs on from one unit to the next, so the first tiles of a unit
// arrive under the last ones of the unit before.
//
// E4M3 pages come as codes and become halves, which they are exactly, on the way into the
// ring.  The keys' scale multiplies the scores, the values' the weights: as a share of
// the largest value scale so far, under which the output is kept.
#include "tcgen05.cuh"
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kRows = 128;            // rows of a row tile
constexpr int kKeys = 128;            // tokens of a key tile
constexpr int kUnitCost = 2;          // tiles that a unit's beginning and end are worth
constexpr int kScaleRing = 8;         // key tiles whose E4M3 scales are kept
constexpr int kSegments = 4;          // segments told ahead
constexpr float kGivenUp = 3e38f;     // maximum that a CTA reports for rows that it gave up
constexpr int kJoinThreads = 128, kJoinBlocks = 32;

template <bool FP8> constexpr int tree_threads() { return FP8 ? 512 : 384; }
template <int D> constexpr int kv_bytes() { return kKeys * D * 2; }
// Key and value tiles as halves, and as codes, under way.  128 channels: what fits.
template <int D, bool FP8, bool WIDE> constexpr int kStages = D == 64 ? 8 : FP8 ? (WIDE ? 3 : 4) : 5;
template <int D, bool FP8, bool WIDE> constexpr int kCodeStages = !FP8 ? 0 : D == 64 ? 6 : WIDE ? 4 : 3;
template <int D, bool FP8, bool WIDE> constexpr size_t tree_smem() {
    return 1024 + (size_t)(WIDE ? 2 : 1) * kRows * D * 2 + (size_t)kStages<D, FP8, WIDE> * kv_bytes<D>() +
           (size_t)kCodeStages<D, FP8, WIDE> * kKeys * D + (WIDE ? 0 : 2 * 2 * kRows * sizeof(float2));
}

// Pages that the queries of a sequence see: pages 0 .. head of the sinks, then pages body0 ..
struct Pages {
    int lo, hi, head, body0, count;
    __device__ __forceinline__ int page(int k) const { return k < head ? k : body0 + k - head; }
};

__device__ __forceinline__ Pages visible_pages(const WindowParams &p, const QuerySpan &s) {
    Pages v;
    v.hi = s.len - 1;
    v.lo = s.first - p.window + 1 > 0 ? s.first - p.window + 1 : 0;    // of a query at depth 0
    v.body0 = v.lo / p.P;
    v.head = min((min(p.sinks, v.lo) + p.P - 1) / p.P, v.body0);
    v.count = s.len <= 0 ? 0 : v.head + v.hi / p.P - v.body0 + 1;
    return v;
}

// Part of a unit: key tiles t0 .. t1 of all of them, for the rows of tokens tok0 ..
struct Segment {
    int b, h, tok0, t0, t1, tiles;       // b < 0: no more
    int last_cta;                        // that has a piece of the unit
    int whole0, whole1;                  // key tiles that every row sees as a whole
    QuerySpan s;
    Pages pages;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

struct TreeShared {
    uint64_t q_full, q_empty, kv_full[8], kv_empty[8], code_full[6], code_empty[6];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free, joined, drained;
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    uint32_t tmem;
    int any_bad;         // some page of this CTA has a bad block-table entry
    int failed;          // a bounded wait gave up: the rows that waited are not written
    int armed[8];        // copies into each stage (E4M3: of codes) so far
    int q_armed;
    int seq0;            // the stretch begins in this sequence,
    long long at0;       // whose first unit lies here on the line
    long long total;
    long long sums[16];
    float ks[kScaleRing][kKeys / 16], vamax[kScaleRing][kKeys / 16];
    float unit[2][2];    // E4M3: unit of each group's output
};

// CTAs that share a line of `total` places (none of their stretches is empty), and where
// the stretch of CTA c begins.
__device__ __forceinline__ int sharers(long long total) { return total < gridDim.x ? (int)total : (int)gridDim.x; }
__device__ __forceinline__ long long stretch(long long total, int c) {
    const int C = sharers(total);
    return c < C ? total * c / C : total;
}

// Walks the units that a CTA's stretch [v0, v1) of the line touches.  Of the unit at u0
// the stretch has the tiles that lie in it, the first kUnitCost places being the unit's
// beginning; `p.whole_units`: it has the whole unit if it begins in the stretch.
struct Walk {
    const TreeParams &p;
    long long v0, v1, u0, total;
    int b, unit, units, tok_per;
    QuerySpan s;
    Pages pages;
    int tiles;
    __device__ __forceinline__ Walk(const TreeParams &p, int first, long long at, long long total, int tok_per)
        : p(p), v0(stretch(total, blockIdx.x)), v1(stretch(total, blockIdx.x + 1)), u0(at), total(total),
          b(first), unit(0), units(0), tok_per(tok_per) {
        if (b < p.w.B) sequence();
    }
    __device__ __forceinline__ void sequence() {
        s = query_span(p.w, b, false);
        pages = visible_pages(p.w, s);
        tiles = (pages.count * p.w.P + kKeys - 1) / kKeys;
        units = p.w.Hkv * ((s.n + tok_per - 1) / tok_per);
        unit = 0;
        // units that end before the stretch
        if (units > 0 && v0 > u0) {
            const long long skip = (v0 - u0) / (tiles + kUnitCost);
            unit = (int)(skip < units ? skip : units);
            u0 += (long long)unit * (tiles + kUnitCost);
        }
    }
    __device__ __forceinline__ bool next(Segment &g) {
        while (b < p.w.B && u0 < v1) {
            if (unit == units) {
                if (++b < p.w.B) sequence();
                continue;
            }
            const int blocks = units / p.w.Hkv;
            const long long lo = v0 - u0 - kUnitCost, hi = v1 - u0 - kUnitCost;
            g.t0 = v0 <= u0 || lo < 0 ? 0 : (int)lo;
            g.t1 = hi < tiles ? (int)(hi > 0 ? hi : 0) : tiles;
            if (p.whole_units) {
                g.t0 = 0;
                g.t1 = u0 >= v0 ? tiles : 0;
            }
            g.b = b;
            g.h = unit / blocks;
            g.tok0 = unit % blocks * tok_per;
            g.tiles = tiles;
            g.s = s;
            g.pages = pages;
            const bool take = g.t1 > g.t0 || (tiles == 0 && u0 >= v0);
            u0 += tiles + kUnitCost;
            ++unit;
            if (!take) continue;
            // the last stretch that begins before the unit's end
            g.last_cta = (int)((u0 * sharers(total) - 1) / total);
            // full tiles of context pages wholly inside the deepest row's window
            const int ppt = kKeys / p.w.P, ctx = s.first;
            g.whole0 = g.whole1 = 0;
            if (ctx > 0) {
                const int clear = max(s.len - 1 - p.w.window + p.w.P, 0) / p.w.P;
                g.whole0 = (pages.head + max(clear - pages.body0, 0) + ppt - 1) / ppt;
                if (pages.head > 0) g.whole0 = max(g.whole0, (pages.head + ppt - 1) / ppt);
                g.whole1 = (pages.head + max(ctx / p.w.P - pages.body0, 0)) / ppt;
            }
            return true;
        }
        return false;
    }
};

__device__ __forceinline__ bool good_page(const WindowParams &p, const int32_t *table, int page) {
    const int phys = table[page];
    return phys >= 0 && phys < p.num_phys;
}

// Bit c: token base + c is at or before x.
__device__ __forceinline__ uint32_t upto16(int x, int base) {
    const int n = x - base;
    return n < 0 ? 0u : n >= 15 ? 0xffffu : (2u << n) - 1u;
}
// Bits `at` .. at + 15 of a mask row of `words` words (at > -16; those that it has not are 0).
__device__ __forceinline__ uint32_t mask16(const uint32_t *row, int words, int at) {
    if (at < 0) return __ldg(row) << -at & 0xffffu;
    const int w = at >> 5;
    const uint32_t lo = w < words ? __ldg(row + w) : 0u, hi = w + 1 < words ? __ldg(row + w + 1) : 0u;
    return __funnelshift_r(lo, hi, at & 31) & 0xffffu;
}

// Two fp32 operations in one instruction; register pairs hold neighbouring columns.
__device__ __forceinline__ float2 fma2(uint32_t x, uint32_t y, float scale, float add) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "r"(x), "r"(y), "f"(scale), "f"(add));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}" : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// Place of the partial output of a CTA: the first piece of a unit, or a later one.
__device__ __forceinline__ int slot_of(int cta, bool first) { return 2 * cta + (first ? 1 : 0); }

// Whether the tile may have value rows that no row of the unit sees.
__device__ __forceinline__ bool hidden_rows(const WindowParams &p, TreeShared &sh, const Segment &g, int tile) {
    const int ppt = kKeys / p.P, k0 = tile * ppt, k1 = k0 + ppt;
    return *(volatile int *)&sh.any_bad != 0 || k1 >= g.pages.count || g.pages.page(k1 - 1) * p.P + p.P > g.s.first ||
           (g.pages.lo > 0 && k0 <= g.pages.head && k1 >= g.pages.head);
}
// Whether some row of the unit may see row r of the tile.
__device__ __forceinline__ bool row_seen(const WindowParams &p, TreeShared &sh, const Segment &g, int tile, int r, int tok_per) {
    const int k = tile * (kKeys / p.P) + r / p.P, pg = g.pages.page(k), at = pg * p.P + r % p.P;
    if (k >= g.pages.count || at > g.pages.hi || (at < g.pages.lo && at >= p.sinks)) return false;
    if (*(volatile int *)&sh.any_bad && !good_page(p, p.block_table + (size_t)g.b * p.max_pages, pg)) return false;
    const int j = at - g.s.first;
    if (j < 0) return true;
    const int end = min(g.s.n, g.tok0 + tok_per);
    for (int t = g.tok0; t < end; ++t)
        if (__ldg(tree_row(p, g.b, t) + (j >> 5)) >> (j & 31) & 1u) return true;
    return false;
}

// T: 16-bit type of q and out (and of the pages); FP8: pages of E4M3 codes.
template <typename T, bool FP8, int D, bool WIDE>
__global__ void __launch_bounds__(tree_threads<FP8>(), 1)
tree_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ CUtensorMap vmap, TreeParams tp) {
    constexpr int NB = D / 64;                        // 64-channel blocks
    constexpr int BLOCK = kRows * 128;                // bytes of one block of a tile
    constexpr int NS = kStages<D, FP8, WIDE>, NC = kCodeStages<D, FP8, WIDE>;
    constexpr int NQ = WIDE ? 2 : 1;                  // row tiles of a unit
    constexpr int LEAD = WIDE ? 1 : 2;                // key tiles ahead of the value tiles in the ring
    constexpr int ROWS = NQ * kRows;
    constexpr int THREADS = tree_threads<FP8>();
    constexpr uint32_t S_COL[2] = {0, 128}, O_COL[2] = {256, 256 + D}, TMEM = 512;
    constexpr int MMA = 8, LOAD = 9, KEEP = 10, PLAN = 11, CONVERT = 12;      // warps
    const WindowParams &p = tp.w;

    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);   // the swizzle counts from 1 KB boundaries
    unsigned char *qtile = smem, *ring = smem + NQ * NB * BLOCK, *codes = ring + NS * kv_bytes<D>();
    float2 *states = reinterpret_cast<float2 *>(codes + NC * kKeys * D);    // two rounds of [group][row]
    __shared__ TreeShared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = kRows / p.G, tok_per = NQ * per;  // tokens of a row tile, of a unit
    const int cta = blockIdx.x;

    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.kv_full[i], FP8 ? 128 : 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < NC; ++i) {
            mbar_init(&sh.code_full[i], 1);
            mbar_init(&sh.code_empty[i], 128);
        }
        for (int i = 0; i < 8; ++i) sh.armed[i] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], kRows + 1);
            mbar_init(&sh.pv_done[i], 1);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], FP8 ? 15 : 11);           // a warp each, but this one's
        }
        mbar_init(&sh.o_free, 2 * kRows);
        mbar_init(&sh.joined, 2 * kRows);
        mbar_init(&sh.drained, 1);
        sh.any_bad = sh.failed = sh.q_armed = 0;
        sh.seq0 = p.B;
        fence_barrier_init();
        if (tp.cuts) tp.cuts[cta] = make_int4(-1, 0, 0, 0);
    }
    if (warp == MMA) tmem_alloc(&sh.tmem, TMEM);

    // The length of the line, and the sequence in which this CTA's stretch begins: a
    // thread adds up a run of sequences, the warps' sums are added in order.
    {
        const int run = (p.B + THREADS - 1) / THREADS, b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
        auto cost = [&](int b, bool report) {
            const QuerySpan s = query_span(p, b, report);
            const Pages v = visible_pages(p, s);
            return (long long)p.Hkv * ((s.n + tok_per - 1) / tok_per) * ((v.count * p.P + kKeys - 1) / kKeys + kUnitCost);
        };
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += cost(b, cta == 0);
        long long before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) sh.sums[warp] = before;
        before -= mine;
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w == warp) before += total;
            total += sh.sums[w];
        }
        if (tid == 0) sh.total = total;
        const long long v0 = stretch(total, cta);
        if (v0 >= before && v0 < before + mine)
            for (int b = b0; b < b1; ++b) {
                const long long c = cost(b, false);
                if (v0 < before + c) {
                    sh.seq0 = b;
                    sh.at0 = before;
                    break;
                }
                before += c;
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    auto give_up = [&] {
        *(volatile int *)&sh.failed = 1;
        if (p.status) atomicOr(p.status, QASA_DEVERR_TIMEOUT);
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {            // a whole warp, which goes on or gives up together
        if (__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_limit_ns))) return true;
        give_up();
        return false;
    };
    // the ring's items of a segment of n tiles: K0 [K1] V0 K .. V, keys LEAD tiles ahead
    auto k_item = [](int j) { return j + max(j - LEAD + 1, 0); };
    auto v_item = [](int j, int n) { return j + min(j + LEAD, n); };
    // row tiles of a segment that have rows
    auto row_tiles = [&](const Segment &g) { return NQ == 2 && g.tok0 + per < g.s.n ? 2 : 1; };

    // registers go to the softmax warps, within what the block was launched with:
    // 256 x 208 + 128 x 88 = 384 x 168, 256 x 184 + 256 x 72 = 512 x 128
    if (warp < MMA) {
        if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    } else {
        if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }

    bool ok = true;
    // segment number k of the stretch, for a whole warp; false after the last one
    auto begin = [&](uint32_t k) {
        ok = ok && wait(&sh.seg_full[k % kSegments], k / kSegments & 1);
        return ok && sh.seg[k % kSegments].b >= 0;
    };
    auto end = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[k % kSegments]);
    };
    if (warp < MMA) {
        // ------------------------------------------------------------ softmax
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // tensor memory lane of this warp, bits 16 up
        const uint32_t sa = tmem + lanes + S_COL[i], oa = tmem + lanes + O_COL[i];
        uint32_t done = 0, tile_base = 0;                         // tiles of this group, of the CTA so far
        for (uint32_t seg = 0; begin(seg); ++seg) {
            const Segment &g = sh.seg[seg % kSegments];
            const int n = g.t1 - g.t0, ppt = kKeys / p.P;
            const int tok = g.tok0 + (WIDE ? i * per : 0) + row / p.G, head = g.h * p.G + row % p.G;
            const bool live = row < per * p.G && tok < g.s.n;
            const bool busy = __any_sync(0xffffffffu, live);      // a warp without rows only keeps pace
            const int32_t *table = p.block_table + (size_t)g.b * p.max_pages;
            const uint32_t *mask = tree_row(p, g.b, live ? tok : 0);
            const int pos = g.s.first + (live ? tree_depth(p, mask, g.s.n) : 0);
            const int mine = WIDE ? (i < row_tiles(g) ? n : 0) : (n + 1 - i) / 2;
            float m = live ? -INFINITY : 0.f, l = 0.f;
            float vref = 0.f, inv_vref = 0.f;                     // E4M3: O is in units of the largest V amax so far
            bool unset = true;                                    // a row of the warp has seen nothing yet
            for (int k = 0; ok && k < mine; ++k) {
                const int j = WIDE ? k : 2 * k + i, tile = g.t0 + j;
                if (!wait(&sh.s_full[i], done & 1)) { ok = false; break; }
                ++done;
                tc_fence_after();
                if (busy) {
                    const uint32_t scales_at = (tile_base + j) % kScaleRing;
                    uint32_t x[kKeys];
                    bool raise = unset, raised = false;
                    const bool bad = *(volatile int *)&sh.any_bad != 0;
                    const bool masked = bad || tile < g.whole0 || tile >= g.whole1;
                    auto scale_o = [&](float f) {                 // the last product into O is complete: S of this tile follows it
                        if (k == 0) return;
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(oa + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(oa + c, o);
                        }
                        tmem_wait_st();
                    };
                    if constexpr (FP8) {
                        float top = 0.f;
#pragma unroll
                        for (int q = 0; q < kKeys / 16; ++q) top = fmaxf(top, sh.vamax[scales_at][q]);
                        if (top > vref) {
                            scale_o(vref / top);
                            vref = top;
                            inv_vref = 1.f / top;
                        }
                    }
                    while (true) {
#pragma unroll
                        for (int c = 0; c < kKeys; c += 32) tmem_ld32(sa + c, x + c);
                        tmem_wait_ld();
                        if (masked) {
                            const int ctx = g.s.first, last = g.s.len - 1;
#pragma unroll
                            for (int q = 0; q < kKeys / 16; ++q) {
                                const int e = tile * ppt + q * 16 / p.P, pg = g.pages.page(e);
                                const int base = pg * p.P + q * 16 % p.P;
                                uint32_t seen = 0;
                                if (e < g.pages.count && (!bad || good_page(p, table, pg))) {
                                    seen = upto16(ctx - 1, base) & (upto16(p.sinks - 1, base) | ~upto16(pos - p.window, base));
                                    if (base + 15 >= ctx)
                                        seen |= mask16(mask, p.mask_words, base - ctx) & upto16(last, base);
                                }
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    if (!(seen >> c & 1u)) x[q * 16 + c] = __float_as_uint(-INFINITY);
                            }
                        }
                        if (raise) {
                            float top = -INFINITY;
#pragma unroll
                            for (int q = 0; q < kKeys / 16; ++q) {
                                float t[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    t[e] = fmaxf(fmaxf(__uint_as_float(x[q * 16 + e]), __uint_as_float(x[q * 16 + 4 + e])),
                                                 fmaxf(__uint_as_float(x[q * 16 + 8 + e]), __uint_as_float(x[q * 16 + 12 + e])));
                                top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * (FP8 ? sh.ks[scales_at][q] : 1.f));
                            }
                            const float m_new = fmaxf(m, top * p.scale_log2 - kHeadroom<T>);
                            const float f = m_new == -INFINITY ? 1.f : exp2_fast(m - m_new);
                            m = m_new;
                            l *= f;
                            scale_o(f);
                            unset = __any_sync(0xffffffffu, m == -INFINITY);
                            raised = true;
                        }
                        const float base = m == -INFINITY ? 0.f : m;
                        float2 sum[4] = {};
#pragma unroll
                        for (int q = 0; q < kKeys / 16; ++q) {
                            float vs = 1.f, scale = p.scale_log2;
                            if constexpr (FP8) {
                                vs = sh.vamax[scales_at][q] * inv_vref;
                                scale *= sh.ks[scales_at][q];
                            }
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                const int e = q * 16 + c;
                                float2 w = fma2(x[e], x[e + 1], scale, -base);
                                w.x = exp2_fast(w.x);
                                w.y = exp2_fast(w.y);
                                sum[c / 2 & 3] = add2(sum[c / 2 & 3], w);
                                // weights in the values' 16-bit type: half a step each, while the sum keeps fp32
                                x[e / 2] = FP8 ? mma16816<T>::pack2(w.x * vs, w.y * vs) : mma16816<T>::pack2(w.x, w.y);
                            }
                        }
                        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                        const float add = sum[0].x + sum[0].y;
                        if (raised || !__any_sync(0xffffffffu, live && !(add <= kMostWeight))) {
                            l += add;
                            break;
                        }
                        raise = true;
                    }
#pragma unroll
                    for (int c = 0; c < kKeys / 2; c += 32) tmem_st32(sa + c, x + c);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&sh.p_full[i]);
            }
            if (ok && mine > 0) {
                ok = wait(&sh.pv_done[i], (done - 1) & 1);
                tc_fence_after();
            }
            tile_base += n;
            if (!ok) break;

            // ---------------------------------------------------------- output
            // WIDE: a thread has its row to itself; else the two groups have a part of the
            // same row each, and a thread of either takes half of the channels.
            if (mine == 0) l = 0.f;
            float f0 = FP8 ? fp8_scale(vref) : 1.f, f1 = 0.f;     // factors of this group's output and of the other's
            if constexpr (!WIDE) {
                float2 *now = states + (seg & 1) * 2 * kRows;
                now[i * kRows + row] = make_float2(m, l);
                if (FP8 && row == 0) sh.unit[seg & 1][i] = f0;       // a warp without rows does not follow it
                tc_fence_before();
                mbar_arrive(&sh.joined);
                ok = wait(&sh.joined, seg & 1);
                if (!ok) break;
                tc_fence_after();
                const float2 other = now[(1 - i) * kRows + row];
                if constexpr (FP8) f1 = sh.unit[seg & 1][1 - i]; else f1 = 1.f;
                const float top = fmaxf(l != 0.f ? m : -INFINITY, other.y != 0.f ? other.x : -INFINITY);
                const float a = l != 0.f ? exp2_fast(m - top) : 0.f, c = other.y != 0.f ? exp2_fast(other.x - top) : 0.f;
                // the same order of the two for both halves of the row
                l = i == 0 ? a * l + c * other.y : c * other.y + a * l;
                m = top;
                f0 *= a;
                f1 *= c;
            }
            const bool whole = g.whole();
            const float inv = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;     // a row that sees nothing is zero; a NaN query's sum is NaN
            f0 *= inv;
            f1 *= inv;
            const int slot = slot_of(cta, g.t0 == 0);
            constexpr int COLS = WIDE ? D : D / 2;
            const int c0 = WIDE ? 0 : i * COLS;
            if (!WIDE || i < row_tiles(g)) {
                T *dst = static_cast<T *>(p.out) + (((size_t)g.b * p.T + tok) * p.Hq + head) * D + c0;
                float4 *part = tp.part_o + ((size_t)slot * (D / 4) + c0 / 4) * ROWS + (WIDE ? i * kRows : 0) + row;
#pragma unroll 1
                for (int c = 0; c < COLS; c += 16) {
                    uint32_t o[16], u[16];
                    if (mine > 0) tmem_ld16(oa + c0 + c, o);
                    if (!WIDE && n > 1 - i) tmem_ld16(tmem + lanes + O_COL[1 - i] + c0 + c, u);
                    tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {                // 0 of something that was never written is not 0
                        v[e] = f0 != 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
                        if (!WIDE) v[e] += f1 != 0.f ? __uint_as_float(u[e]) * f1 : 0.f;
                    }
                    if (whole) {
                        if (live)
#pragma unroll
                            for (int e = 0; e < 16; e += 8) *reinterpret_cast<uint4 *>(dst + c + e) = chunk16<T>::pack(v + e);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            part[(size_t)(c + e) / 4 * ROWS] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
                if (!whole && (WIDE || i == 0)) tp.part_ml[(size_t)slot * ROWS + (WIDE ? i * kRows : 0) + row] = make_float2(m, l);
            }
            tc_fence_before();
            mbar_arrive(&sh.o_free);
            if (tid == 0 && g.t0 == 0 && !whole)
                tp.cuts[cta] = make_int4(g.b, g.h, g.tok0, g.last_cta);
            end(seg);
        }
    } else if (warp == MMA) {
        // ----------------------------------------------------------- products
        constexpr uint32_t qk = f16_idesc<T>(kRows, kKeys, false), pv = f16_idesc<T>(kRows, D, true);
        if (lane == 0) {
            auto wait_one = [&](uint64_t *bar, uint32_t parity) {
                if (mbar_wait_bounded(bar, parity, p.wait_limit_ns)) return true;
                give_up();
                return false;
            };
            const uint64_t qd = swz128_desc(smem_u32(qtile), 16, 1024), kd = swz128_desc(smem_u32(ring), 16, 1024);
            const uint64_t vd = swz128_desc(smem_u32(ring), BLOCK, 1024);
            uint32_t item = 0, count[2] = {0, 0};                 // ring items before the segment, tiles of each group
            auto scores = [&](int i, uint32_t at) {
                const uint64_t a = qd + (uint64_t)((WIDE ? i : 0) * NB * BLOCK >> 4);
                const uint64_t k0 = kd + (uint64_t)(at % NS * (kv_bytes<D>() >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = ((k / 4) * BLOCK + (k % 4) * 32) >> 4;
                    mma_ss(tmem + S_COL[i], a + off, k0 + off, qk, k > 0);
                }
                tc_commit(&sh.s_full[i]);
            };
            auto output = [&](int i, uint32_t at, bool add) {
                const uint64_t v0 = vd + (uint64_t)(at % NS * (kv_bytes<D>() >> 4));
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(tmem + O_COL[i], tmem + S_COL[i] + 8 * k, v0 + (uint64_t)(k * 2048 >> 4), pv, add || k > 0);
                tc_commit(&sh.pv_done[i]);
            };
            uint32_t loaded = 0;                                  // query tiles so far
            for (uint32_t seg = 0; ok; ++seg) {
                ok = wait_one(&sh.seg_full[seg % kSegments], seg / kSegments & 1);
                const Segment &g = sh.seg[seg % kSegments];
                if (!ok || g.b < 0) break;
                const int n = g.t1 - g.t0, groups = row_tiles(g);
                mbar_arrive(&sh.seg_empty[seg % kSegments]);
                if (n == 0) continue;                             // a sequence without tokens: zeros need no products
                auto first_scores = [&](int i, int j) {
                    // the weights of the last segment lie over the scores until its last output product is complete
                    ok = ok && (count[i] == 0 || wait_one(&sh.pv_done[i], (count[i] - 1) & 1));
                    if (!ok) return;
                    tc_fence_after();
                    scores(i, item + k_item(j));
                };
                auto keys_ready = [&](int j) {
                    const uint32_t at = item + k_item(j);
                    return wait_one(&sh.kv_full[at % NS], at / NS & 1);
                };
                ok = wait_one(&sh.q_full, loaded & 1) && keys_ready(0);
                ++loaded;
                tc_fence_after();
                if constexpr (WIDE) {
                    first_scores(0, 0);
                    if (groups > 1) first_scores(1, 0);
                    if (ok) tc_commit(&sh.kv_empty[(item + k_item(0)) % NS]);
                } else {
                    first_scores(0, 0);
                    if (ok) tc_commit(&sh.kv_empty[(item + k_item(0)) % NS]);
                    if (n > 1) {
                        ok = ok && keys_ready(1);
                        tc_fence_after();
                        first_scores(1, 1);
                        if (ok) tc_commit(&sh.kv_empty[(item + k_item(1)) % NS]);
                    }
                }
                if (ok && n <= LEAD) tc_commit(&sh.q_empty);      // no more scores in this segment
                for (int j = 0; ok && j < n; ++j) {
                    const uint32_t vt = item + v_item(j, n), kt = item + k_item(j + LEAD);
#pragma unroll
                    for (int x = 0; x < NQ; ++x) {
                        const int i = WIDE ? x : j & 1;
                        if (!ok || (WIDE && x >= groups)) continue;
                        ok = wait_one(&sh.p_full[i], count[i] & 1);      // the weights, this value tile and the next key tile
                        if (ok && j < LEAD && seg > 0) ok = wait_one(&sh.o_free, (seg - 1) & 1);
                        if (!ok) continue;
                        tc_fence_after();
                        output(i, vt, j >= LEAD);
                        ++count[i];
                        const bool last_group = !WIDE || x == groups - 1;
                        if (last_group) tc_commit(&sh.kv_empty[vt % NS]);
                        if (j + LEAD < n) {
                            // the weights lie over the scores: they are free once the output product is complete
                            ok = wait_one(&sh.pv_done[i], (count[i] - 1) & 1);
                            if (!ok) continue;
                            tc_fence_after();
                            scores(i, kt);
                            if (last_group) {
                                tc_commit(&sh.kv_empty[kt % NS]);
                                if (j + LEAD == n - 1) tc_commit(&sh.q_empty);
                            }
                        }
                    }
                }
                item += 2 * n;
            }
            // nothing of this CTA is under way when its tensor memory goes back
            tc_commit(&sh.drained);
            if (!mbar_wait_bounded(&sh.drained, 0, p.drain_limit_ns)) give_up();
        }
        __syncwarp();
    } else if (warp == LOAD) {
        // -------------------------------------------------------- pages by TMA
        // 16-bit: a lane brings one box of a tile, block lane % NB of page lane / NB.  E4M3: a
        // lane brings the codes of a page, one contiguous stretch.
        constexpr int PER_PAGE = FP8 ? 1 : NB;
        constexpr int RS = FP8 ? NC : NS;                         // stages that copies go to
        if (lane == 0) {
            prefetch_tensormap(&qmap);
            if (!FP8) {
                prefetch_tensormap(&kmap);
                prefetch_tensormap(&vmap);
            }
        }
        uint32_t item = 0, loaded = 0, tile_base = 0;
        const int ppt = kKeys / p.P;
        for (uint32_t seg = 0; begin(seg); ++seg) {
            const Segment &g = sh.seg[seg % kSegments];
            const int n = g.t1 - g.t0;
            const int32_t *table = p.block_table + (size_t)g.b * p.max_pages;
            float2 amax = make_float2(0.f, 0.f);                  // of the lane's page
            auto look_up = [&](int j) {                           // its first pool row, or -1
                const int k = (g.t0 + j) * ppt + lane / PER_PAGE;
                if (lane >= ppt * PER_PAGE || j >= n || k >= g.pages.count) return -1;
                const int phys = table[g.pages.page(k)];
                if (phys >= 0 && phys < p.num_phys) {
                    if constexpr (FP8) amax = *reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + g.h) * 4);
                    return (phys * p.Hkv + g.h) * p.P;
                }
                *(volatile int *)&sh.any_bad = 1;
                if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
                return -1;
            };
            auto bring = [&](int v, int row) {                    // the keys or values of a tile
                const uint32_t st = item % RS;
                uint64_t *full = FP8 ? &sh.code_full[st] : &sh.kv_full[st], *empty = FP8 ? &sh.code_empty[st] : &sh.kv_empty[st];
                ok = item < RS || wait(empty, (item / RS - 1) & 1);
                if (!ok) return;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0)) * p.P * (FP8 ? D : 128);
                if (lane == 0) {
                    sh.armed[st] = item / RS + 1;
                    mbar_arrive_expect_tx(full, bytes);
                }
                __syncwarp();
                if (row >= 0) {
                    if constexpr (FP8)
                        bulk_load(codes + (st * kKeys + lane * p.P) * D,
                                  static_cast<const uint8_t *>(v ? p.v_pool : p.k_pool) + (size_t)row * D, p.P * D, full);
                    else
                        tma_load_2d(ring + st * kv_bytes<D>() + (lane % NB) * BLOCK + (lane / NB) * p.P * 128, v ? &vmap : &kmap,
                                    full, (lane % NB) * 64, row);
                }
                ++item;
            };
            int row = look_up(0), before = -1;                    // of this tile and of the one before
            for (int t = 0; ok && t < n + LEAD - 1; ++t) {
                if (t < n) {
                    if constexpr (FP8) {
                        // a page without keys has the scale 0, under which a hidden score's -inf would be NaN
                        const int at = (tile_base + t) % kScaleRing;
                        for (int q = lane * p.P / 16; lane < ppt && q < (lane + 1) * p.P / 16; ++q) {
                            sh.ks[at][q] = row >= 0 ? fmaxf(fp8_scale(amax.x), 1e-30f) : 1.f;
                            sh.vamax[at][q] = row >= 0 ? amax.y : 0.f;
                        }
                        __syncwarp();
                    }
                    bring(0, row);
                }
                if (ok && t == (n < LEAD ? n : LEAD) - 1) {       // the queries, behind the first keys
                    ok = loaded == 0 || wait(&sh.q_empty, (loaded - 1) & 1);
                    if (ok && lane == 0) {
                        const int q_tiles = row_tiles(g);
                        sh.q_armed = loaded + 1;
                        mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(q_tiles * NB * per * p.G * 128));
                        for (int i = 0; i < q_tiles; ++i)
                            for (int c = 0; c < NB; ++c)
                                tma_load_3d(qtile + (i * NB + c) * BLOCK, &qmap, &sh.q_full, c * 64, g.h * p.G,
                                            g.b * p.T + g.tok0 + i * per);
                    }
                    ++loaded;
                }
                const int next = look_up(t + 1);
                if (ok && t >= LEAD - 1) bring(1, LEAD == 1 ? row : before);
                before = row;
                row = next;
            }
            tile_base += n;
            end(seg);
        }
    } else if (warp == KEEP) {
        // --------------------------------------------------- tiles looked after
        // Values that no row of the unit sees may be anything, and 0 * NaN is not 0: such rows
        // become zeros.  Only the tiles with drafted tokens, the pages where the sinks end
        // and the window begins, and tiles with bad or no pages have them.  (E4M3: done by
        // the warps that convert.)
        uint32_t item = 0, count[2] = {0, 0};
        for (uint32_t seg = 0; begin(seg); ++seg) {
            const Segment &g = sh.seg[seg % kSegments];
            const int n = g.t1 - g.t0, groups = row_tiles(g);
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t vt = item + v_item(j, n), st = vt % NS;
                ok = wait(&sh.kv_full[st], vt / NS & 1);
                if (!ok) break;
                if constexpr (!FP8) {
                    if (hidden_rows(p, sh, g, g.t0 + j)) {
                        for (int r = lane; r < kKeys; r += 32)
                            if (!row_seen(p, sh, g, g.t0 + j, r, tok_per))
#pragma unroll
                                for (int c = 0; c < NB * 8; ++c)
                                    *reinterpret_cast<uint4 *>(ring + st * kv_bytes<D>() + (c / 8) * BLOCK + r * 128 + c % 8 * 16) =
                                        make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                }
                if (j + LEAD < n) {
                    const uint32_t kt = item + k_item(j + LEAD);
                    ok = wait(&sh.kv_full[kt % NS], kt / NS & 1);
                }
                // one arrival in each phase: not before the last one is over
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const int i = WIDE ? x : j & 1;
                    if (!ok || (WIDE && x >= groups)) continue;
                    ok = count[i] == 0 || wait(&sh.p_full[i], (count[i] - 1) & 1);
                    ++count[i];
                    if (ok && lane == 0) mbar_arrive(&sh.p_full[i]);
                }
            }
            item += 2 * n;
            end(seg);
        }
    } else if (warp == PLAN) {
        // ------------------------------------------------------------ segments
        if (lane == 0) {
            Walk walk(tp, sh.seq0, sh.at0, sh.total, tok_per);
            Segment next;
            for (uint32_t seg = 0;; ++seg) {
                if (!walk.next(next)) next.b = -1;
                if (seg >= kSegments &&
                    !mbar_wait_bounded(&sh.seg_empty[seg % kSegments], (seg / kSegments - 1) & 1, p.wait_limit_ns)) {
                    give_up();
                    break;
                }
                sh.seg[seg % kSegments] = next;
                mbar_arrive(&sh.seg_full[seg % kSegments]);
                if (next.b < 0) break;
            }
        }
        __syncwarp();
    } else if (FP8 && warp >= CONVERT) {
        // ------------------------------------------------------ codes to halves
        constexpr int CPR = D / 16;                               // 16-code chunks of a row
        const int me = tid - CONVERT * 32;
        uint32_t item = 0;
        for (uint32_t seg = 0; begin(seg); ++seg) {
            const Segment &g = sh.seg[seg % kSegments];
            const int n = g.t1 - g.t0;
            for (int y = 0; ok && y < 2 * n; ++y, ++item) {
                // item y of the segment: the values of tile j if y is v_item(j, n)
                const int j = y == 2 * n - 1 ? n - 1 : max(y - LEAD, 0) / 2;
                const bool v = y == v_item(j, n);
                const int tile = g.t0 + j;
                const uint32_t cs = item % (NC ? NC : 1), st = item % NS;
                ok = wait(&sh.code_full[cs], item / (NC ? NC : 1) & 1) && (item < NS || wait(&sh.kv_empty[st], (item / NS - 1) & 1));
                if (!ok) break;
                const bool clean = v && hidden_rows(p, sh, g, tile);
                const unsigned char *from = codes + cs * kKeys * D;
                unsigned char *to = ring + st * kv_bytes<D>();
#pragma unroll 4
                for (int x = me; x < kKeys * CPR; x += 128) {
                    const int r = x / CPR, c = x % CPR;
                    uint4 w = *reinterpret_cast<const uint4 *>(from + x * 16), lo, hi;
                    if (clean && !row_seen(p, sh, g, tile, r, tok_per)) w = make_uint4(0, 0, 0, 0);
                    codes_to_h(w.x, &lo.x);
                    codes_to_h(w.y, &lo.z);
                    codes_to_h(w.z, &hi.x);
                    codes_to_h(w.w, &hi.z);
                    unsigned char *base = to + (2 * c / 8) * BLOCK + r * 128;
                    const int a = 2 * c % 8 ^ (r & 7), odd = c / 4 & 1;      // the two blocks' chunks lie in the same banks
                    *reinterpret_cast<uint4 *>(base + (odd ? a ^ 1 : a) * 16) = odd ? hi : lo;
                    *reinterpret_cast<uint4 *>(base + (odd ? a : a ^ 1) * 16) = odd ? lo : hi;
                }
                fence_async_smem();
                mbar_arrive(&sh.code_empty[cs]);
                mbar_arrive(&sh.kv_full[st]);
            }
            end(seg);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*(volatile int *)&sh.failed) {
        // Every copy has been waited for by the warps that used it, unless some wait gave
        // up: no copy may land after the CTA's end.
        if (tid == 0) {
            if (sh.q_armed > 0) (void)mbar_wait_bounded(&sh.q_full, (sh.q_armed - 1) & 1, p.drain_limit_ns);
            for (int st = 0; st < (FP8 ? NC : NS); ++st)
                if (sh.armed[st] > 0)
                    (void)mbar_wait_bounded(FP8 ? &sh.code_full[st] : &sh.kv_full[st], (sh.armed[st] - 1) & 1, p.drain_limit_ns);
        }
        // rows that other CTAs have parts of stay as they were
        if (tp.cuts)
            for (int r = tid; r < 2 * ROWS; r += THREADS) tp.part_ml[(size_t)2 * cta * ROWS + r] = make_float2(kGivenUp, -1.f);
    }
    if (warp == MMA) {
        tc_fence_after();
        tmem_free(tmem, TMEM);
    }
}

// Joins the pieces of the units that borders of stretches cut: the unit whose first piece
// CTA blockIdx.x has goes on in the CTAs after it, up to cuts[].w.  A thread takes eight
// channels of a row, its pieces in the order of the CTAs.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeParams tp) {
    constexpr int ROWS = (WIDE ? 2 : 1) * kRows;
    pdl_wait();
    const int cta = blockIdx.x;
    const int4 cut = tp.cuts[cta];
    if (cut.x < 0) return;
    const WindowParams &p = tp.w;
    const QuerySpan s = query_span(p, cut.x, false);
    const int per = kRows / p.G, tile_rows = per * p.G, rows = min((s.n - cut.z) * p.G, (WIDE ? 2 : 1) * tile_rows);
    for (int x = blockIdx.y * kJoinThreads + threadIdx.x; x < rows * (D / 8); x += kJoinBlocks * kJoinThreads) {
        const int r = x % rows, c = x / rows;                     // neighbours have neighbouring rows
        const int at = r / tile_rows * kRows + r % tile_rows;
        float top = -INFINITY;
        for (int k = cta; k <= cut.w; ++k) {
            const float2 ml = tp.part_ml[(size_t)slot_of(k, k == cta) * ROWS + at];
            if (ml.y != 0.f) top = fmaxf(top, ml.x);
        }
        float sum = 0.f, o[8] = {};
#pragma unroll 4
        for (int k = cta; k <= cut.w; ++k) {
            const int slot = slot_of(k, k == cta);
            const float2 ml = tp.part_ml[(size_t)slot * ROWS + at];
            const float4 *part = tp.part_o + ((size_t)slot * (D / 4) + 2 * c) * ROWS + at;
            const float4 a = part[0], b = part[ROWS];
            const float f = ml.y != 0.f ? exp2_fast(ml.x - top) : 0.f;
            if (ml.y == 0.f) continue;                            // NaN included: it goes through to the row
            sum = fmaf(f, ml.y, sum);
            o[0] = fmaf(f, a.x, o[0]); o[1] = fmaf(f, a.y, o[1]); o[2] = fmaf(f, a.z, o[2]); o[3] = fmaf(f, a.w, o[3]);
            o[4] = fmaf(f, b.x, o[4]); o[5] = fmaf(f, b.y, o[5]); o[6] = fmaf(f, b.z, o[6]); o[7] = fmaf(f, b.w, o[7]);
        }
        if (sum < 0.f) continue;                                  // a CTA gave up: the row stays as it was
        const float inv = sum != 0.f ? 1.f / sum : 0.f;           // a row that sees nothing is zero
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
        const int tok = cut.z + r / p.G;
        T *dst = static_cast<T *>(p.out) + (((size_t)cut.x * p.T + tok) * p.Hq + cut.y * p.G + r % p.G) * D + 8 * c;
        *reinterpret_cast<uint4 *>(dst) = chunk16<T>::pack(o);
    }
}

template <typename T, bool FP8, int D, bool WIDE>
cudaError_t launch_t(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const TreeParams &p, int ctas,
                     cudaStream_t stream) {
    constexpr size_t smem = tree_smem<D, FP8, WIDE>();
    static_assert(smem + sizeof(TreeShared) <= 227 << 10, "shared memory of an SM");
    auto kernel = tree_kernel<T, FP8, D, WIDE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(tree_threads<FP8>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    e = cudaLaunchKernelEx(&cfg, kernel, q, k, v, p);
    if (e != cudaSuccess || !p.cuts) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)ctas, kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D, WIDE>, p);
}

template <typename T, bool FP8>
cudaError_t launch_d(int D, bool wide, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const TreeParams &p,
                     int ctas, cudaStream_t stream) {
    if (D == 64) return wide ? launch_t<T, FP8, 64, true>(q, k, v, p, ctas, stream) : launch_t<T, FP8, 64, false>(q, k, v, p, ctas, stream);
    return wide ? launch_t<T, FP8, 128, true>(q, k, v, p, ctas, stream) : launch_t<T, FP8, 128, false>(q, k, v, p, ctas, stream);
}

}  // namespace

// Workspace of a call with this many CTAs: cuts, then maxima and sums, then partial outputs.
TreeWorkspace tree_workspace(int D, bool wide, int ctas) {
    const size_t rows = wide ? 2 * kRows : kRows;
    TreeWorkspace w;
    w.ml = (size_t)ctas * sizeof(int4);
    w.o = w.ml + 2 * (size_t)ctas * rows * sizeof(float2);
    w.bytes = w.o + 2 * (size_t)ctas * rows * D * sizeof(float);
    return w;
}

cudaError_t launch_tree(qasa_dtype dt, int D, bool wide, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                        const TreeParams &p, int ctas, cudaStream_t stream) {
    switch (dt) {
    case QASA_DTYPE_F16: return launch_d<__half, false>(D, wide, q, k, v, p, ctas, stream);
    case QASA_DTYPE_BF16: return launch_d<__nv_bfloat16, false>(D, wide, q, k, v, p, ctas, stream);
    case QASA_DTYPE_E4M3: return launch_d<__half, true>(D, wide, q, k, v, p, ctas, stream);
    default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace qasa
