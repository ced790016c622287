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
// ring.  The keys' scale multiplies the scores.  The values' scale, as a share of the
// largest one so far, under which the output is kept, goes into the weights' exponents; the
// sum of a page's weights is freed of it afterwards.
//
// No maximum is sought where none is needed: weights are taken against the maximum so far,
// 32 tokens at a time, and only where these then sum to more than kMostWeight does it rise,
// by a whole number, so that what there is of the tile's 16-bit weights is scaled exactly.
//
// Measured (device time with the join; d = 128, 32 query heads): 16 ragged trees of up to 24
// tokens over 500 to 4000, f16, 35 us (2.2 TB/s: 13 us are the start, the first tile and the
// join); 64 tokens over 32704, bf16, 48 us (2.8 TB/s, 0.71 PFLOP/s); 64 x 32 tokens over 8160,
// E4M3, 320 us (0.86 PFLOP/s).  One row tile per KV head (64 x 16 tokens over 8000, f16) streams
// at 5.6 TB/s.  In the middle of a call a pair of row tiles takes 3450 cycles for 128 tokens of
// 16-bit pages: 1650 for a group's softmax, 1800 until its next scores, the two groups in turn.
// E4M3: 4600 to 5050, 2500 and 2150 to 2500 (the softmax looks up scales and shares, and the
// converting warps, busy 45 % of the time, share the issue slots and shared memory).  The 108 tiles of
// a CTA of the large case are 510 to 550 thousand cycles, its start 15, each of its one or two ends of
// units 13: 600 thousand, 308 us at the 1.96 GHz that it runs at, and the join.
//
// Measured and slower: the whole tile's softmax unrolled (its 800 instructions are fetched by
// all SMs at once in every launch, and the two groups then meet: E4M3 400 us) or 64 tokens at
// a time (404); key tiles of 64 tokens with scores made ahead into a second buffer (580; 16 x 24
// tokens 44): more, smaller products and more barriers; E4M3 codes to halves by shifts and
// masks in place of the conversion instruction (407); the join with 8 pieces under way (328).
#include "tcgen05.cuh"
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kRows = 128;            // rows of a row tile
constexpr int kKeys = 128;            // tokens of a key tile
constexpr int kUnitCost = 2;          // tiles that a unit's beginning and end are worth
constexpr int kScaleRing = 16;        // key tiles whose E4M3 scales are kept (a power of two)
constexpr int kSegments = 4;          // segments told ahead
constexpr float kLeastShare = -60.f;  // log2 of the least share of the largest value scale that a weight carries
constexpr float kGivenUp = 3e38f;     // maximum that a CTA reports for rows that it gave up
constexpr int kJoinThreads = 128, kJoinBatch = 4;

template <bool FP8> constexpr int tree_threads() { return FP8 ? 512 : 384; }
template <int D> constexpr int kv_bytes() { return kKeys * D * 2; }
// Key and value tiles as halves, and as codes, under way.  128 channels: what fits.
template <int D, bool FP8, bool WIDE> constexpr int kStages = D == 64 ? 8 : FP8 ? 4 : 5;
template <int D, bool FP8, bool WIDE> constexpr int kCodeStages = !FP8 ? 0 : D == 64 ? 6 : WIDE ? 2 : 3;
template <int D, bool FP8, bool WIDE> constexpr size_t tree_smem() {
    return 1024 + (size_t)(WIDE ? 2 : 1) * kRows * D * 2 + (size_t)kStages<D, FP8, WIDE> * kv_bytes<D>() +
           (size_t)kCodeStages<D, FP8, WIDE> * kKeys * D + (WIDE ? 0 : 2 * 2 * kRows * sizeof(float2));
}

// Pages that the queries of a sequence see: pages 0 .. head of the sinks, then pages body0 ..
struct Pages {
    int lo, hi, head, body0, count;
    __device__ __forceinline__ int page(int k) const { return k < head ? k : body0 + k - head; }
};

__device__ __forceinline__ int page_shift(const WindowParams &p) { return p.P == 32 ? 5 : 4; }

__device__ __forceinline__ Pages visible_pages(const WindowParams &p, const QuerySpan &s) {
    Pages v;
    v.hi = s.len - 1;
    v.lo = s.first - p.window + 1 > 0 ? s.first - p.window + 1 : 0;    // of a query at depth 0
    const int shift = page_shift(p);
    v.body0 = v.lo >> shift;
    v.head = min((min(p.sinks, v.lo) + p.P - 1) >> shift, v.body0);
    v.count = s.len <= 0 ? 0 : v.head + (v.hi >> shift) - v.body0 + 1;
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
    uint64_t s_full[2], p_full[2], pv_done[2], o_free[2], joined, drained;
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    Segment seg[kSegments];
    uint32_t tmem;
    int any_bad;         // some page of this CTA has a bad block-table entry
    int failed;          // a bounded wait gave up: the rows that waited are not written
    int armed[8];        // copies into each stage (E4M3: of codes) so far
    int q_armed;
    int seq0, at0;       // the stretch begins in this sequence, whose first unit lies here on the line
    QuerySpan span0;
    int total, sums[16];
    float ks[kScaleRing][kKeys / 16], lv[kScaleRing][kKeys / 16];   // E4M3: factor of the scores, log2 of the values' amax
    float unit[2][2];    // E4M3: unit of each group's output
};

// How a line of `total` places (below 2^31) is shared: the first `more` CTAs have each + 1
// places, the others `each`; with fewer places than CTAs the last ones have none.
struct Line {
    int each, more;
    __device__ __forceinline__ explicit Line(int total) {
        each = (int)((uint32_t)total / gridDim.x);
        more = total - each * (int)gridDim.x;
    }
    __device__ __forceinline__ int begin(int c) const { return each * c + min(c, more); }
    // the last CTA whose stretch begins before place `end` > 0
    __device__ __forceinline__ int last_before(int end) const {
        const int border = more * (each + 1);
        return end <= border ? (int)((uint32_t)(end - 1) / (uint32_t)(each + 1))
                             : more + (int)((uint32_t)(end - 1 - border) / (uint32_t)each);
    }
};

// Units of a KV head of a sequence with n queries, tok_per of them to a unit; inv = 1 / tok_per,
// exact enough for up to 1024 tokens.
__device__ __forceinline__ int unit_blocks(int n, int tok_per, float inv) {
    return __float2int_rd(((float)(n + tok_per - 1) + 0.5f) * inv);
}

// Walks the units that a CTA's stretch [v0, v1) of the line touches.  Of the unit at u0
// the stretch has the tiles that lie in it, the first kUnitCost places being the unit's
// beginning; `p.whole_units`: it has the whole unit if it begins in the stretch.
struct Walk {
    const TreeParams &p;
    const Line line;
    int v0, v1, u0;
    int b, unit, blocks, units, tok_per;
    float inv_tok;
    QuerySpan s;
    Pages pages;
    int tiles;
    // the stretch begins in sequence `first`, of span `s`, whose first unit is at place `at`
    __device__ __forceinline__ Walk(const TreeParams &p, int first, const QuerySpan &s, int at, int total, int tok_per, float inv_tok)
        : p(p), line(total), v0(line.begin(blockIdx.x)), v1(line.begin(blockIdx.x + 1)), u0(at), b(first), unit(0), blocks(0),
          units(0), tok_per(tok_per), inv_tok(inv_tok), s(s) {
        if (b < p.w.B) sequence();
    }
    __device__ __forceinline__ void sequence() {
        pages = visible_pages(p.w, s);
        tiles = (pages.count * p.w.P + kKeys - 1) / kKeys;
        blocks = unit_blocks(s.n, tok_per, inv_tok);
        units = p.w.Hkv * blocks;
        unit = 0;
        // units that end before the stretch
        if (units > 0 && v0 > u0) {
            unit = min((int)((uint32_t)(v0 - u0) / (uint32_t)(tiles + kUnitCost)), units);
            u0 += unit * (tiles + kUnitCost);
        }
    }
    __device__ __forceinline__ bool next(Segment &g) {
        while (b < p.w.B && u0 < v1) {
            if (unit == units) {
                if (++b < p.w.B) {
                    s = query_span(p.w, b, false);
                    sequence();
                }
                continue;
            }
            g.t0 = v0 <= u0 ? 0 : max(v0 - u0 - kUnitCost, 0);
            g.t1 = min(max(v1 - u0 - kUnitCost, 0), tiles);
            if (p.whole_units) {
                g.t0 = 0;
                g.t1 = u0 >= v0 ? tiles : 0;
            }
            g.b = b;
            g.h = blocks == 1 ? unit : (int)((uint32_t)unit / (uint32_t)blocks);
            g.tok0 = (unit - g.h * blocks) * tok_per;
            g.tiles = tiles;
            g.s = s;
            g.pages = pages;
            const bool take = g.t1 > g.t0 || (tiles == 0 && u0 >= v0);
            u0 += tiles + kUnitCost;
            ++unit;
            if (!take) continue;
            // the last stretch that begins before the unit's end
            g.last_cta = line.last_before(u0);
            // full tiles of context pages wholly inside the deepest row's window
            const int shift = page_shift(p.w), ppt = kKeys >> shift, ctx = s.first;
            g.whole0 = g.whole1 = 0;
            if (ctx > 0) {
                const int clear = max(s.len - 1 - p.w.window + p.w.P, 0) >> shift;
                g.whole0 = (pages.head + max(clear - pages.body0, 0) + ppt - 1) >> (7 - shift);
                if (pages.head > 0) g.whole0 = max(g.whole0, (pages.head + ppt - 1) >> (7 - shift));
                g.whole1 = (pages.head + max((ctx >> shift) - pages.body0, 0)) >> (7 - shift);
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
// The words of mask rows that hold the drafted tokens of a key tile: first word, and the
// first token's number among the drafted ones.
constexpr int kMaskWords = 5;
__device__ __forceinline__ int tile_word(const WindowParams &p, const Segment &g, int tile) {
    const int k = tile * (kKeys >> page_shift(p));
    const int at = k < g.pages.head ? 0 : (g.pages.page(k) << page_shift(p)) - g.s.first;
    return max(at, 0) >> 5;
}
__device__ __forceinline__ void load_words(const WindowParams &p, const uint32_t *row, int word, uint32_t *w) {
#pragma unroll
    for (int i = 0; i < kMaskWords; ++i) w[i] = word + i < p.mask_words ? __ldg(row + word + i) : 0u;
}
// Bits at .. at + 15 (at > -16) of words that begin with number `word`.
__device__ __forceinline__ uint32_t bits16(const uint32_t *w, int word, int at) {
    if (at < 0) return w[0] << -at & 0xffffu;
    const int i = (at >> 5) - word;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int x = 0; x < kMaskWords; ++x) {
        if (x == i) lo = w[x];
        if (x == i + 1) hi = w[x];
    }
    return __funnelshift_r(lo, hi, at & 31) & 0xffffu;
}

// Which tokens of a key tile a query at `pos` with these mask words sees, all pages taken for good.
struct Seen { uint32_t w[4]; };
__device__ __forceinline__ Seen visible(const WindowParams &p, const Segment &g, int tile, int pos, const uint32_t *words,
                                        int word) {
    Seen r = {};
    const int shift = page_shift(p), ctx = g.s.first;
#pragma unroll 1
    for (int q = 0; q < kKeys / 16; ++q) {
        const int k = (tile << (7 - shift)) + (q >> (shift - 4));
        if (k >= g.pages.count) break;
        const int base = (g.pages.page(k) << shift) + (q * 16 & (p.P - 1));
        uint32_t seen = upto16(ctx - 1, base) & (upto16(p.sinks - 1, base) | ~upto16(pos - p.window, base));
        if (base + 15 >= ctx) seen |= bits16(words, word, base - ctx) & upto16(g.s.len - 1, base);
        const uint32_t put = seen << (q & 1) * 16;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x == q >> 1) r.w[x] |= put;
    }
    return r;
}
// Only the tokens of good pages.
__device__ __forceinline__ void only_good(const WindowParams &p, const Segment &g, int tile, Seen &r) {
    const int shift = page_shift(p);
#pragma unroll 1
    for (int q = 0; q < kKeys / 16; ++q) {
        const int k = (tile << (7 - shift)) + (q >> (shift - 4));
        if (k < g.pages.count && good_page(p, p.block_table + (size_t)g.b * p.max_pages, g.pages.page(k))) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x == q >> 1) r.w[x] &= ~(0xffffu << (q & 1) * 16);
    }
}

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (elem<T>::id == QASA_DTYPE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
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
    const int ppt = kKeys >> page_shift(p), k0 = tile * ppt, k1 = k0 + ppt;
    return *(volatile int *)&sh.any_bad != 0 || k1 >= g.pages.count || g.pages.page(k1 - 1) * p.P + p.P > g.s.first ||
           (g.pages.lo > 0 && k0 <= g.pages.head && k1 >= g.pages.head);
}
// Union of the mask words of the unit's tokens, for a whole warp.
__device__ __forceinline__ void any_words(const WindowParams &p, const Segment &g, int tok_per, int word, uint32_t *any) {
    const int end = min(g.s.n, g.tok0 + tok_per);
#pragma unroll
    for (int i = 0; i < kMaskWords; ++i) any[i] = 0;
    for (int t = g.tok0 + (threadIdx.x & 31); t < end; t += 32) {
        uint32_t w[kMaskWords];
        load_words(p, tree_row(p, g.b, t), word, w);
#pragma unroll
        for (int i = 0; i < kMaskWords; ++i) any[i] |= w[i];
    }
#pragma unroll
    for (int i = 0; i < kMaskWords; ++i) any[i] = __reduce_or_sync(0xffffffffu, any[i]);
}
// The rows of the tile that some row of the unit may see, for a whole warp.
__device__ __forceinline__ Seen seen_rows(const WindowParams &p, TreeShared &sh, const Segment &g, int tile, int tok_per) {
    const int word = tile_word(p, g, tile);
    uint32_t any[kMaskWords];
    any_words(p, g, tok_per, word, any);
    Seen r = visible(p, g, tile, g.s.first, any, word);
    if (*(volatile int *)&sh.any_bad) only_good(p, g, tile, r);
    return r;
}
__device__ __forceinline__ bool row_seen(const Seen &s, int r) {
    const uint32_t w = r < 64 ? (r < 32 ? s.w[0] : s.w[1]) : (r < 96 ? s.w[2] : s.w[3]);
    return w >> (r & 31) & 1u;
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
    // The scales of a tile are written when those copies alone are waited for that lie NS + NC items before its
    // keys: with two items to a tile, a softmax may still read the scales of a tile that much further back.
    static_assert(!FP8 || (NS + NC + 1) / 2 + LEAD <= kScaleRing, "a tile's scales stay until its softmax is done");
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
        // An output may be written again when it has been read: WIDE by its own group, else (the
        // first barrier alone) by both.  Segments in which it was not written do not count: a group
        // that idles through some would otherwise arrive in the other's place.
        for (int i = 0; i < NQ; ++i) mbar_init(&sh.o_free[i], WIDE ? kRows : 2 * kRows);
        mbar_init(&sh.joined, 2 * kRows);
        mbar_init(&sh.drained, 1);
        sh.any_bad = sh.failed = sh.q_armed = 0;
        sh.seq0 = p.B;
        fence_barrier_init();
        if (tp.cuts) tp.cuts[cta] = make_int4(-1, 0, 0, 0);
    }
    if (warp == MMA) tmem_alloc(&sh.tmem, TMEM);
    if (warp == LOAD && lane == 0) {
        prefetch_tensormap(&qmap);
        if (!FP8) {
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
    }

    // The length of the line, and the sequence in which this CTA's stretch begins: a
    // thread adds up a run of sequences, the warps' sums are added in order.
    const float inv_tok = 1.f / tok_per;
    {
        const int run = p.B <= THREADS ? 1 : (p.B + THREADS - 1) / THREADS, b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
        auto cost = [&](const QuerySpan &s) {
            const Pages v = visible_pages(p, s);
            return p.Hkv * unit_blocks(s.n, tok_per, inv_tok) * ((v.count * p.P + kKeys - 1) / kKeys + kUnitCost);
        };
        int mine = 0, c = 0;
        QuerySpan s{};
        for (int b = b0; b < b1; ++b) {
            s = query_span(p, b, cta == 0);
            c = cost(s);
            mine += c;
        }
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) sh.sums[warp] = before;
        before -= mine;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w == warp) before += total;
            total += sh.sums[w];
        }
        if (tid == 0) sh.total = total;
        const int v0 = Line(total).begin(cta);
        if (v0 >= before && v0 < before + mine)
            for (int b = b0;; ++b) {
                if (run > 1) {
                    s = query_span(p, b, false);
                    c = cost(s);
                }
                if (v0 < before + c) {
                    sh.seq0 = b;
                    sh.at0 = before;
                    sh.span0 = s;
                    break;
                }
                before += c;
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();              // the joining kernel takes the SMs that are done, and waits there for the others
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
    // 256 x 192 + 128 x 120 = 384 x 168, 256 x 160 + 256 x 96 = 512 x 128
    if (warp < MMA) {
        if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    } else {
        if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
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
            const int n = g.t1 - g.t0;
            const int tok = g.tok0 + (WIDE ? i * per : 0) + row / p.G, head = g.h * p.G + row % p.G;
            const bool live = row < per * p.G && tok < g.s.n;
            const bool busy = __any_sync(0xffffffffu, live);      // a warp without rows only keeps pace
            const uint32_t *mask = tree_row(p, g.b, live ? tok : 0);
            int pos = -1;                                         // context and depth, once a tile needs it
            const int mine = WIDE ? (i < row_tiles(g) ? n : 0) : (n + 1 - i) / 2;
            float m = live ? -INFINITY : 0.f, l = 0.f;
            float lref = -INFINITY;                               // E4M3: O is in units of 2^lref, the largest V amax so far
            bool unset = true;                                    // a row of the warp has seen nothing yet
            for (int k = 0; ok && k < mine; ++k) {
                const int j = WIDE ? k : 2 * k + i, tile = g.t0 + j;
                bool masked = tile < g.whole0 || tile >= g.whole1;
                Seen seen = {{~0u, ~0u, ~0u, ~0u}};
                if (busy && masked) {                             // before the scores are there
                    uint32_t words[kMaskWords];
                    const int word = tile_word(p, g, tile);
                    load_words(p, mask, word, words);
                    if (pos < 0) pos = max(g.s.first + (p.window < g.s.len ? tree_depth(p, mask, g.s.n) : 0), 0);
                    seen = visible(p, g, tile, pos, words, word);
                }
                if (!wait(&sh.s_full[i], done & 1)) { ok = false; break; }
                ++done;
                tc_fence_after();
                if (busy) {
                    const uint32_t scales_at = (tile_base + j) % kScaleRing;
                    if (*(volatile int *)&sh.any_bad) {
                        only_good(p, g, tile, seen);
                        masked = true;
                    }
                    auto scale_o = [&](float f) {                 // the last product into O is complete: S of this tile follows it
                        if (k == 0) return;
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(oa + c, o);
                            tmem_wait_ld16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(oa + c, o);
                        }
                        tmem_wait_st();
                    };
                    if constexpr (FP8) {
                        float top = -INFINITY;
#pragma unroll
                        for (int q = 0; q < kKeys / 16; ++q) top = fmaxf(top, sh.lv[scales_at][q]);
                        if (top > lref) {
                            scale_o(exp2_fast(lref - top));
                            lref = top;
                        }
                    }
                    // 32 tokens at a time, in a loop: its instructions, which every SM fetches anew in
                    // every launch, are a quarter of those of the whole tile
                    auto load_chunk = [&](int c, uint32_t *x) {
                        tmem_ld32(sa + 32 * c, x);
                        const uint32_t w = c < 2 ? (c == 0 ? seen.w[0] : seen.w[1]) : (c == 2 ? seen.w[2] : seen.w[3]);
                        tmem_wait_ld32(x);
                        if (masked)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(w >> e & 1u)) x[e] = __float_as_uint(-INFINITY);
                    };
                    auto scale_of = [&](int c, int h) { return FP8 ? sh.ks[scales_at][2 * c + h] : p.scale_log2; };
                    auto largest = [&](int c, const uint32_t *x) {
                        float top = -INFINITY;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float t[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                t[e] = fmaxf(fmaxf(__uint_as_float(x[h * 16 + e]), __uint_as_float(x[h * 16 + 4 + e])),
                                             fmaxf(__uint_as_float(x[h * 16 + 8 + e]), __uint_as_float(x[h * 16 + 12 + e])));
                            top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale_of(c, h));
                        }
                        return top;
                    };
                    if (unset) {                                  // the tile's own maximum
                        float top = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < kKeys / 32; ++c) {
                            uint32_t x[32];
                            load_chunk(c, x);
                            top = fmaxf(top, largest(c, x));
                        }
                        const float m_new = fmaxf(m, top - kHeadroom<T>);
                        const float f = m_new == -INFINITY ? 1.f : exp2_fast(m - m_new);
                        m = m_new;
                        l *= f;
                        scale_o(f);
                        unset = __any_sync(0xffffffffu, m == -INFINITY);
                    }
#pragma unroll 1
                    for (int c = 0; c < kKeys / 32; ++c) {
                        uint32_t x[32], w16[16];
                        load_chunk(c, x);
                        float add;
                        for (bool again = false;; again = true) {
                            const float base = m == -INFINITY ? 0.f : m;
                            add = 0.f;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float scale = scale_of(c, h);
                                const float share = FP8 ? fmaxf(sh.lv[scales_at][2 * c + h] - lref, kLeastShare) : 0.f;
                                float2 sum[2] = {};
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    float2 w = fma2(x[h * 16 + e], x[h * 16 + e + 1], scale, share - base);
                                    w.x = exp2_fast(w.x);
                                    w.y = exp2_fast(w.y);
                                    sum[e / 2 & 1] = add2(sum[e / 2 & 1], w);
                                    // weights in the values' 16-bit type, which both operands of the product share: half a
                                    // step each, while the sum keeps fp32 (what the rounding takes off would be a second
                                    // product, and columns that tensor memory has not)
                                    w16[(h * 16 + e) / 2] = mma16816<T>::pack2(w.x, w.y);
                                }
                                sum[0] = add2(sum[0], sum[1]);
                                const float s2 = sum[0].x + sum[0].y;
                                add = FP8 ? fmaf(s2, exp2_fast(-share), add) : add + s2;
                            }
                            if (again || !__any_sync(0xffffffffu, live && !(add <= kMostWeight))) break;
                            // Weights that grow large: the maximum rises by a whole number, so that what there
                            // is of the tile's weights is scaled by a power of two, without another rounding.
                            float rise = add <= kMostWeight ? 0.f : ceilf(largest(c, x) - kHeadroom<T> - m);
                            rise = rise > 0.f ? rise : 0.f;
                            const float f = rise < 127.f ? __int_as_float((127 - (int)rise) << 23) : 0.f;
                            m += rise;
                            l *= f;
                            scale_o(f);
                            tmem_wait_st();
#pragma unroll 1
                            for (int before = 0; before < c; ++before) {
                                uint32_t y[16];
                                tmem_ld16(sa + 16 * before, y);
                                tmem_wait_ld16(y);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float2 v = unpack2<T>(y[e]);
                                    y[e] = mma16816<T>::pack2(v.x * f, v.y * f);
                                }
                                tmem_st16(sa + 16 * before, y);
                            }
                        }
                        // over scores that have been read: columns 16 c .. of chunk c / 2
                        tmem_st16(sa + 16 * c, w16);
                        l += add;
                    }
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
            float f0 = FP8 && mine > 0 ? fp8_scale(exp2_fast(lref)) : 1.f, f1 = 0.f;     // factors of this group's output and of the other's
            if constexpr (!WIDE) {
                float2 *now = states + (seg & 1) * 2 * kRows;
                now[i * kRows + row] = make_float2(m, l);
                if (FP8 && row == 0) sh.unit[seg & 1][i] = f0;       // a warp without rows does not follow it
                tc_fence_before();
                mbar_arrive(&sh.joined);
                // with the long limit: a row is written by both groups or by none
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.joined, seg & 1, p.drain_limit_ns));
                if (!ok) {
                    give_up();
                    break;
                }
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
                for (int c = 0; c < COLS; c += 32) {
                    uint32_t o[32], u[32];
                    if (mine > 0) tmem_ld32(oa + c0 + c, o);
                    if (!WIDE && n > 1 - i) tmem_ld32(tmem + lanes + O_COL[1 - i] + c0 + c, u);
                    tmem_wait_ld32(o);
                    if (!WIDE) tmem_wait_ld32(u);
#pragma unroll
                    for (int e8 = 0; e8 < 32; e8 += 8) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {             // 0 of something that was never written is not 0
                            v[e] = f0 != 0.f ? __uint_as_float(o[e8 + e]) * f0 : 0.f;
                            if (!WIDE) v[e] += f1 != 0.f ? __uint_as_float(u[e8 + e]) * f1 : 0.f;
                        }
                        if (whole) {
                            if (live) *reinterpret_cast<uint4 *>(dst + c + e8) = chunk16<T>::pack(v);
                        } else {
                            float4 *to = part + (size_t)(c + e8) / 4 * ROWS;
                            to[0] = make_float4(v[0], v[1], v[2], v[3]);
                            to[ROWS] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
                if (!whole && (WIDE || i == 0)) tp.part_ml[(size_t)slot * ROWS + (WIDE ? i * kRows : 0) + row] = make_float2(m, l);
            }
            tc_fence_before();
            if (WIDE ? mine > 0 : n > 0) mbar_arrive(&sh.o_free[WIDE ? i : 0]);
            if (tid == 0 && g.t0 == 0 && !whole)
                tp.cuts[cta] = make_int4(g.b, g.h, g.tok0 | min(g.s.n - g.tok0, tok_per) << 16, g.last_cta);
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
            uint32_t outputs[2] = {0, 0};                         // segments in which each output was written before
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
                        if (ok && j < LEAD) {
                            const int o = WIDE ? i : 0;
                            ok = outputs[o] == 0 || wait_one(&sh.o_free[o], (outputs[o] - 1) & 1);
                            if (WIDE) ++outputs[o];
                        }
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
                if (!WIDE) ++outputs[0];
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
        uint32_t item = 0, loaded = 0, tile_base = 0;
        const int ppt = kKeys >> page_shift(p);
        for (uint32_t seg = 0; begin(seg); ++seg) {
            const Segment &g = sh.seg[seg % kSegments];
            const int n = g.t1 - g.t0;
            const int32_t *table = p.block_table + (size_t)g.b * p.max_pages;
            // a lane holds the place of page number `from` + lane of the list, and of the one 32 further on
            struct Place { int row; float2 amax; };               // first pool row, or -1
            auto look_up = [&](int at) {
                Place x{-1, make_float2(0.f, 0.f)};
                const int k = at + lane;
                if (k >= min(g.pages.count, g.t1 * ppt)) return x;
                const int phys = table[g.pages.page(k)];
                if (phys >= 0 && phys < p.num_phys) {
                    x.row = (phys * p.Hkv + g.h) * p.P;
                    if constexpr (FP8) x.amax = *reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + g.h) * 4);
                } else {
                    *(volatile int *)&sh.any_bad = 1;
                    if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
                }
                return x;
            };
            int from = g.t0 * ppt;
            Place here = look_up(from), there = look_up(from + 32);
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
            auto bring_queries = [&] {
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
            };
            // the first queries at once, later ones, which wait for the unit before, behind the first keys
            const int queries_at = loaded == 0 ? -1 : (n < LEAD ? n : LEAD) - 1;
            if (n > 0 && queries_at < 0) bring_queries();
            int row = -1, before = -1;                            // the lane's page of this tile and of the one before
            for (int t = 0; ok && t < n + LEAD - 1; ++t) {
                if (t < n) {
                    const int at = (g.t0 + t) * ppt;
                    if (at - from >= 32) {
                        from += 32;
                        here = there;
                        there = look_up(from + 32);
                    }
                    row = __shfl_sync(0xffffffffu, here.row, (at - from + lane / PER_PAGE) & 31);
                    if (lane >= ppt * PER_PAGE) row = -1;
                    if constexpr (FP8) {
                        const float ka = __shfl_sync(0xffffffffu, here.amax.x, (at - from + lane) & 31);
                        const float va = __shfl_sync(0xffffffffu, here.amax.y, (at - from + lane) & 31);
                        // a page without keys has the scale 0, under which a hidden score's -inf would be NaN
                        const float ks = row >= 0 ? fmaxf(fp8_scale(ka), 1e-30f) * p.scale_log2 : 1.f;
                        const float lv = row >= 0 && va > 0.f ? log2f(va) : -140.f;
                        for (int q = lane * p.P / 16; lane < ppt && q < (lane + 1) * p.P / 16; ++q) {
                            sh.ks[(tile_base + t) % kScaleRing][q] = ks;
                            sh.lv[(tile_base + t) % kScaleRing][q] = lv;
                        }
                        __syncwarp();
                    }
                    bring(0, row);
                }
                if (ok && t == queries_at) bring_queries();
                if (ok && t >= LEAD - 1) bring(1, LEAD == 1 ? row : before);
                before = row;
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
                        const Seen seen = seen_rows(p, sh, g, g.t0 + j, tok_per);
                        for (int r = lane; r < kKeys; r += 32)
                            if (!row_seen(seen, r))
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
            Walk walk(tp, sh.seq0, sh.span0, sh.at0, sh.total, tok_per, inv_tok);
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
        // A thread takes the same chunk of every eighth (or a multiple) row, so that its places in
        // the swizzled tile are a stride apart.  The halves of a chunk's codes go to two places; the
        // two 64-channel blocks lie in the same banks: half of the lanes store them the other way round.
        const uint32_t me = tid - CONVERT * 32, c = me % CPR, r0 = me / CPR;
        constexpr uint32_t ROW_STEP = 128 / CPR;
        const bool swap = c / 4 & 1;
        const uint32_t place = (2 * c / 8) * BLOCK + r0 * 128, chunk = (2 * c % 8 ^ (r0 & 7)) * 16;
        const uint32_t first = place + (swap ? chunk ^ 16 : chunk), second = place + (swap ? chunk : chunk ^ 16);
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
                Seen seen = {};
                if (clean) seen = seen_rows(p, sh, g, tile, tok_per);
                const unsigned char *from = codes + cs * kKeys * D + me * 16;
                unsigned char *to = ring + st * kv_bytes<D>();
                constexpr int BATCH = 4, STEPS = kKeys * CPR / 128;
#pragma unroll
                for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
                    uint4 w[BATCH];
#pragma unroll
                    for (int u = 0; u < BATCH; ++u) w[u] = *reinterpret_cast<const uint4 *>(from + (s0 + u) * 2048);
                    if (clean)
#pragma unroll
                        for (int u = 0; u < BATCH; ++u)
                            if (!row_seen(seen, r0 + (s0 + u) * ROW_STEP)) w[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < BATCH; ++u) {
                        uint4 h;
                        codes_to_h(swap ? w[u].z : w[u].x, &h.x);
                        codes_to_h(swap ? w[u].w : w[u].y, &h.z);
                        *reinterpret_cast<uint4 *>(to + first + (s0 + u) * ROW_STEP * 128) = h;
                        codes_to_h(swap ? w[u].x : w[u].z, &h.x);
                        codes_to_h(swap ? w[u].y : w[u].w, &h.z);
                        *reinterpret_cast<uint4 *>(to + second + (s0 + u) * ROW_STEP * 128) = h;
                    }
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
// CTA blockIdx.y has goes on in the CTAs after it, up to cuts[].w.  A thread takes eight
// channels of a row and its pieces in the order of the CTAs, kJoinBatch of them under way at
// once, states and outputs together: after the cut's record one round trip to L2 is all
// that a unit of few pieces waits for.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeParams tp) {
    constexpr int ROWS = (WIDE ? 2 : 1) * kRows;
    const int cta = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const WindowParams &p = tp.w;
    const int per = kRows / p.G, tile_rows = per * p.G;
    const int r = (int)(blockIdx.x / (D / 32)) * 32 + lane, c = (int)(blockIdx.x % (D / 32)) * 4 + warp;   // row, eight channels
    pdl_wait();
    const int4 cut = tp.cuts[cta];
    const int tok0 = cut.z & 0xffff, rows = (cut.z >> 16) * p.G;
    if (cut.x < 0 || r >= rows) return;
    const int at = r < tile_rows ? r : kRows + r - tile_rows;
    float top = -INFINITY, sum = 0.f, o[8] = {};
    for (int k0 = cta; k0 <= cut.w; k0 += kJoinBatch) {
        float2 ml[kJoinBatch];
        float4 a[kJoinBatch], b[kJoinBatch];
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u) {
            const int k = k0 + u, slot = slot_of(k, k == cta);
            ml[u] = make_float2(-INFINITY, 0.f);
            a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k <= cut.w) {
                const float4 *part = tp.part_o + ((size_t)slot * (D / 4) + 2 * c) * ROWS + at;
                ml[u] = tp.part_ml[(size_t)slot * ROWS + at];
                a[u] = part[0];
                b[u] = part[ROWS];
            }
        }
        float now = top;
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u)
            if (ml[u].y != 0.f) now = fmaxf(now, ml[u].x);
        const float old = now == top ? 1.f : exp2_fast(top - now);
        top = now;
        sum *= old;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= old;
#pragma unroll
        for (int u = 0; u < kJoinBatch; ++u) {
            if (ml[u].y == 0.f) continue;                         // its output was never written; NaN included goes through
            const float f = exp2_fast(ml[u].x - top);
            sum = fmaf(f, ml[u].y, sum);
            o[0] = fmaf(f, a[u].x, o[0]); o[1] = fmaf(f, a[u].y, o[1]); o[2] = fmaf(f, a[u].z, o[2]); o[3] = fmaf(f, a[u].w, o[3]);
            o[4] = fmaf(f, b[u].x, o[4]); o[5] = fmaf(f, b[u].y, o[5]); o[6] = fmaf(f, b[u].z, o[6]); o[7] = fmaf(f, b[u].w, o[7]);
        }
    }
    if (sum < 0.f) return;                                        // a CTA gave up: the row stays as it was
    const float inv = sum != 0.f ? 1.f / sum : 0.f;               // a row that sees nothing is zero
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    T *dst = static_cast<T *>(p.out) + (((size_t)cut.x * p.T + tok0 + r / p.G) * p.Hq + cut.y * p.G + r % p.G) * D + 8 * c;
    *reinterpret_cast<uint4 *>(dst) = chunk16<T>::pack(o);
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
    cfg.gridDim = dim3((WIDE ? 2 : 1) * kRows / 32 * (D / 32), (unsigned)ctas);
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
