// window_prompt.cu -- windowed attention for many query rows per KV head: prompts
// and prompt chunks, on the fifth-generation tensor cores.
//
//   S = Q K^T,  P = exp2(scale S - m),  O += P V,  out = O / sum P
//
// What bounds it: 4 d multiply-adds per visible (row, token) pair on the tensor
// cores, and one exponential per pair on the other pipes; keys and values are
// read once per 256 rows, from L2.  What it takes in fact is the chain of one row
// tile, S -> softmax -> O -> next S, which the other tile's chain overlaps.
//
// Rows: the G query heads of a KV head see the same keys, so a row tile packs
// (token, head) rows, 128 / G tokens of G heads: the keys are shared by the whole
// group and a tile spans few positions, which keeps partly hidden key tiles few.
// A CTA owns NQ row tiles and goes through their visible pages, sinks first, 128
// tokens at a time.  Its warps, for NQ = 2:
//   0-3, 4-7   one row tile each: a thread owns a row, reads its 128 scores from tensor
//              memory, and writes the weights back as the next product's 16-bit operand
//              over them; no shuffles (two threads to a row were slower, 342 against
//              318 us for a prompt of 8192: the products then take twice as long)
//   8          one thread issues the products, those of one tile while the other tile's
//              softmax runs; it is held while the tensor core is busy, so each wait of
//              its own is idle time there (two issuing threads: 435 against 336 us)
//   9          brings pages by TMA into a ring of key and value tiles
//   11         E4M3 caches: finds the largest value scale
//   10         zeroes hidden value rows of edge tiles, and waits for the tiles in the
//              issuing thread's place: the barrier of the weights takes its arrival too
// Tensor memory: S0, S1 (P over them), O0, O1.
//
// Where a call has fewer CTAs than the SMs hold (a few drafted tokens of a few
// sequences), a cluster shares a CTA's rows: each takes a stretch of the key tiles,
// and the partial outputs are joined through distributed shared memory, always in
// the same order.
//
// No maximum is sought where it is not needed: a tile's weights are taken against
// the maximum so far, and only where a row's weights of the tile then sum to more
// than kMostWeight is the tile's own maximum found, O and the sum rescaled and the
// tile done again.  Up to there nothing is lost: the sums are fp32, and 16-bit
// weights keep their relative half step whatever their size (window.cuh).
//
// E4M3 caches: a kernel before this one writes the codes of the pages in question as
// halves, which they are exactly (converting them here, once per 256 rows, kept the
// other warps waiting: 125 us for 2 x 2048 tokens over 1024).  The keys' scale then
// multiplies the scores and the values' scale the weights.
#include "tcgen05.cuh"
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kRows = 128;            // rows of a row tile
constexpr int kKeys = 128;            // tokens of a key tile
constexpr int kMostJoined = 8;        // CTAs that share the key tiles of their rows
constexpr float kGivenUp = 3e38f;     // maximum that a CTA reports for rows that it gave up
constexpr int kScaleRing = 8;         // key tiles whose E4M3 scales are kept

template <int D> constexpr int kv_bytes() { return kKeys * D * 2; }
constexpr int kStages = 5;            // key and value tiles in the ring
template <int D, int NQ> constexpr size_t prompt_smem() {
    return 1024 + (size_t)NQ * kRows * D * 2 + (size_t)kStages * kv_bytes<D>();
}

struct PromptShared {
    uint64_t q_full, kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2], pv_done[2], vmax_ready, drained;
    uint32_t tmem;
    int any_bad;         // some page of this CTA has a bad block-table entry
    int failed;          // a bounded wait gave up: the rows that waited are not written
    int armed[kStages];  // copies into each stage so far
    float vmax;          // E4M3: the largest V amax among the CTA's pages
    float ks[kScaleRing][kKeys / 16], vamax[kScaleRing][kKeys / 16];
};

// Pages that some query at [first, last] sees: pages 0 .. head of the sinks, then pages body0 ..
struct Pages {
    int lo, hi, head, body0, count;
    __device__ __forceinline__ int page(int k) const { return k < head ? k : body0 + k - head; }
};

__device__ __forceinline__ Pages visible_pages(int first, int last, int window, int sinks, int P) {
    Pages v;
    v.hi = last;
    v.lo = first - window + 1 > 0 ? first - window + 1 : 0;
    v.body0 = v.lo / P;
    v.head = min((min(sinks, v.lo) + P - 1) / P, v.body0);
    v.count = last < 0 ? 0 : v.head + last / P - v.body0 + 1;
    return v;
}

__device__ __forceinline__ bool good_page(const WindowParams &p, const int32_t *table, int page) {
    const int phys = table[page];
    return phys >= 0 && phys < p.num_phys;
}

// Bit c: token base + c is at or before x.
__device__ __forceinline__ uint32_t upto16(int x, int base) {
    const int n = x - base;
    return n < 0 ? 0u : n >= 15 ? 0xffffu : (2u << n) - 1u;
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
// NQ: row tiles of a CTA.  One where two CTAs fit an SM (64 channels): each brings its
// own keys, but the first loads and the last stores of one run under the other's
// products.
template <int NQ> constexpr int prompt_threads() { return NQ * 128 + 128; }

// T: 16-bit type of q, out and the pages; SCALED: pages of E4M3 values (as halves);
// JOIN: a cluster shares the key tiles (apart, as the other form's softmax is slower
// with the registers that this one wants).
template <typename T, bool SCALED, int D, int NQ, bool JOIN>
__global__ void __launch_bounds__(prompt_threads<NQ>(), NQ == 1 ? 2 : 1)
window_prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, WindowParams p) {
    constexpr int NB = D / 64;                        // 64-channel blocks
    constexpr int BLOCK = kRows * 128;                // bytes of one block of a tile
    constexpr int NS = kStages;
    constexpr uint32_t S_COL[2] = {0, 128}, O_COL[2] = {NQ * 128, NQ * 128 + D}, TMEM = NQ * 256;
    constexpr int MMA = 4 * NQ, LOAD = MMA + 1, KEEP = MMA + 2, LARGEST = MMA + 3;      // warps
    static_assert(NQ == 2 || D == 64, "tensor memory of two CTAs");

    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);   // the swizzle counts from 1 KB boundaries
    unsigned char *qtile = smem, *ring = smem + NQ * NB * BLOCK;
    __shared__ PromptShared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cluster = JOIN ? p.cluster : 1;
    const int rank = JOIN ? blockIdx.x % cluster : 0, unit = blockIdx.x / cluster;
    // later positions first: they see the most keys
    const int h = unit % p.Hkv, b = unit / p.Hkv % p.B;
    const int pair = p.row_tiles - 1 - unit / p.Hkv / p.B;
    const int seq = p.b0 + b;                         // E4M3: the workspace holds some sequences at a time
    const int per = kRows / p.G;                      // tokens of a row tile
    const QuerySpan s = query_span(p, seq, h == 0 && rank == 0 && pair == p.row_tiles - 1 && tid == 0);
    const int t0 = pair * NQ * per;
    if (t0 >= s.n) return;                            // the same for the whole cluster
    const int t_end = min(s.n, t0 + NQ * per);
    const Pages pages = visible_pages(s.first + t0, s.first + t_end - 1, p.window, p.sinks, p.P);
    const int ppt = kKeys / p.P;                      // pages of a key tile
    const int32_t *table = p.block_table + (size_t)seq * p.max_pages;
    // key tiles that each row tile goes through: up to its last position
    int tiles[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        tiles[i] = 0;
        if (i >= NQ) continue;
        const int last = s.first + min(s.n, t0 + (i + 1) * per) - 1;
        tiles[i] = t0 + i * per >= s.n || last < 0 ? 0 : (pages.head + max(last / p.P - pages.body0 + 1, 0) + ppt - 1) / ppt;
    }
    // this CTA's stretch: key tiles j0 .. j0 + n of the list, numbered from 0 below
    const int all = max(tiles[0], tiles[1]);
    const int j0 = JOIN ? all * rank / cluster : 0, n = JOIN ? all * (rank + 1) / cluster - j0 : all;
    if constexpr (JOIN) {
        tiles[0] = min(max(tiles[0] - j0, 0), n);
        tiles[1] = min(max(tiles[1] - j0, 0), n);
    }

    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
            sh.armed[i] = 0;
        }
        mbar_init(&sh.vmax_ready, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], kRows + 1);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.any_bad = 0;
        sh.failed = 0;
        fence_barrier_init();
    }
    if (warp == MMA) tmem_alloc(&sh.tmem, TMEM);
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
    // registers go to the softmax warps, within what the block was launched with:
    // 256 x 208 + 128 x 88 = 384 x 168, 128 x 184 + 128 x 72 = 256 x 128
    if (warp < MMA) {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    } else {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }

    float m = -INFINITY, l = 0.f;                     // of a softmax thread's row
    if (warp < MMA) {
        // ------------------------------------------------------------ softmax
        const int i = warp >> 2;
        const int row = tid & 127;
        const int tok = t0 + i * per + row / p.G, g = row % p.G;
        const bool live = row < per * p.G && tok < s.n;
        const int pos = s.first + tok;
        const int first = s.first + t0 + i * per, last = s.first + min(s.n, t0 + (i + 1) * per) - 1;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // tensor memory lane of this warp, bits 16 up
        const uint32_t sa = tmem + lanes + S_COL[i], oa = tmem + lanes + O_COL[i];
        float vscale = 1.f;
        if (!live) m = 0.f;
        bool ok = true;
        // Key tiles [whole0, whole1) are seen as a whole by every row of the row tile:
        // full tiles of window pages up to the first row's position (tiles of sinks
        // alone take the masked way).
        int whole0 = 0, whole1 = 0;
        if (first >= 0) {
            const int clear = max(last - p.window + p.P, 0) / p.P;     // first page wholly inside the last row's window
            whole0 = (pages.head + max(clear - pages.body0, 0) + ppt - 1) / ppt;
            if (pages.head > 0) whole0 = max(whole0, (pages.head + ppt - 1) / ppt);
            whole1 = (pages.head + max((first + 1) / p.P - pages.body0, 0)) / ppt;
            whole0 -= j0;
            whole1 -= j0;
        }
        bool unset = true;                    // a row of the warp has seen nothing yet
        if constexpr (SCALED) {
            ok = tiles[i] == 0 || wait(&sh.vmax_ready, 0);
            if (ok && tiles[i] > 0) vscale = sh.vmax > 0.f ? 1.f / sh.vmax : 0.f;
        }
        for (int j = 0; ok && j < tiles[i]; ++j) {
            if (!wait(&sh.s_full[i], j & 1)) { ok = false; break; }
            tc_fence_after();
            uint32_t x[kKeys];
            bool raise = unset, raised = false;
            const bool bad = *(volatile int *)&sh.any_bad != 0;
            const bool masked = bad || j < whole0 || j >= whole1;
            while (true) {
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(sa + c, x + c);
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int q = 0; q < kKeys / 16; ++q) {
                        const int k = (j0 + j) * ppt + q * 16 / p.P, pg = pages.page(k);
                        const int base = pg * p.P + q * 16 % p.P;
                        uint32_t seen = 0;
                        if (k < pages.count && (!bad || good_page(p, table, pg)))
                            seen = upto16(pos, base) & (upto16(p.sinks - 1, base) | ~upto16(pos - p.window, base));
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
                        top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) *
                                             (SCALED ? sh.ks[j % kScaleRing][q] : 1.f));
                    }
                    const float m_new = fmaxf(m, top * p.scale_log2 - kHeadroom<T>);
                    const float f = m_new == -INFINITY ? 1.f : exp2_fast(m - m_new);
                    m = m_new;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) { // the last product into O is complete: S of this tile follows it
                            uint32_t o[16];
                            tmem_ld16(oa + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(oa + c, o);
                        }
                        tmem_wait_st();
                    }
                    unset = __any_sync(0xffffffffu, m == -INFINITY);
                    raised = true;
                }
                const float base = m == -INFINITY ? 0.f : m;
                float2 sum[4] = {};
#pragma unroll
                for (int q = 0; q < kKeys / 16; ++q) {
                    float vs = 1.f, scale = p.scale_log2;
                    if constexpr (SCALED) {
                        vs = sh.vamax[j % kScaleRing][q] * vscale;
                        scale *= sh.ks[j % kScaleRing][q];
                    }
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const int e = q * 16 + c;
                        float2 w = fma2(x[e], x[e + 1], scale, -base);
                        w.x = exp2_fast(w.x);
                        w.y = exp2_fast(w.y);
                        sum[c / 2 & 3] = add2(sum[c / 2 & 3], w);
                        // weights in the values' 16-bit type: half a step each, while the sum keeps fp32
                        x[e / 2] = SCALED ? mma16816<T>::pack2(w.x * vs, w.y * vs) : mma16816<T>::pack2(w.x, w.y);
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
            tc_fence_before();
            mbar_arrive(&sh.p_full[i]);
        }
        if (ok && tiles[i] > 0) {
            ok = wait(&sh.pv_done[i], (tiles[i] - 1) & 1);
            tc_fence_after();
        }
        if constexpr (JOIN) {
            if (!ok) { m = kGivenUp; l = -1.f; }      // outweighs the other shares: the row's sum comes out negative
        } else if (ok) {
            float inv = l != 0.f ? 1.f / l : 0.f;     // a row that sees nothing is zero; a NaN query's sum is NaN
            if constexpr (SCALED) inv *= tiles[i] > 0 ? fp8_scale(sh.vmax) : 0.f;
            T *dst = static_cast<T *>(p.out) + (((size_t)seq * p.T + tok) * p.Hq + h * p.G + g) * D;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (tiles[i] > 0) {
                    tmem_ld32(oa + c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (live && l != 0.f) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float v[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[y] = __uint_as_float(o[e + y]) * inv;
                        *reinterpret_cast<uint4 *>(dst + c + e) = chunk16<T>::pack(v);
                    }
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(0, 0, 0, 0);
                }
            }
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
            auto scores = [&](int i, int stage) {
                const uint64_t a = qd + (uint64_t)(i * NB * BLOCK >> 4), k0 = kd + (uint64_t)(stage * (kv_bytes<D>() >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = ((k / 4) * BLOCK + (k % 4) * 32) >> 4;
                    mma_ss(tmem + S_COL[i], a + off, k0 + off, qk, k > 0);
                }
                tc_commit(&sh.s_full[i]);
            };
            auto output = [&](int i, int stage, bool add) {
                const uint64_t v0 = vd + (uint64_t)(stage * (kv_bytes<D>() >> 4));
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(tmem + O_COL[i], tmem + S_COL[i] + 8 * k, v0 + (uint64_t)(k * 2048 >> 4), pv, add || k > 0);
                tc_commit(&sh.pv_done[i]);
            };
            bool ok = n == 0 || (wait_one(&sh.q_full, 0) && wait_one(&sh.kv_full[0], 0));
            if (ok && n > 0) {
                tc_fence_after();
                if (tiles[0] > 0) scores(0, 0);
                if (tiles[1] > 0) scores(1, 0);
                tc_commit(&sh.kv_empty[0]);
            }
            for (int j = 0; ok && j < n; ++j) {
                const int vst = (2 * j + 1) % NS, kst = (2 * j + 2) % NS;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok || j >= tiles[i]) continue;
                    ok = wait_one(&sh.p_full[i], j & 1);    // the weights, this value tile and the next key tile
                    if (!ok) continue;
                    tc_fence_after();
                    output(i, vst, j > 0);
                    if (i == 1 || j >= tiles[1]) tc_commit(&sh.kv_empty[vst]);
                    if (j + 1 < tiles[i]) {
                        // the weights lie over the scores: they are free once the output product is complete
                        ok = wait_one(&sh.pv_done[i], j & 1);
                        if (!ok) continue;
                        tc_fence_after();
                        scores(i, kst);
                    }
                }
                if (ok && j + 1 < n) tc_commit(&sh.kv_empty[kst]);
            }
            // nothing of this CTA is under way when its tensor memory goes back
            tc_commit(&sh.drained);
            if (!mbar_wait_bounded(&sh.drained, 0, p.drain_limit_ns)) give_up();
        }
        __syncwarp();
    } else if (warp == LOAD) {
        // -------------------------------------------------------- pages by TMA
        // A lane brings one box of a tile: block lane % NB of page lane / NB.
        if (lane == 0) {
            prefetch_tensormap(&qmap);
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        if (n > 0 && lane == 0) {
            const int q_tiles = tiles[1] > 0 ? 2 : 1;           // the first tile has rows; its keys may all be hidden
            mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(q_tiles * NB * per * p.G * 128));
            for (int i = 0; i < q_tiles; ++i)
                for (int c = 0; c < NB; ++c)
                    tma_load_3d(qtile + (i * NB + c) * BLOCK, &qmap, &sh.q_full, c * 64, h * p.G, seq * p.T + t0 + i * per);
        }
        // E4M3: the pages of the whole call lie one after the other in the workspace
        Pages call{};
        if constexpr (SCALED) call = visible_pages(s.first, s.first + s.n - 1, p.window, p.sinks, p.P);
        float2 amax = make_float2(0.f, 0.f);                    // of the lane's page
        auto look_up = [&](int j) {                             // its first pool row, or -1
            const int k = (j0 + j) * ppt + lane / NB;
            if (lane >= ppt * NB || j >= n || k >= pages.count) return -1;
            const int pg = pages.page(k), phys = table[pg];
            if (phys >= 0 && phys < p.num_phys) {
                if constexpr (SCALED) {
                    amax = *reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + h) * 4);
                    const int at = pg < call.head ? pg : call.head + pg - call.body0;
                    return ((b * p.ws_pages + at) * p.Hkv + h) * p.P;
                }
                return (phys * p.Hkv + h) * p.P;
            }
            *(volatile int *)&sh.any_bad = 1;
            if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
            return -1;
        };
        int row = look_up(0);
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            if constexpr (SCALED) {
                // a page without keys has the scale 0, under which a hidden score's -inf would be NaN
                const int pg = lane / NB;
                for (int q = pg * p.P / 16; lane % NB == 0 && pg < ppt && q < (pg + 1) * p.P / 16; ++q) {
                    sh.ks[j % kScaleRing][q] = row >= 0 ? fmaxf(fp8_scale(amax.x), 1e-30f) : 1.f;
                    sh.vamax[j % kScaleRing][q] = row >= 0 ? amax.y : 0.f;
                }
            }
            const int next = look_up(j + 1);
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0)) * p.P * 128;
            for (int v = 0; v < 2; ++v) {
                const int at = 2 * j + v, st = at % NS;
                ok = at < NS || wait(&sh.kv_empty[st], (at / NS - 1) & 1);
                if (!ok) break;
                __syncwarp();
                if (lane == 0) {
                    sh.armed[st] = at / NS + 1;
                    mbar_arrive_expect_tx(&sh.kv_full[st], bytes);
                }
                __syncwarp();
                if (row >= 0)
                    tma_load_2d(ring + st * kv_bytes<D>() + (lane % NB) * BLOCK + (lane / NB) * p.P * 128, v ? &vmap : &kmap,
                                &sh.kv_full[st], (lane % NB) * 64, row);
            }
            row = next;
        }
    } else if (SCALED && warp == LARGEST) {
        // Weights carry the values' scales as a share of the largest one, so that
        // small scales lose nothing in 16 bits.
        float top = 0.f;
        for (int k = lane; k < pages.count; k += 32) {
            const int pg = pages.page(k);
            if (good_page(p, table, pg)) top = fmaxf(top, p.scales[((size_t)table[pg] * p.Hkv + h) * 4 + 1]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) {
            sh.vmax = top;
            mbar_arrive(&sh.vmax_ready);
        }
    } else if (warp == KEEP) {
        // --------------------------------------------------- tiles looked after
        // Values that no row sees may be anything, and 0 * NaN is not 0: such rows
        // become zeros.  Only the last page, the
        // pages where the sinks end and the window begins, and tiles with bad or no
        // pages have them.
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            const int vi = 2 * j + 1, st = vi % NS;
            ok = wait(&sh.kv_full[st], vi / NS & 1);
            if (!ok) break;
            const bool bad = *(volatile int *)&sh.any_bad != 0;
            const int k0 = (j0 + j) * ppt, k1 = k0 + ppt;
            if ((bad || k1 >= pages.count || (pages.lo > 0 && k0 <= pages.head && k1 >= pages.head))) {
                for (int r = lane; r < kKeys; r += 32) {
                    const int k = k0 + r / p.P, pg = pages.page(k), at = pg * p.P + r % p.P;
                    const bool seen = k < pages.count && at <= pages.hi && (at >= pages.lo || at < p.sinks) &&
                                      (!bad || good_page(p, table, pg));
                    if (!seen)
#pragma unroll
                        for (int c = 0; c < NB * 8; ++c)
                            *reinterpret_cast<uint4 *>(ring + st * kv_bytes<D>() + (c / 8) * BLOCK + r * 128 + c % 8 * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (j + 1 < n) ok = wait(&sh.kv_full[(vi + 1) % NS], (vi + 1) / NS & 1);
            // one arrival in each phase: not before the last one is over
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || j >= tiles[i]) continue;
                ok = j == 0 || wait(&sh.p_full[i], (j - 1) & 1);
                if (ok && lane == 0) mbar_arrive(&sh.p_full[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // Every copy has been waited for by the warps that used it, unless some wait gave
    // up: no copy may land after the CTA's end.
    if (tid == 0 && *(volatile int *)&sh.failed) {
        if (n > 0) (void)mbar_wait_bounded(&sh.q_full, 0, p.drain_limit_ns);
        for (int st = 0; st < NS; ++st)
            if (sh.armed[st] > 0) (void)mbar_wait_bounded(&sh.kv_full[st], (sh.armed[st] - 1) & 1, p.drain_limit_ns);
    }
    if constexpr (JOIN) {
        // Rows of D + 4 floats over the queries and the ring, which nothing uses any
        // more; the cluster's CTAs join and write a share of the rows each.
        constexpr int PITCH = D + 4;
        float *part = reinterpret_cast<float *>(qtile);
        float2 *state = reinterpret_cast<float2 *>(part + NQ * kRows * PITCH);    // maximum and sum of every row
        static_assert(NQ * kRows * (PITCH * 4 + 8) <= NQ * NB * BLOCK + NS * kv_bytes<D>(), "partial outputs");
        __syncthreads();                              // the copies' end, had one of the waits given up
        tc_fence_after();
        if (warp < MMA) {
            const int i = warp >> 2, row = tid & 127;
            const uint32_t oa = tmem + ((uint32_t)(warp & 3) << 21) + NQ * 128 + i * D;
            state[i * kRows + row] = make_float2(m, tiles[i] > 0 ? l : 0.f);
            if (tiles[i] > 0)
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(oa + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(part + (i * kRows + row) * PITCH + c + e) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
        }
        tc_fence_before();
        cluster_sync();
        if (warp < MMA) {
            const float unitv = SCALED ? fp8_scale(sh.vmax) : 1.f;
            const int rows0 = min(per, s.n - t0) * p.G, rows1 = NQ == 2 ? min(per, max(s.n - t0 - per, 0)) * p.G : 0;
            for (int x = rank * MMA * 32 + tid; x < (rows0 + rows1) * (D / 4); x += cluster * MMA * 32) {
                const int y = x / (D / 4), c = x % (D / 4) * 4, i = y >= rows0, row = i ? y - rows0 : y, r = i * kRows + row;
                float2 ml[kMostJoined];
                float4 v[kMostJoined];
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int k = 0; k < kMostJoined; ++k)
                    if (k < cluster) {
                        ml[k] = ld_cluster_v2(map_rank(state + r, k));
                        v[k] = ld_cluster_v4(map_rank(part + r * PITCH + c, k));   // anything where the sum is 0
                    }
#pragma unroll
                for (int k = 0; k < kMostJoined; ++k)
                    if (k < cluster && ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kMostJoined; ++k)
                    if (k < cluster && ml[k].y != 0.f) {          // NaN included: it goes through to the row
                        const float f = exp2_fast(ml[k].x - top);
                        sum = fmaf(f, ml[k].y, sum);
                        o.x = fmaf(f, v[k].x, o.x); o.y = fmaf(f, v[k].y, o.y);
                        o.z = fmaf(f, v[k].z, o.z); o.w = fmaf(f, v[k].w, o.w);
                    }
                if (sum < 0.f) continue;              // a CTA gave up: the row stays as it was
                const float inv = sum != 0.f ? unitv / sum : 0.f;  // a row that sees nothing is zero
                const int tok = t0 + i * per + row / p.G;
                T *dst = static_cast<T *>(p.out) + (((size_t)seq * p.T + tok) * p.Hq + h * p.G + row % p.G) * D + c;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(mma16816<T>::pack2(o.x * inv, o.y * inv),
                                                             mma16816<T>::pack2(o.z * inv, o.w * inv));
            }
        }
        cluster_sync();                               // nobody leaves while its part is read
    }
    if (warp == MMA) {
        tc_fence_after();
        tmem_free(tmem, TMEM);
    }
}

// The codes of the pages that some query of the call sees, as halves, page after page
// of a sequence: [batch][ws_pages][Hkv][P][d], keys then values.  One block of 256
// threads per (page, sequence); bound by the 5 bytes read and written per code pair.
__global__ void __launch_bounds__(256) unpack_codes_kernel(WindowParams p, int d, __half *keys, __half *values) {
    const int b = blockIdx.y, seq = p.b0 + b;
    const QuerySpan s = query_span(p, seq, false);
    if (s.n <= 0) return;
    const Pages call = visible_pages(s.first, s.first + s.n - 1, p.window, p.sinks, p.P);
    const int k = blockIdx.x;
    if (k >= call.count) return;
    const int phys = p.block_table[(size_t)seq * p.max_pages + call.page(k)];
    if (phys < 0 || phys >= p.num_phys) return;                 // reported where it is looked up for its use
    const size_t page = (size_t)p.Hkv * p.P * d;                // codes of a page
    const size_t from = phys * page, to = ((size_t)b * p.ws_pages + k) * page;
    const uint4 *src[2] = {reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.k_pool) + from),
                           reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.v_pool) + from)};
    __half *dst[2] = {keys + to, values + to};
#pragma unroll 2
    for (int x = threadIdx.x; x < (int)(page / 8); x += 256) {  // keys, then values
        const int v = x >= (int)(page / 16), at = x - v * (int)(page / 16);
        const uint4 c = ld_global_nc_v4(src[v] + at);
        uint4 lo, hi;
        codes_to_h(c.x, &lo.x);
        codes_to_h(c.y, &lo.z);
        codes_to_h(c.z, &hi.x);
        codes_to_h(c.w, &hi.z);
        reinterpret_cast<uint4 *>(dst[v])[2 * at] = lo;
        reinterpret_cast<uint4 *>(dst[v])[2 * at + 1] = hi;
    }
}

template <typename T, bool SCALED, int D>
cudaError_t launch_t(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, WindowParams p, cudaStream_t stream) {
    constexpr int NQ = D == 64 ? 1 : 2;
    constexpr size_t smem = prompt_smem<D, NQ>();
    const int per = NQ * (kRows / p.G);
    p.row_tiles = (p.T + per - 1) / per;
    const long long units = (long long)p.row_tiles * p.B * p.Hkv;
    // As many CTAs to a unit as fill the SMs, while each has two key tiles.  Clusters of
    // more than four find no place together in every part of the device: past half of
    // the slots they run one after another (4 x 16 tokens over 8192, window 2048, d 128:
    // 30.8 us with eight, 20.6 us with four).
    const long long slots = (NQ == 1 ? 2 : 1) * (long long)p.sms;
    const long long fill = slots / units, work = p.most_tiles / (2 * kKeys / 16);
    p.cluster = (int)(fill < work ? fill : work);
    if (p.cluster < 1) p.cluster = 1;
    if (p.cluster > kMostJoined) p.cluster = kMostJoined;
    if (p.cluster > 4 && units * p.cluster > slots / 2) p.cluster = 4;
    if (units * p.cluster > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kernel = p.cluster > 1 ? window_prompt_kernel<T, SCALED, D, NQ, true> : window_prompt_kernel<T, SCALED, D, NQ, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * p.cluster));
    cfg.blockDim = dim3(prompt_threads<NQ>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, q, k, v, p);
}

}  // namespace

cudaError_t launch_unpack_codes(int D, const WindowParams &p, void *keys, void *values, cudaStream_t stream) {
    unpack_codes_kernel<<<dim3(p.ws_pages, p.B), 256, 0, stream>>>(p, D, static_cast<__half *>(keys),
                                                                   static_cast<__half *>(values));
    return cudaGetLastError();
}

cudaError_t launch_window_prompt(qasa_dtype dt, int D, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                 const WindowParams &p, cudaStream_t stream) {
    switch (dt) {
    case QASA_DTYPE_F16:
        return D == 64 ? launch_t<__half, false, 64>(q, k, v, p, stream) : launch_t<__half, false, 128>(q, k, v, p, stream);
    case QASA_DTYPE_BF16:
        return D == 64 ? launch_t<__nv_bfloat16, false, 64>(q, k, v, p, stream)
                       : launch_t<__nv_bfloat16, false, 128>(q, k, v, p, stream);
    case QASA_DTYPE_E4M3:
        return D == 64 ? launch_t<__half, true, 64>(q, k, v, p, stream) : launch_t<__half, true, 128>(q, k, v, p, stream);
    default: return cudaErrorInvalidConfiguration;
    }
}

}  // namespace qasa
