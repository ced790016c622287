// window_prompt.cu -- windowed attention for many query rows per KV head: prompts
// and prompt chunks, on the fifth-generation tensor cores.
//
//   S = Q K^T,  P = exp2(scale S - m),  O += P V,  out = O / sum P
//
// What bounds it: 4 d multiply-adds per visible (row, token) pair on the tensor
// cores, and one exponential per pair on the other pipes; keys and values are
// read once per 256 rows, from L2.
//
// Rows: the G query heads of a KV head see the same keys, so a row tile packs
// (token, head) rows, 128 / G tokens of G heads: the keys are shared by the whole
// group and a tile spans few positions, which keeps partly hidden key tiles few.
// A CTA owns two row tiles and goes through their visible pages, sinks first,
// 128 tokens at a time:
//   warps 0-3, 4-7   one row tile each: a thread owns a row, reads its 128 scores
//                    from tensor memory, and writes the weights back as the next
//                    product's 16-bit operand over them; no shuffles
//   warp 8           issues the products, S of one tile while the other tile's
//                    softmax runs
//   warp 9           brings pages by TMA into a ring of key and value tiles
//   warps 12-15      E4M3 caches only: read codes, write f16 tiles into the ring
// Tensor memory (512 columns): S0, S1 (P over them), O0, O1.
//
// The running maximum is raised only when a row's scores pass it by more than
// 2^8: until then weights up to 256 are exact enough in 16 bits and fp32 sums, and
// O needs no rescaling.
#include "tcgen05.cuh"
#include "window.cuh"

namespace qasa {

namespace {

constexpr int kRows = 128;            // rows of a row tile
constexpr int kKeys = 128;            // tokens of a key tile
constexpr float kSlack = 8.f;         // log2 units the scores may pass the running maximum
constexpr int kScaleRing = 8;         // key tiles whose E4M3 scales are kept

template <int D> constexpr int kv_bytes() { return kKeys * D * 2; }
template <int D> constexpr int ring_stages() { return D == 128 ? 5 : 8; }
template <int D> constexpr size_t prompt_smem() {
    return 1024 + (size_t)2 * kRows * D * 2 + (size_t)ring_stages<D>() * kv_bytes<D>();
}

struct PromptShared {
    uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2], pv_done[2], drained;
    uint32_t tmem;
    int any_bad;         // some page of this CTA has a bad block-table entry
    int failed;          // a bounded wait gave up: nothing is written
    uint32_t vref;       // E4M3: bits of the largest V scale among the CTA's pages
    float ks[kScaleRing][kKeys / 16], vs[kScaleRing][kKeys / 16];
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
__device__ __forceinline__ void mul2(uint32_t &x, uint32_t &y, float scale) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}" : "+r"(x), "+r"(y) : "f"(scale));
}

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(FP8 ? 512 : 384, 1)
window_prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, WindowParams p) {
    constexpr int NB = D / 64;                        // 64-channel blocks
    constexpr int BLOCK = kRows * 128;                // bytes of one block of a tile
    constexpr int NS = ring_stages<D>();
    constexpr uint32_t S_COL[2] = {0, 128}, O_COL[2] = {256, 256 + D};

    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);   // the swizzle counts from 1 KB boundaries
    unsigned char *qtile = smem, *ring = smem + 2 * NB * BLOCK;
    __shared__ PromptShared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // later positions first: they see the most keys
    const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv % p.B;
    const int pair = p.row_tiles - 1 - (int)(blockIdx.x / p.Hkv / p.B);
    const int per = kRows / p.G;                      // tokens of a row tile
    const QuerySpan s = query_span(p, b, h == 0 && pair == p.row_tiles - 1 && tid == 0);
    const int t0 = pair * 2 * per;
    if (t0 >= s.n) return;
    const int t_end = min(s.n, t0 + 2 * per);
    const Pages pages = visible_pages(s.first + t0, s.first + t_end - 1, p.window, p.sinks, p.P);
    const int ppt = kKeys / p.P;                      // pages of a key tile
    const int32_t *table = p.block_table + (size_t)b * p.max_pages;
    // key tiles that each row tile goes through: up to its last position
    int tiles[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = s.first + min(s.n, t0 + (i + 1) * per) - 1;
        tiles[i] = t0 + i * per >= s.n || last < 0 ? 0 : (pages.head + max(last / p.P - pages.body0 + 1, 0) + ppt - 1) / ppt;
    }
    const int n = max(tiles[0], tiles[1]);

    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.kv_full[i], FP8 ? 128 : 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], kRows);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.any_bad = 0;
        sh.failed = 0;
        sh.vref = 0;
        fence_barrier_init();
    }
    if (warp == 8) tmem_alloc(&sh.tmem, 512);
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
    // 256 x 208 + 128 x 88 = 384 x 168, and 256 x 184 + 128 x 56 + 128 x 88 = 512 x 128
    if (warp < 8) {
        if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    } else if (FP8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int i = warp >> 2;
        const int row = tid & 127;
        const int tok = t0 + i * per + row / p.G, g = row % p.G;
        const bool live = row < per * p.G && tok < s.n;
        const int pos = s.first + tok;
        const int first = s.first + t0 + i * per, last = s.first + min(s.n, t0 + (i + 1) * per) - 1;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // tensor memory lane of this warp, bits 16 up
        const uint32_t sa = tmem + lanes + S_COL[i], oa = tmem + lanes + O_COL[i];
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        // Whether every row of this row tile sees the whole key tile j.
        auto whole_tile = [&](int j) {
            const int k0 = j * ppt, k1 = k0 + ppt - 1;
            if (k1 >= pages.count) return false;
            const int base = pages.page(k0) * p.P, end = pages.page(k1) * p.P + p.P;     // the pages lie in between
            return end - 1 <= first && (end <= p.sinks || base > last - p.window);
        };
        for (int j = 0; j < tiles[i]; ++j) {
            if (!wait(&sh.s_full[i], j & 1)) { ok = false; break; }
            tc_fence_after();
            uint32_t x[kKeys];
            tmem_ld32(sa, x);
            tmem_ld32(sa + 32, x + 32);
            tmem_ld32(sa + 64, x + 64);
            tmem_ld32(sa + 96, x + 96);
            tmem_wait_ld();
            const bool bad = *(volatile int *)&sh.any_bad != 0;
            if constexpr (FP8) {
#pragma unroll
                for (int q = 0; q < kKeys / 16; ++q) {
                    const float ks = sh.ks[j % kScaleRing][q];
#pragma unroll
                    for (int c = 0; c < 16; c += 2) mul2(x[q * 16 + c], x[q * 16 + c + 1], ks);
                }
            }
            if (bad || !whole_tile(j)) {
#pragma unroll
                for (int q = 0; q < kKeys / 16; ++q) {
                    const int k = j * ppt + q * 16 / p.P, pg = pages.page(k);
                    const int base = pg * p.P + q * 16 % p.P;
                    uint32_t seen = 0;
                    if (k < pages.count && (!bad || good_page(p, table, pg)))
                        seen = upto16(pos, base) & (upto16(p.sinks - 1, base) | ~upto16(pos - p.window, base));
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (!(seen >> c & 1u)) x[q * 16 + c] = __float_as_uint(-INFINITY);
                }
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kKeys; c += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tops[e] = fmaxf(tops[e], fmaxf(__uint_as_float(x[c + e]), __uint_as_float(x[c + 4 + e])));
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * p.scale_log2;
            if (j == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, top > m + kSlack)) {
                const float m_new = fmaxf(m, top);
                const float f = m_new == -INFINITY ? 1.f : exp2_fast(m - m_new);
                m = m_new;
                l *= f;
#pragma unroll
                for (int c = 0; c < D; c += 32) {     // the last product into O is complete: S of this tile follows it
                    uint32_t o[32];
                    tmem_ld32(oa + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st32(oa + c, o);
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            float2 sum[4] = {};
#pragma unroll
            for (int q = 0; q < kKeys / 16; ++q) {
                float vs = 1.f;
                if constexpr (FP8) vs = sh.vs[j % kScaleRing][q];
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    const int e = q * 16 + c;
                    float2 w = fma2(x[e], x[e + 1], p.scale_log2, -base);
                    w.x = exp2_fast(w.x);
                    w.y = exp2_fast(w.y);
                    sum[c / 2 & 3] = add2(sum[c / 2 & 3], w);
                    // weights in the values' 16-bit type: half a step each, while the sum keeps fp32
                    x[e / 2] = FP8 ? mma16816<T>::pack2(w.x * vs, w.y * vs) : mma16816<T>::pack2(w.x, w.y);
                }
            }
            sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            l += sum[0].x + sum[0].y;
            tmem_st32(sa, x);
            tmem_st32(sa + 32, x + 32);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.p_full[i]);
        }
        if (ok && tiles[i] > 0) {
            ok = wait(&sh.pv_done[i], (tiles[i] - 1) & 1);
            tc_fence_after();
        }
        if (ok) {
            float inv = l > 0.f ? 1.f / l : 0.f;      // a row that sees nothing is zero
            if constexpr (FP8) inv *= __uint_as_float(*(volatile uint32_t *)&sh.vref);
            T *dst = static_cast<T *>(p.out) + (((size_t)b * p.T + tok) * p.Hq + h * p.G + g) * D;
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
                if (live && l > 0.f) {
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
    } else if (warp == 8) {
        // ----------------------------------------------------------- products
        constexpr uint32_t qk = f16_idesc<T>(kRows, kKeys, false), pv = f16_idesc<T>(kRows, D, true);
        const uint32_t q_addr = smem_u32(qtile), r_addr = smem_u32(ring);
        auto scores = [&](int i, int stage) {
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * BLOCK + (k % 4) * 32;
                    mma_ss(tmem + S_COL[i], swz128_desc(q_addr + i * NB * BLOCK + off, 16, 1024),
                           swz128_desc(r_addr + stage * kv_bytes<D>() + off, 16, 1024), qk, k > 0);
                }
                tc_commit(&sh.s_full[i]);
            }
            __syncwarp();
        };
        auto output = [&](int i, int stage, bool add) {
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(tmem + O_COL[i], tmem + S_COL[i] + 8 * k,
                           swz128_desc(r_addr + stage * kv_bytes<D>() + k * 2048, BLOCK, 1024), pv, add || k > 0);
                tc_commit(&sh.pv_done[i]);
            }
            __syncwarp();
        };
        auto release = [&](int stage) {
            if (lane == 0) tc_commit(&sh.kv_empty[stage]);
            __syncwarp();
        };
        // Values that no row sees may be anything, and 0 * NaN is not 0: such rows
        // of an edge tile become zeros.
        auto clean = [&](int j, int stage) {
            const bool bad = *(volatile int *)&sh.any_bad != 0;
            bool any = bad || (j + 1) * ppt > pages.count;
            for (int k = j * ppt; k < min((j + 1) * ppt, pages.count); ++k) {
                const int base = pages.page(k) * p.P;
                any |= base + p.P - 1 > pages.hi || (base < pages.lo && base + p.P > p.sinks);
            }
            if (!any) return;
            for (int r = lane; r < kKeys; r += 32) {
                const int k = j * ppt + r / p.P, pg = pages.page(k), at = pg * p.P + r % p.P;
                const bool seen = k < pages.count && at <= pages.hi && (at >= pages.lo || at < p.sinks) &&
                                  (!bad || good_page(p, table, pg));
                if (!seen)
#pragma unroll
                    for (int c = 0; c < NB * 8; ++c)
                        *reinterpret_cast<uint4 *>(ring + stage * kv_bytes<D>() + (c / 8) * BLOCK + r * 128 + c % 8 * 16) =
                            make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
        };
        bool ok = n == 0 || (wait(&sh.q_full, 0) && wait(&sh.kv_full[0], 0));
        if (ok && n > 0) {
            tc_fence_after();
            for (int i = 0; i < 2; ++i)
                if (tiles[i] > 0) scores(i, 0);
            release(0);
        }
        for (int j = 0; ok && j < n; ++j) {
            const int vi = 2 * j + 1, ki = 2 * j + 2, vst = vi % NS, kst = ki % NS;
            ok = wait(&sh.kv_full[vst], vi / NS & 1);
            if (!ok) break;
            if constexpr (!FP8) clean(j, vst);
            bool have_k = false;
            for (int i = 0; ok && i < 2; ++i) {
                if (j >= tiles[i]) continue;
                ok = wait(&sh.p_full[i], j & 1);
                if (!ok) break;
                tc_fence_after();
                output(i, vst, j > 0);
                if (i == 1 || j >= tiles[1]) release(vst);
                if (j + 1 < tiles[i]) {
                    if (!have_k) {
                        ok = wait(&sh.kv_full[kst], ki / NS & 1);
                        have_k = true;
                    }
                    // the weights lie over the scores: they are free once the output product is complete
                    ok = ok && wait(&sh.pv_done[i], j & 1);
                    if (!ok) break;
                    tc_fence_after();
                    scores(i, kst);
                }
            }
            if (ok && have_k) release(kst);
        }
        // nothing of this CTA is under way when its tensor memory goes back
        if (lane == 0) tc_commit(&sh.drained);
        __syncwarp();
        if (!mbar_wait_bounded(&sh.drained, 0, p.drain_limit_ns)) give_up();
    } else if (!FP8 && warp == 9) {
        // -------------------------------------------------------- pages by TMA
        if (lane == 0) {
            prefetch_tensormap(&qmap);
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        int issued = 0;
        if (n > 0) {
            if (lane == 0) {
                const int q_tiles = tiles[1] > 0 ? 2 : 1;       // the first tile has rows; its keys may all be hidden
                mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(q_tiles * NB * per * p.G * 128));
                for (int i = 0; i < q_tiles; ++i)
                    for (int c = 0; c < NB; ++c)
                        tma_load_3d(qtile + (i * NB + c) * BLOCK, &qmap, &sh.q_full, c * 64, h * p.G,
                                    b * p.T + t0 + i * per);
            }
            // a lane brings block lane % NB of page lane / NB of a tile
            auto look_up = [&](int j) {
                const int k = j * ppt + lane / NB;
                if (lane >= ppt * NB || j >= n || k >= pages.count) return -1;
                const int phys = table[pages.page(k)];
                if (phys >= 0 && phys < p.num_phys) return phys;
                *(volatile int *)&sh.any_bad = 1;
                if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
                return -1;
            };
            int phys = look_up(0);
            bool ok = true;
            for (int j = 0; ok && j < n; ++j) {
                const int next = look_up(j + 1);
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, phys >= 0)) * p.P * 128;
                for (int v = 0; v < 2; ++v) {
                    const int at = 2 * j + v, st = at % NS;
                    ok = at < NS || wait(&sh.kv_empty[st], (at / NS - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], bytes);
                    __syncwarp();
                    if (phys >= 0)
                        tma_load_2d(ring + st * kv_bytes<D>() + (lane % NB) * BLOCK + (lane / NB) * p.P * 128,
                                    v ? &vmap : &kmap, &sh.kv_full[st], (lane % NB) * 64, (phys * p.Hkv + h) * p.P);
                    issued = at + 1;
                }
                phys = next;
            }
            // every copy has landed before the CTA may end
            if (!mbar_wait_bounded(&sh.q_full, 0, p.drain_limit_ns)) give_up();
            for (int at = max(0, issued - NS); at < issued; ++at)
                if (!mbar_wait_bounded(&sh.kv_full[at % NS], at / NS & 1, p.drain_limit_ns)) give_up();
        }
    } else if (FP8 && warp == 9) {
        if (n > 0) {
            if (lane == 0) {
                const int q_tiles = tiles[1] > 0 ? 2 : 1;
                mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(q_tiles * NB * per * p.G * 128));
                for (int i = 0; i < q_tiles; ++i)
                    for (int c = 0; c < NB; ++c)
                        tma_load_3d(qtile + (i * NB + c) * BLOCK, &qmap, &sh.q_full, c * 64, h * p.G,
                                    b * p.T + t0 + i * per);
            }
            if (!mbar_wait_bounded(&sh.q_full, 0, p.drain_limit_ns)) give_up();
        }
    } else if (FP8 && warp >= 12) {
        // --------------------------------------------- E4M3 codes to f16 tiles
        // Codes are exact in f16; the keys' scale multiplies the scores and the
        // values' scale the weights, as a share of the largest one (vref), so that
        // small scales lose nothing in 16 bits.
        constexpr int CPR = D / 16, RPI = 32 / CPR, IT = 32 / RPI;   // chunks per row, rows per step, steps
        const int cw = warp - 12, chunk = lane % CPR, rsub = lane / CPR;
        float top = 0.f;
        for (int k = tid - 384; k < pages.count; k += 128) {
            const int pg = pages.page(k);
            if (good_page(p, table, pg)) top = fmaxf(top, p.scales[((size_t)table[pg] * p.Hkv + h) * 4 + 1]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) atomicMax(&sh.vref, __float_as_uint(fp8_scale(top)));
        named_barrier_sync(1, 128);
        const float vref = __uint_as_float(*(volatile uint32_t *)&sh.vref);
        const unsigned char *pools[2] = {static_cast<const unsigned char *>(p.k_pool),
                                         static_cast<const unsigned char *>(p.v_pool)};
        // this warp's 32 rows of a tile: one page of 32 or two of 16
        auto look_up = [&](int j, int &phys) {                       // lane x < 2: rows [16 x, 16 x + 16)
            phys = -1;
            const int k = j * ppt + (cw * 32 + (lane & 1) * 16) / p.P;
            if (j < n && k < pages.count) {
                const int t = table[pages.page(k)];
                if (t >= 0 && t < p.num_phys) phys = t;
                else {
                    *(volatile int *)&sh.any_bad = 1;
                    if (p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
                }
            }
        };
        uint4 w[IT];
        auto fetch = [&](int v, int phys_x) {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int r = it * RPI + rsub;                       // row of this warp's 32
                const int phys = __shfl_sync(0xffffffffu, phys_x, r / 16);
                w[it] = make_uint4(0, 0, 0, 0);
                if (phys >= 0)
                    w[it] = ld_global_nc_v4(pools[v] + (((size_t)phys * p.Hkv + h) * p.P + (cw * 32 + r) % p.P) * D + chunk * 16);
            }
        };
        int phys = -1, next = -1;
        look_up(0, phys);
        if (n > 0) fetch(0, phys);
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            look_up(j + 1, next);
            if (lane < 2) {
                float ks = 0.f, vs = 0.f;
                if (phys >= 0) {
                    const float2 a = *reinterpret_cast<const float2 *>(p.scales + ((size_t)phys * p.Hkv + h) * 4);
                    ks = fp8_scale(a.x);
                    vs = vref > 0.f ? fp8_scale(a.y) / vref : 0.f;
                }
                sh.ks[j % kScaleRing][cw * 2 + lane] = ks;
                sh.vs[j % kScaleRing][cw * 2 + lane] = vs;
            }
            for (int v = 0; v < 2; ++v) {
                const int at = 2 * j + v, st = at % NS;
                ok = at < NS || wait(&sh.kv_empty[st], (at / NS - 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int r = cw * 32 + it * RPI + rsub;
                    if (v) {
                        const int k = j * ppt + r / p.P, tok = pages.page(k) * p.P + r % p.P;
                        if (tok > pages.hi || (tok < pages.lo && tok >= p.sinks)) w[it] = make_uint4(0, 0, 0, 0);
                    }
                    uint4 a, c;
                    e4m3x16_to_h(w[it], a, c);
                    unsigned char *row = ring + st * kv_bytes<D>() + (chunk / 4) * BLOCK + r * 128;
                    *reinterpret_cast<uint4 *>(row + (((chunk % 4 * 2) ^ (r & 7)) << 4)) = a;
                    *reinterpret_cast<uint4 *>(row + (((chunk % 4 * 2 + 1) ^ (r & 7)) << 4)) = c;
                }
                fetch(1 - v, v ? next : phys);                       // the tile after this one
                fence_async_smem();
                mbar_arrive(&sh.kv_full[st]);
            }
            phys = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

template <typename T, bool FP8, int D>
cudaError_t launch_t(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, WindowParams p, cudaStream_t stream) {
    auto kernel = window_prompt_kernel<T, FP8, D>;
    constexpr size_t smem = prompt_smem<D>();
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int per = 2 * (kRows / p.G);
    p.row_tiles = (p.T + per - 1) / per;
    const long long blocks = (long long)p.row_tiles * p.B * p.Hkv;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)blocks, FP8 ? 512 : 384, smem, stream>>>(q, k, v, p);
    return cudaGetLastError();
}

}  // namespace

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
