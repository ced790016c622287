// append_rotated.cu -- kv append with the position rotation applied on the way.
//
// One call takes the raw queries, keys and values of the new tokens (rows of one
// projection's output, any batch and token stride), rotates the channel pairs of
// q and k by their position's angles, writes k and v into their pages and q into
// its own buffer, and keeps the page boxes (and, for E4M3 pages, the scales)
// current exactly as qasa_kv_append does for keys rotated beforehand:
//     y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin        (fp32)
// with (cos, sin) of (position, pair) read from the caller's fp32 table.  A
// rotated value is rounded once, to the cache's type (16-bit pools, q) or to the
// page's E4M3 code; the box folds the stored value, so that it bounds what the
// pool holds.
//
// Two roles share a launch, told apart by blockIdx.x:
//   KV  one warp per (sequence, touched page, KV head, K or V), as the box and the
//       scale are one fold over the page's new rows (four warps to a page's rows were
//       slower, 28.9 against 18.7 us for the K and V of 2 x 4096 tokens: the chain of
//       loads before the rows is what a warp spends its time on);
//   Q   one warp per (token, span of query heads): the token's angles are read once,
//       and neighbouring lane groups read neighbouring heads, one contiguous span.
// It is bound by the rows' traffic for prompts (each read and written once), and by
// the chain length -> block table -> page for a decode step, so every warp has all
// its loads under way at once.
// In both a lane holds two 16-byte chunks of a row that rotate with each other:
// chunks (j, j + R/2) for half-split pairs, chunks (2j, 2j + 1) for neighbouring
// pairs; either way its angles are entries [j * EPC, (j + 1) * EPC) of the table
// row, so one addressing rule serves both.
#include "qasa_device.cuh"
#include "qasa_launch.h"

namespace qasa {

namespace {

constexpr int kWarps = 4;

// What a lane does with a row: its two chunks and whether they rotate.
struct LanePair {
    int ca, cb;      // first channels of the two chunks
    int angle;       // first entry of the table row
    bool turns;
};

template <int EPC, bool INTER>
__device__ __forceinline__ LanePair lane_pair(int j, int rot) {
    LanePair l;
    const int turning = rot / (2 * EPC);   // lanes of a row that rotate
    l.turns = j < turning;
    l.angle = j * EPC;
    if (l.turns && !INTER) {
        l.ca = j * EPC;
        l.cb = l.ca + rot / 2;
    } else {   // neighbouring chunks; past the rotated channels in both forms
        l.ca = 2 * j * EPC;
        l.cb = l.ca + EPC;
    }
    return l;
}

template <int EPC> struct Angles { float c[EPC], s[EPC]; };

template <int EPC>
__device__ __forceinline__ void load_angles(Angles<EPC> &a, const RotatedParams &p, int pos, const LanePair &l) {
    if (!l.turns) return;
    const float *row = p.table + (size_t)pos * p.rot + l.angle;
#pragma unroll
    for (int e = 0; e < EPC; e += 4) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(row + e));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(row + p.rot / 2 + e));
        a.c[e] = c.x; a.c[e + 1] = c.y; a.c[e + 2] = c.z; a.c[e + 3] = c.w;
        a.s[e] = s.x; a.s[e + 1] = s.y; a.s[e + 2] = s.z; a.s[e + 3] = s.w;
    }
}

// The two chunks' values, rotated where the lane's channels rotate.
template <typename T, bool INTER>
__device__ __forceinline__ void rotate(const uint4 &a, const uint4 &b, const Angles<chunk16<T>::n> &t, const LanePair &l,
                                       float *ya, float *yb) {
    constexpr int EPC = chunk16<T>::n;
    chunk16<T>::unpack(a, ya);
    chunk16<T>::unpack(b, yb);
    if (!l.turns) return;
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < EPC; e += 2) {
            const float a0 = ya[e], a1 = ya[e + 1], b0 = yb[e], b1 = yb[e + 1];
            const int i = e / 2, k = EPC / 2 + e / 2;
            ya[e] = fmaf(a0, t.c[i], -(a1 * t.s[i]));
            ya[e + 1] = fmaf(a1, t.c[i], a0 * t.s[i]);
            yb[e] = fmaf(b0, t.c[k], -(b1 * t.s[k]));
            yb[e + 1] = fmaf(b1, t.c[k], b0 * t.s[k]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
            const float x = ya[e], y = yb[e];
            ya[e] = fmaf(x, t.c[e], -(y * t.s[e]));
            yb[e] = fmaf(y, t.c[e], x * t.s[e]);
        }
    }
}

// The new tokens of sequence b that this call can place: positions L0 .. L0 + n.
// `report`: this thread records what is wrong with the sequence.
__device__ __forceinline__ int new_tokens(const RotatedParams &p, int b, int &L0, bool report) {
    L0 = p.seq_lens[b];
    int n = p.append_lens ? p.append_lens[b] : p.T, err = 0;
    if (n < 0 || n > p.T) { err |= QASA_DEVERR_APPEND; n = n < 0 ? 0 : p.T; }
    if (L0 < 0) { err |= QASA_DEVERR_SEQ_LEN; n = 0; }
    if (n > p.max_positions - L0) {      // also keeps L0 + n inside 32 bits
        if (n > 0) err |= QASA_DEVERR_POSITION;
        n = max(0, p.max_positions - L0);
    }
    if (err && report && p.status) atomicOr(p.status, err);
    return n;
}

constexpr int kBatch = 4;      // rows of every lane group under way

// Q role.  Task = (token, span of p.q_span head batches).
template <typename T, int D, bool INTER>
__device__ __forceinline__ void rotate_q(const RotatedParams &p, int b, int block) {
    constexpr int EPC = chunk16<T>::n, LPR = D / (2 * EPC), RPP = 32 / LPR;
    const int lane = threadIdx.x & 31, task = block * kWarps + (threadIdx.x >> 5);
    const int batches = (p.Hq + RPP * kBatch - 1) / (RPP * kBatch), spans = (batches + p.q_span - 1) / p.q_span;
    const int tok = task / spans, first = task % spans * p.q_span;
    if (tok >= p.T) return;
    const LanePair l = lane_pair<EPC, INTER>(lane % LPR, p.rot);
    const T *q = static_cast<const T *>(p.q) + (size_t)b * p.q_batch + (size_t)tok * p.q_token;
    T *out = static_cast<T *>(p.q_out) + ((size_t)b * p.T + tok) * p.Hq * D;
    uint4 a[kBatch], c[kBatch];
    auto fetch = [&](int batch) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = (batch * kBatch + u) * RPP + lane / LPR;
            if (h < p.Hq) {                    // q_out may be q itself: plain loads
                a[u] = *reinterpret_cast<const uint4 *>(q + (size_t)h * D + l.ca);
                c[u] = *reinterpret_cast<const uint4 *>(q + (size_t)h * D + l.cb);
            }
        }
    };
    // a token past the count is in the caller's memory all the same: where few can be,
    // the rows do not wait for the counts
    const bool early = !p.append_lens || p.T <= 8;
    if (early) fetch(first);
    int L0;
    const int n = new_tokens(p, b, L0, block == 0 && threadIdx.x == 0);
    if (tok >= n) return;
    if (!early) fetch(first);
    Angles<EPC> t;
    load_angles<EPC>(t, p, L0 + tok, l);
    const int last = min(first + p.q_span, batches);
    for (int batch = first; batch < last; ++batch) {
        if (batch > first) fetch(batch);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = (batch * kBatch + u) * RPP + lane / LPR;
            if (h < p.Hq) {
                float ya[EPC], yb[EPC];
                rotate<T, INTER>(a[u], c[u], t, l, ya, yb);
                *reinterpret_cast<uint4 *>(out + (size_t)h * D + l.ca) = chunk16<T>::pack(ya);
                *reinterpret_cast<uint4 *>(out + (size_t)h * D + l.cb) = chunk16<T>::pack(yb);
            }
        }
    }
}

// A warp's page of the KV role: its tokens, and whether this call writes its slot
// 0.  False where there is nothing to do.
struct PageSpan { int t_lo, t_hi, L0, page0, logical; bool fresh; };

__device__ __forceinline__ bool page_span(const RotatedParams &p, int b, int page, bool report, PageSpan &s) {
    const int n = new_tokens(p, b, s.L0, report && page == 0);
    s.logical = s.L0 / p.P + page;
    s.page0 = s.logical * p.P;
    s.t_lo = max(s.L0, s.page0);
    s.t_hi = min(s.L0 + n, s.page0 + p.P);
    s.fresh = s.t_lo == s.page0;
    return n > 0 && s.t_lo < s.t_hi;
}

// Its physical page, or -1; asked for after the rows, which do not wait for it.
__device__ __forceinline__ int physical_page(const RotatedParams &p, int b, const PageSpan &s, bool report) {
    int phys = -1, err = QASA_DEVERR_SEQ_LEN;
    if (s.logical < p.max_pages) {
        phys = p.block_table[(size_t)b * p.max_pages + s.logical];
        err = QASA_DEVERR_PAGE_ID;
        if (phys >= 0 && phys < p.num_phys) return phys;
    }
    if (report && p.status) atomicOr(p.status, err);
    return -1;
}

// One warp's task of the KV role: K (0) or V (1) of head h.  False for none.
__device__ __forceinline__ bool kv_task(const RotatedParams &p, int block, int &h, int &which) {
    const int task = block * kWarps + (threadIdx.x >> 5);
    h = task >> 1;
    which = task & 1;
    return h < p.Hkv;
}

// Minima and maxima of the stored keys of a lane's chunk pair, in the pool's own
// type (exact, and half the registers of fp32 for 16-bit pools; E4M3 codes go as
// halves).  A number wins over a NaN, as in the other box code.
template <typename T> struct Box {
    static constexpr int N = 8;                  // words of a chunk pair
    uint32_t lo[N], hi[N];
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (sizeof(T) == 4) r = __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
        else if constexpr (elem<T>::id == QASA_DTYPE_BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (sizeof(T) == 4) r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        else if constexpr (elem<T>::id == QASA_DTYPE_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ void clear() {
        const uint32_t inf = sizeof(T) == 4 ? 0x7f800000u : elem<T>::id == QASA_DTYPE_BF16 ? 0x7f807f80u : 0x7c007c00u;
        const uint32_t minus = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
#pragma unroll
        for (int i = 0; i < N; ++i) { lo[i] = inf; hi[i] = inf | minus; }
    }
    __device__ __forceinline__ void fold(const uint4 &a, const uint4 &b) {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < N; ++i) { lo[i] = least(lo[i], w[i]); hi[i] = most(hi[i], w[i]); }
    }
    template <int LPR> __device__ __forceinline__ void join() {      // the warp's lane groups
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                lo[i] = least(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
                hi[i] = most(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
            }
    }
};

// KV role, pools of the inputs' type.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void append_kv(const RotatedParams &p, int b, int page, int block) {
    constexpr int EPC = chunk16<T>::n, LPR = D / (2 * EPC), RPP = 32 / LPR;
    PageSpan s;
    int h, which;
    if (!page_span(p, b, page, block == 0 && threadIdx.x == 0, s) || !kv_task(p, block, h, which)) return;
    const int lane = threadIdx.x & 31, mine = s.t_lo + lane / LPR;
    const LanePair l = lane_pair<EPC, INTER>(lane % LPR, p.rot);
    const T *src = (which ? static_cast<const T *>(p.v_new) + (size_t)b * p.v_batch
                          : static_cast<const T *>(p.k_new) + (size_t)b * p.k_batch) + (size_t)h * D;
    const long long stride = which ? p.v_token : p.k_token;
    uint4 a[kBatch], c[kBatch];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int t = t0 + u * RPP;
            if (t < s.t_hi) {
                const T *row = src + (size_t)(t - s.L0) * stride;
                a[u] = ld_global_nc_v4(row + l.ca);
                c[u] = ld_global_nc_v4(row + l.cb);
            }
        }
    };
    fetch(mine);
    const int phys = physical_page(p, b, s, block == 0 && threadIdx.x == 0);
    if (phys < 0) return;
    T *dst = static_cast<T *>(which ? p.v_pool : p.k_pool) + ((size_t)phys * p.Hkv + h) * p.P * D;
    Box<T> box;
    box.clear();
    for (int t0 = mine; t0 < s.t_hi; t0 += RPP * kBatch) {
        if (t0 > mine) fetch(t0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int t = t0 + u * RPP;
            if (t >= s.t_hi) continue;
            if (!which) {
                Angles<EPC> ang;
                load_angles<EPC>(ang, p, t, l);
                float y[2 * EPC];
                rotate<T, INTER>(a[u], c[u], ang, l, y, y + EPC);
                a[u] = chunk16<T>::pack(y);
                c[u] = chunk16<T>::pack(y + EPC);
                box.fold(a[u], c[u]);            // the box bounds what is stored
            }
            T *row = dst + (size_t)(t - s.page0) * D;
            *reinterpret_cast<uint4 *>(row + l.ca) = a[u];
            *reinterpret_cast<uint4 *>(row + l.cb) = c[u];
        }
    }
    if (which) return;
    box.template join<LPR>();
    if (lane < LPR) {
        T *row = static_cast<T *>(p.bounds) + ((size_t)phys * p.Hkv + h) * 2 * D;
        uint4 *la = reinterpret_cast<uint4 *>(row + l.ca), *lb = reinterpret_cast<uint4 *>(row + l.cb);
        uint4 *ha = reinterpret_cast<uint4 *>(row + D + l.ca), *hb = reinterpret_cast<uint4 *>(row + D + l.cb);
        if (!s.fresh) {
            box.fold(*la, *lb);
            box.fold(*ha, *hb);
        }
        *la = make_uint4(box.lo[0], box.lo[1], box.lo[2], box.lo[3]);
        *lb = make_uint4(box.lo[4], box.lo[5], box.lo[6], box.lo[7]);
        *ha = make_uint4(box.hi[0], box.hi[1], box.hi[2], box.hi[3]);
        *hb = make_uint4(box.hi[4], box.hi[5], box.hi[6], box.hi[7]);
    }
}

// Eight floats from eight codes.
__device__ __forceinline__ void codes_to_f(const uint2 &w, float *f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e4m3_to_f(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu);
}
// Two codes (low byte first), ties to even, saturating.
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(lo), "f"(hi));
    return c;
}
// Codes of y / s, the quotient rounded to fp32 as everywhere, eight at a time.
__device__ __noinline__ uint2 quantise8_exact(float4 a, float4 b, float s) {
    const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[2] = {0u, 0u};
    if (s > 0.f)
#pragma unroll
        for (int e = 0; e < 8; e += 2) w[e >> 2] |= code2(__fdiv_rn(y[e], s), __fdiv_rn(y[e + 1], s)) << (8 * (e & 2));
    return make_uint2(w[0], w[1]);
}
// The division is needed only where a code border lies near: the product with the
// reciprocal `inv` is within 2^-22 of the quotient (half a step each for the
// reciprocal, the product and the quotient), so where products scaled by 1 - 2^-21
// and 1 + 2^-21 have the same code, the quotient has it too.  The exact way is out
// of line: the kernel's rows run into the instruction cache's size otherwise.
__device__ __forceinline__ uint2 quantise8(const float *y, float s, float inv) {
    uint32_t w[2] = {0u, 0u};
    bool same = inv < INFINITY;                // a scale of 0, or one whose reciprocal is too large
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float a = y[e] * inv, b = y[e + 1] * inv;
        const uint32_t in = code2(a * (1.f - 0x1p-21f), b * (1.f - 0x1p-21f));
        const uint32_t out = code2(a * (1.f + 0x1p-21f), b * (1.f + 0x1p-21f));
        same = same && in == out;
        w[e >> 2] |= out << (8 * (e & 2));
    }
    if (!same) {
        const uint2 x = quantise8_exact(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), s);
        w[0] = x.x;
        w[1] = x.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] &= ((w[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // zero is +0
    return make_uint2(w[0], w[1]);
}

// Eight codes as halves, exactly, and back (halves that are codes' values).
__device__ __forceinline__ uint4 codes_to_halves(const uint2 &w) {
    return make_uint4(e4m3x2_to_h2(w.x), e4m3x2_to_h2(w.x >> 16), e4m3x2_to_h2(w.y), e4m3x2_to_h2(w.y >> 16));
}
__device__ __forceinline__ uint2 halves_to_codes(const uint32_t *h) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h[i]));
        w[i >> 1] |= (uint32_t)c << (16 * (i & 1));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] &= ((w[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // zero is +0
    return make_uint2(w[0], w[1]);
}

// KV role, E4M3 pools: the page's scale follows the largest |value|, so the new
// rows are gone through twice (largest value, then codes); where they fit they stay
// in registers in between.  Where the scale grows the codes already in the page are
// re-quantised, all in the fp32 steps that qasa_kv_append takes.
template <int D, bool INTER>
__device__ __forceinline__ void append_kv_fp8(const RotatedParams &p, int b, int page, int block) {
    constexpr int EPC = 8, LPR = D / (2 * EPC), RPP = 32 / LPR;
    PageSpan s;
    int h, which;
    if (!page_span(p, b, page, block == 0 && threadIdx.x == 0, s) || !kv_task(p, block, h, which)) return;
    const int lane = threadIdx.x & 31, mine = s.t_lo + lane / LPR;
    LanePair l = lane_pair<EPC, INTER>(lane % LPR, p.rot);
    if (which) l.turns = false;                  // V goes in as it is, through the same chunks
    const __half *src = (which ? static_cast<const __half *>(p.v_new) + (size_t)b * p.v_batch
                               : static_cast<const __half *>(p.k_new) + (size_t)b * p.k_batch) + (size_t)h * D;
    const long long stride = which ? p.v_token : p.k_token;
    uint4 a[kBatch], c[kBatch];                  // rows as they came, one chunk pair per lane
    auto fetch = [&](int t0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int t = t0 + u * RPP;
            if (t < s.t_hi) {
                const __half *row = src + (size_t)(t - s.L0) * stride;
                a[u] = __ldg(reinterpret_cast<const uint4 *>(row + l.ca));
                c[u] = __ldg(reinterpret_cast<const uint4 *>(row + l.cb));
            }
        }
    };
    auto values = [&](int u, int t, float *y) {
        Angles<EPC> ang;
        load_angles<EPC>(ang, p, t, l);
        rotate<__half, INTER>(a[u], c[u], ang, l, y, y + EPC);
    };
    fetch(mine);
    const int phys = physical_page(p, b, s, block == 0 && threadIdx.x == 0);
    if (phys < 0) return;
    uint8_t *pool = static_cast<uint8_t *>(which ? p.v_pool : p.k_pool) + ((size_t)phys * p.Hkv + h) * p.P * D;
    float *sc = p.scales + ((size_t)phys * p.Hkv + h) * 4 + which;
    const float old = s.fresh ? 0.f : *sc;
    float mx = 0.f;
    for (int t0 = mine; t0 < s.t_hi; t0 += RPP * kBatch) {
        if (t0 > mine) fetch(t0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (t0 + u * RPP < s.t_hi) {
                float y[2 * EPC];
                values(u, t0 + u * RPP, y);
#pragma unroll
                for (int e = 0; e < 2 * EPC; ++e) mx = fmaxf(mx, fabsf(y[e]));
            }
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float amax = fmaxf(old, mx);
    const float s_old = fp8_scale(old), s_new = fp8_scale(amax), inv = 1.f / s_new;
    const bool requant = !s.fresh && amax > old;
    auto requant_codes = [&](const uint2 &w) {
        float v[EPC];
        codes_to_f(w, v);
#pragma unroll
        for (int e = 0; e < EPC; ++e) v[e] = __fmul_rn(v[e], s_old);
        return quantise8(v, s_new, inv);
    };
    if (requant)
#pragma unroll 1
        for (int t = s.page0 + lane / LPR; t < s.t_lo; t += RPP) {
            uint8_t *row = pool + (size_t)(t - s.page0) * D;
            uint2 *ra = reinterpret_cast<uint2 *>(row + l.ca), *rb = reinterpret_cast<uint2 *>(row + l.cb);
            *ra = requant_codes(*ra);
            *rb = requant_codes(*rb);
        }
    const bool once = s.t_hi - s.t_lo <= RPP * kBatch;
    Box<__half> box;
    box.clear();
    for (int t0 = mine; t0 < s.t_hi; t0 += RPP * kBatch) {
        if (!once) fetch(t0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int t = t0 + u * RPP;
            if (t >= s.t_hi) continue;
            uint8_t *row = pool + (size_t)(t - s.page0) * D;
            float y[2 * EPC];
            values(u, t, y);
            const uint2 qa = quantise8(y, s_new, inv), qb = quantise8(y + EPC, s_new, inv);
            *reinterpret_cast<uint2 *>(row + l.ca) = qa;
            *reinterpret_cast<uint2 *>(row + l.cb) = qb;
            if (!which) box.fold(codes_to_halves(qa), codes_to_halves(qb));
        }
    }
    if (!which) {
        box.template join<LPR>();
        if (lane < LPR) {
            uint8_t *row = static_cast<uint8_t *>(p.bounds) + ((size_t)phys * p.Hkv + h) * 2 * D;
#pragma unroll 1
            for (int side = 0; side < 2 && !s.fresh; ++side) {        // the old box, under the new scale
                uint2 oa = *reinterpret_cast<const uint2 *>(row + side * D + l.ca);
                uint2 ob = *reinterpret_cast<const uint2 *>(row + side * D + l.cb);
                if (requant) { oa = requant_codes(oa); ob = requant_codes(ob); }
                box.fold(codes_to_halves(oa), codes_to_halves(ob));
            }
            *reinterpret_cast<uint2 *>(row + l.ca) = halves_to_codes(box.lo);
            *reinterpret_cast<uint2 *>(row + l.cb) = halves_to_codes(box.lo + 4);
            *reinterpret_cast<uint2 *>(row + D + l.ca) = halves_to_codes(box.hi);
            *reinterpret_cast<uint2 *>(row + D + l.cb) = halves_to_codes(box.hi + 4);
        }
    }
    if (lane == 0) *sc = amax;
}

// T: the type of q and of the new rows; FP8: E4M3 pools.
template <typename T, int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(32 * kWarps, 5) append_rotated_kernel(RotatedParams p) {
    const int b = blockIdx.y, x = blockIdx.x;
    if (x < p.kv_blocks) {
        const int per_page = (2 * p.Hkv + kWarps - 1) / kWarps;
        if constexpr (FP8) append_kv_fp8<D, INTER>(p, b, x / per_page, x % per_page);
        else append_kv<T, D, INTER>(p, b, x / per_page, x % per_page);
    } else {
        rotate_q<T, D, INTER>(p, b, x - p.kv_blocks);
    }
}

template <typename T, int D, bool FP8>
cudaError_t launch_t(RotatedParams p, int batch, cudaStream_t stream) {
    constexpr int RPP = 32 / (D / (2 * chunk16<T>::n));
    const long long pages = ((long long)p.T + p.P - 2) / p.P + 1;   // the most that T tokens touch
    const long long kv = pages * ((2 * p.Hkv + kWarps - 1) / kWarps);
    // A warp of the Q role takes one batch of heads.  Counts may leave tokens out, whose
    // warps only come and go: from 12 warps to a quarter of an SM on (which holds five at
    // a time) it then takes more, up to a whole token.  E4M3, counts between 1 and T,
    // with a batch each and with a token: 16 x 1024 tokens of 32 heads 37.0 and 33.7 us,
    // 8 x 1024 20.7 and 19.1, 16 x 512 of 64 heads 45.0 and 41.1 (a limit of 24 misses
    // the second, one of 6 is level).  Without counts a token to a warp gives nothing:
    // 2 x 4096 bf16 tokens 34.9 and 35.3 us, 1 x 1024 of 64 heads 8.8 and 9.5.
    const long long batches = (p.Hq + RPP * kBatch - 1) / (RPP * kBatch);
    const long long spread = p.append_lens ? batches * p.T * batch / (12LL * 4 * p.sms) : 1;
    p.q_span = (int)(spread < 1 ? 1 : spread < batches ? spread : batches > 0 ? batches : 1);
    const long long q = p.q ? ((batches + p.q_span - 1) / p.q_span * p.T + kWarps - 1) / kWarps : 0;
    if (kv + q > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.kv_blocks = (int)kv;
    (p.interleaved ? append_rotated_kernel<T, D, FP8, true> : append_rotated_kernel<T, D, FP8, false>)
        <<<dim3((unsigned)(kv + q), batch), 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rotated(qasa_dtype dt, int D, const RotatedParams &p, int batch, cudaStream_t stream) {
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
