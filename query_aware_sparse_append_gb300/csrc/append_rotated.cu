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
//   KV  one warp per (sequence, touched page, KV head), as the box is one fold
//       over the page's new rows;
//   Q   rows (token, query head) of a sequence spread over the warps, heads
//       fastest, so that neighbouring lane groups read one contiguous span and
//       share a position's table row.
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

template <int EPC>
__device__ __forceinline__ LanePair lane_pair(int j, int rot, int interleaved) {
    LanePair l;
    const int turning = rot / (2 * EPC);   // lanes of a row that rotate
    l.turns = j < turning;
    l.angle = j * EPC;
    if (l.turns && !interleaved) {
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
template <typename T>
__device__ __forceinline__ void rotate(const uint4 &a, const uint4 &b, const Angles<chunk16<T>::n> &t, const LanePair &l,
                                       int interleaved, float *ya, float *yb) {
    constexpr int EPC = chunk16<T>::n;
    chunk16<T>::unpack(a, ya);
    chunk16<T>::unpack(b, yb);
    if (!l.turns) return;
    if (interleaved) {
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

// Q role: kRows rows of every lane group in flight.
template <typename T, int D>
__device__ __forceinline__ void rotate_q(const RotatedParams &p, int b, int block) {
    constexpr int EPC = chunk16<T>::n, LPR = D / (2 * EPC), RPP = 32 / LPR, kRows = 4;
    int L0;
    const int n = new_tokens(p, b, L0, block == 0 && threadIdx.x == 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const LanePair l = lane_pair<EPC>(lane % LPR, p.rot, p.interleaved);
    const long long first = ((long long)block * kWarps + warp) * (RPP * kRows) + lane / LPR;
    const long long rows = (long long)n * p.Hq;
    const T *q = static_cast<const T *>(p.q) + (size_t)b * p.q_batch;
    T *out = static_cast<T *>(p.q_out) + (size_t)b * p.T * p.Hq * D;
    uint4 a[kRows], c[kRows];
    Angles<EPC> t[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long r = first + (long long)u * RPP;
        if (r < rows) {
            const int tok = (int)(r / p.Hq), h = (int)(r % p.Hq);
            const T *row = q + (size_t)tok * p.q_token + (size_t)h * D;
            a[u] = *reinterpret_cast<const uint4 *>(row + l.ca);     // q_out may be q itself: plain loads
            c[u] = *reinterpret_cast<const uint4 *>(row + l.cb);
            load_angles<EPC>(t[u], p, L0 + tok, l);
        }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long r = first + (long long)u * RPP;
        if (r < rows) {
            float ya[EPC], yb[EPC];
            rotate<T>(a[u], c[u], t[u], l, p.interleaved, ya, yb);
            T *row = out + (size_t)r * D;
            *reinterpret_cast<uint4 *>(row + l.ca) = chunk16<T>::pack(ya);
            *reinterpret_cast<uint4 *>(row + l.cb) = chunk16<T>::pack(yb);
        }
    }
}

// A warp's page of the KV role: its tokens, physical page and whether this call
// writes its slot 0.  False where there is nothing to do.
struct PageSpan { int t_lo, t_hi, L0, page0, phys; bool fresh; };

__device__ __forceinline__ bool page_span(const RotatedParams &p, int b, int page, bool report, PageSpan &s) {
    int L0;
    const int n = new_tokens(p, b, L0, report && page == 0);
    const int pi = L0 / p.P + page;
    s.L0 = L0;
    s.page0 = pi * p.P;
    s.t_lo = max(L0, s.page0);
    s.t_hi = min(L0 + n, s.page0 + p.P);
    if (n <= 0 || s.t_lo >= s.t_hi) return false;
    if (pi >= p.max_pages) {
        if (report && p.status) atomicOr(p.status, QASA_DEVERR_SEQ_LEN);
        return false;
    }
    s.phys = p.block_table[(size_t)b * p.max_pages + pi];
    if (s.phys < 0 || s.phys >= p.num_phys) {
        if (report && p.status) atomicOr(p.status, QASA_DEVERR_PAGE_ID);
        return false;
    }
    s.fresh = s.t_lo == s.page0;
    return true;
}

// KV role, pools of the inputs' type.
template <typename T, int D>
__device__ __forceinline__ void append_kv(const RotatedParams &p, int b, int page, int h0) {
    constexpr int EPC = chunk16<T>::n, LPR = D / (2 * EPC), RPP = 32 / LPR;
    PageSpan s;
    if (!page_span(p, b, page, h0 == 0 && threadIdx.x == 0, s)) return;
    const int lane = threadIdx.x & 31, h = h0 + (threadIdx.x >> 5);
    if (h >= p.Hkv) return;
    const int rsub = lane / LPR;
    const LanePair l = lane_pair<EPC>(lane % LPR, p.rot, p.interleaved);
    const T *k = static_cast<const T *>(p.k_new) + (size_t)b * p.k_batch + (size_t)h * D;
    const T *v = static_cast<const T *>(p.v_new) + (size_t)b * p.v_batch + (size_t)h * D;
    const size_t tile = ((size_t)s.phys * p.Hkv + h) * p.P;
    float lo[2 * EPC], hi[2 * EPC];
#pragma unroll
    for (int e = 0; e < 2 * EPC; ++e) { lo[e] = INFINITY; hi[e] = -INFINITY; }
    for (int t = s.t_lo + rsub; t < s.t_hi; t += RPP) {
        const size_t tok = (size_t)(t - s.L0);
        const uint4 ka = ld_global_nc_v4(k + tok * p.k_token + l.ca), kb = ld_global_nc_v4(k + tok * p.k_token + l.cb);
        const uint4 va = ld_global_nc_v4(v + tok * p.v_token + l.ca), vb = ld_global_nc_v4(v + tok * p.v_token + l.cb);
        Angles<EPC> ang;
        load_angles<EPC>(ang, p, t, l);
        const size_t dst = (tile + (t - s.page0)) * D;
        float y[2 * EPC];
        rotate<T>(ka, kb, ang, l, p.interleaved, y, y + EPC);
        const uint4 ra = chunk16<T>::pack(y), rb = chunk16<T>::pack(y + EPC);
        T *kp = static_cast<T *>(p.k_pool) + dst, *vp = static_cast<T *>(p.v_pool) + dst;
        *reinterpret_cast<uint4 *>(kp + l.ca) = ra;
        *reinterpret_cast<uint4 *>(kp + l.cb) = rb;
        *reinterpret_cast<uint4 *>(vp + l.ca) = va;
        *reinterpret_cast<uint4 *>(vp + l.cb) = vb;
        chunk16<T>::unpack(ra, y);          // the box bounds what is stored
        chunk16<T>::unpack(rb, y + EPC);
#pragma unroll
        for (int e = 0; e < 2 * EPC; ++e) { lo[e] = fminf(lo[e], y[e]); hi[e] = fmaxf(hi[e], y[e]); }
    }
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 2 * EPC; ++e) {
            lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], off));
            hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], off));
        }
    if (rsub == 0) {
        T *box = static_cast<T *>(p.bounds) + ((size_t)s.phys * p.Hkv + h) * 2 * D;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c = half ? l.cb : l.ca;
            float *lh = lo + half * EPC, *hh = hi + half * EPC;
            if (!s.fresh) {
                float ol[EPC], oh[EPC];
                chunk16<T>::unpack(*reinterpret_cast<const uint4 *>(box + c), ol);
                chunk16<T>::unpack(*reinterpret_cast<const uint4 *>(box + D + c), oh);
#pragma unroll
                for (int e = 0; e < EPC; ++e) { lh[e] = fminf(lh[e], ol[e]); hh[e] = fmaxf(hh[e], oh[e]); }
            }
            *reinterpret_cast<uint4 *>(box + c) = chunk16<T>::pack(lh);
            *reinterpret_cast<uint4 *>(box + D + c) = chunk16<T>::pack(hh);
        }
    }
}

// Eight codes from / to eight floats.
__device__ __forceinline__ void codes_to_f(const uint2 &w, float *f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e4m3_to_f(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu);
}
__device__ __forceinline__ uint2 f_to_codes(const float *f) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= e4m3_from_f(f[e]) << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

// KV role, E4M3 pools: the page's scale follows the largest |value|, so the new
// rows are read twice (largest value, then codes; the second time from L1), and
// where the scale grows the codes already in the page are re-quantised, all in
// the fp32 steps that qasa_kv_append takes.
template <int D>
__device__ __forceinline__ void append_kv_fp8(const RotatedParams &p, int b, int page, int h0) {
    constexpr int EPC = 8, LPR = D / (2 * EPC), RPP = 32 / LPR;
    PageSpan s;
    if (!page_span(p, b, page, h0 == 0 && threadIdx.x == 0, s)) return;
    const int lane = threadIdx.x & 31, h = h0 + (threadIdx.x >> 5);
    if (h >= p.Hkv) return;
    const int rsub = lane / LPR;
    const LanePair turn = lane_pair<EPC>(lane % LPR, p.rot, p.interleaved);
    const size_t tile = ((size_t)s.phys * p.Hkv + h) * p.P;
    float *sc = p.scales + ((size_t)s.phys * p.Hkv + h) * 4;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {             // 0: K (rotated, with its box), 1: V
        const __half *src = static_cast<const __half *>(kv ? p.v_new : p.k_new) +
                            (size_t)b * (kv ? p.v_batch : p.k_batch) + (size_t)h * D;
        const long long stride = kv ? p.v_token : p.k_token;
        uint8_t *pool = static_cast<uint8_t *>(kv ? p.v_pool : p.k_pool);
        LanePair l = turn;
        if (kv) l.turns = false;                 // V goes in as it is, through the same chunks
        auto values = [&](int t, float *y) {
            const __half *row = src + (size_t)(t - s.L0) * stride;
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row + l.ca));
            const uint4 c = __ldg(reinterpret_cast<const uint4 *>(row + l.cb));
            Angles<EPC> ang;
            load_angles<EPC>(ang, p, t, l);
            rotate<__half>(a, c, ang, l, p.interleaved, y, y + EPC);
        };
        float mx = 0.f;
        for (int t = s.t_lo + rsub; t < s.t_hi; t += RPP) {
            float y[2 * EPC];
            values(t, y);
#pragma unroll
            for (int e = 0; e < 2 * EPC; ++e) mx = fmaxf(mx, fabsf(y[e]));
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float old = s.fresh ? 0.f : sc[kv];
        const float amax = fmaxf(old, mx);
        const float s_old = fp8_scale(old), s_new = fp8_scale(amax);
        const bool requant = !s.fresh && amax > old;
        auto quant = [&](float *y) {
#pragma unroll
            for (int e = 0; e < EPC; ++e) y[e] = s_new == 0.f ? 0.f : __fdiv_rn(y[e], s_new);
        };
        auto requant_codes = [&](const uint2 &w) {
            float y[EPC];
            codes_to_f(w, y);
#pragma unroll
            for (int e = 0; e < EPC; ++e) y[e] = __fmul_rn(y[e], s_old);
            quant(y);
            return f_to_codes(y);
        };
        if (requant)
            for (int t = s.page0 + rsub; t < s.t_lo; t += RPP) {
                uint8_t *row = pool + (tile + (t - s.page0)) * D;
                uint2 *ra = reinterpret_cast<uint2 *>(row + l.ca), *rb = reinterpret_cast<uint2 *>(row + l.cb);
                *ra = requant_codes(*ra);
                *rb = requant_codes(*rb);
            }
        float lo[2 * EPC], hi[2 * EPC];
#pragma unroll
        for (int e = 0; e < 2 * EPC; ++e) { lo[e] = INFINITY; hi[e] = -INFINITY; }
        for (int t = s.t_lo + rsub; t < s.t_hi; t += RPP) {
            float y[2 * EPC];
            values(t, y);
            quant(y);
            quant(y + EPC);
            const uint2 a = f_to_codes(y), c = f_to_codes(y + EPC);
            uint8_t *row = pool + (tile + (t - s.page0)) * D;
            *reinterpret_cast<uint2 *>(row + l.ca) = a;
            *reinterpret_cast<uint2 *>(row + l.cb) = c;
            if (kv == 0) {
                codes_to_f(a, y);
                codes_to_f(c, y + EPC);
#pragma unroll
                for (int e = 0; e < 2 * EPC; ++e) { lo[e] = fminf(lo[e], y[e]); hi[e] = fmaxf(hi[e], y[e]); }
            }
        }
        if (kv == 0) {
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
                for (int e = 0; e < 2 * EPC; ++e) {
                    lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], off));
                    hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], off));
                }
            if (rsub == 0) {
                uint8_t *box = static_cast<uint8_t *>(p.bounds) + ((size_t)s.phys * p.Hkv + h) * 2 * D;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint8_t *bc = box + (half ? l.cb : l.ca);
                    float *lh = lo + half * EPC, *hh = hi + half * EPC;
                    if (!s.fresh) {
                        uint2 wl = *reinterpret_cast<const uint2 *>(bc), wh = *reinterpret_cast<const uint2 *>(bc + D);
                        if (requant) { wl = requant_codes(wl); wh = requant_codes(wh); }
                        float ol[EPC], oh[EPC];
                        codes_to_f(wl, ol);
                        codes_to_f(wh, oh);
#pragma unroll
                        for (int e = 0; e < EPC; ++e) { lh[e] = fminf(lh[e], ol[e]); hh[e] = fmaxf(hh[e], oh[e]); }
                    }
                    *reinterpret_cast<uint2 *>(bc) = f_to_codes(lh);     // exact: codes' own values
                    *reinterpret_cast<uint2 *>(bc + D) = f_to_codes(hh);
                }
            }
        }
        __syncwarp();
        if (lane == 0) sc[kv] = amax;
    }
}

// T: the type of q and of the new rows; FP8: E4M3 pools.
template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(32 * kWarps) append_rotated_kernel(RotatedParams p) {
    const int b = blockIdx.y, x = blockIdx.x;
    if (x < p.kv_blocks) {
        const int per_page = (p.Hkv + kWarps - 1) / kWarps;
        if constexpr (FP8) append_kv_fp8<D>(p, b, x / per_page, x % per_page * kWarps);
        else append_kv<T, D>(p, b, x / per_page, x % per_page * kWarps);
    } else {
        rotate_q<T, D>(p, b, x - p.kv_blocks);
    }
}

template <typename T, int D, bool FP8>
cudaError_t launch_t(RotatedParams p, int batch, cudaStream_t stream) {
    constexpr int rows_per_block = kWarps * 4 * (32 / (D / (2 * chunk16<T>::n)));
    const long long pages = ((long long)p.T + p.P - 2) / p.P + 1;   // the most that T tokens touch
    const long long kv = pages * ((p.Hkv + kWarps - 1) / kWarps);
    const long long q = p.q ? ((long long)p.T * p.Hq + rows_per_block - 1) / rows_per_block : 0;
    if (kv + q > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.kv_blocks = (int)kv;
    append_rotated_kernel<T, D, FP8><<<dim3((unsigned)(kv + q), batch), 32 * kWarps, 0, stream>>>(p);
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
