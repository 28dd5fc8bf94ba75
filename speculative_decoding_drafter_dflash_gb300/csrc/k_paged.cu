// Paged 4-bit KV cache: append of new rows (per-head norms, rotary positions and quantisation in
// one pass) and gather of cached rows.
#include "paged.cuh"

namespace df {

namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendMaxTokens = 4;          // tokens of one CTA
constexpr int kAppendMaxHalf = 128;          // rotary pairs (rotary_dim <= 256)

// Bound of the F32 error of a normed and rotated value a cos - b sin, in units of |a| + |b|: the
// sum of squares (d / 32 + 5 roundings on the longest path, halved by the root: 7), root and
// reciprocal (2), the two products (2), cos and sin (an angle within 1.5 units, 2 of the
// functions), the rotation (2), 16.5 in all; 20 units of 2^-24 are taken.
constexpr float kRotErr = 20.f * 5.9604645e-8f;
// Relative error of the divisions by 6 and by the scale in the fast path, with room.
constexpr float kDivErr = 2.3841858e-7f;

// E4M3 value nearest to v >= 0, ties to even (v may be infinite).
__device__ double e4m3_nearest(double v) {
    if (v >= 448.0) return 448.0;
    int e = v > 0.0 ? ilogb(v) : -6;
    e = e < -6 ? -6 : e;
    const double s = rint(ldexp(v, 3 - e));
    return fmin(ldexp(s, e - 3), 448.0);
}

// The same decisions as the fast path's, in float64: for rows where a value's F32 error band
// crosses a boundary. About one row in a thousand comes here, so its cost is not the kernel's.
template <int EPL>
__device__ __noinline__ void quantise_f64(const float *x, const float *w, bool norm, float eps,
                                          int half, long long pos0, const double *inv_freq,
                                          const int32_t *positions, size_t pos_stride,
                                          const uint8_t *axis, int n_axes, double inv_scale,
                                          uint32_t &codes, uint32_t &scale_byte) {
    constexpr int D = 32 * EPL, LPB = 16 / EPL;
    const int lane = threadIdx.x & 31;
    double y[EPL];
    double r = 1.0;
    if (norm) {
        double ss = 0.0;
        for (int u = 0; u < EPL; ++u) ss += (double)x[u] * (double)x[u];
        for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        r = 1.0 / sqrt(ss / D + (double)eps);
    }
    for (int u = 0; u < EPL; ++u) y[u] = (double)x[u] * r * (double)w[u];
    if (half > 0) {
        const int step = half / EPL, e0 = lane * EPL;
        const int src = e0 < half ? lane + step : (e0 < 2 * half ? lane - step : lane);
        for (int u = 0; u < EPL; ++u) {
            const double other = __shfl_sync(0xffffffffu, y[u], src);
            if (e0 < 2 * half) {
                const int p = (e0 < half ? e0 : e0 - half) + u;
                long long pos = pos0;
                if (positions) {
                    int ax = axis ? axis[p] : 0;
                    if (ax >= n_axes) ax = 0;
                    pos = positions[(size_t)ax * pos_stride];
                }
                double sn, cs;
                sincos((double)pos * inv_freq[p], &sn, &cs);
                y[u] = e0 < half ? y[u] * cs - other * sn : y[u] * cs + other * sn;
            }
        }
    }
    double amax = 0.0;
    for (int u = 0; u < EPL; ++u) {
        y[u] = isnan(y[u]) ? 0.0 : fmin(fmax(y[u] * inv_scale, -3.0e38), 3.0e38);
        amax = fmax(amax, fabs(y[u]));
    }
    for (int m = LPB / 2; m >= 1; m >>= 1) amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const double s = e4m3_nearest(amax / 6.0);
    scale_byte = f32x2_to_e4m3((float)s, 0.f) & 0xff;
    codes = 0;
    for (int u = 0; u < EPL; ++u) {
        double c = s > 0.0 ? fabs(y[u]) / s : 0.0;
        const double step = c < 2.0 ? 0.5 : (c < 4.0 ? 1.0 : 2.0);
        c = fmin(rint(c / step) * step, 6.0);
        codes |= (f32x2_to_e2m1((float)copysign(c, y[u]), 0.f) & 0xf) << (4 * u);
    }
}

// One warp per (token, head slot): q heads, then k heads, then v heads. A lane holds EPL = d / 32
// consecutive dims, so a block of 16 is 16 / EPL lanes and the partner of a rotary pair is the
// same element of another lane (rotary_dim is a multiple of 16, so half of it is one of EPL).
// The CTA first takes the cosine and sine of its tokens' angles into shared memory, where the
// q and k heads share them. An angle is position * inv_freq reduced to a turn: inv_freq / 2 pi as
// a 64-bit fixed-point fraction times the position, modulo 2^64, which is exact up to the
// fraction's own 2^-53 and takes integer multiplies instead of GB300's slow FP64; only the top
// 32 bits of the turn enter cos and sin.
//
// Bound: the F32 rows read and written (at 16 q and 8 KV heads of 128 dims, 24 KB a token; the
// cache adds 1.2 KB). A code is decided twice, at both ends of the value's F32 error band; where
// the two differ the row is taken again in float64 (quantise_f64), so the codes are those of the
// real-number definition.
template <int EPL>
__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_append_kernel(const __grid_constant__ KvAppendArgs a, int tokens_per_cta, int slots_per_cta) {
    DF_TRACE_KERNEL(TK_KV_APPEND);
    constexpr int D = 32 * EPL, LPB = 16 / EPL;
    constexpr int U = EPL == 8 ? 2 : 4;      // rows of a warp loaded together
    __shared__ unsigned long long freq[kAppendMaxHalf];
    __shared__ float2 cs[kAppendMaxTokens][kAppendMaxHalf];
    __shared__ int4 tok[kAppendMaxTokens];   // sequence, row index i (-1: none), first row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = a.rope.rotary_dim / 2, nkv = a.c.n_kv_heads, nq = a.nq;
    const int total = a.c.batch * a.n_max;
    const int t0 = blockIdx.x * tokens_per_cta;
    const int nt = min(tokens_per_cta, total - t0);
    const int slots = nq + 2 * nkv;
    const int s0 = blockIdx.y * slots_per_cta, ns = min(slots_per_cta, slots - s0);
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < nt) {
        const int t = t0 + threadIdx.x, b = t / a.n_max, i = t - b * a.n_max;
        int n = a.n_new ? a.n_new[b] : a.n_max;
        if (n < 0 || n > a.n_max) {
            set_status(a.status, DF_ESHAPE);
            n = min(max(n, 0), a.n_max);
        }
        const int len = a.c.seq_len[b];
        if (len < 0) set_status(a.status, DF_ECAPACITY);
        tok[threadIdx.x] = make_int4(b, i < n ? i : -1, len, 0);
    }
    if (threadIdx.x < half) {
        double f = a.rope.inv_freq[threadIdx.x] * 0.15915494309189533577;
        f -= floor(f);
        // f in [0, 1]; 2^64 f stays below 2^64 because f = 1 - 2^-53 at most
        freq[threadIdx.x] = f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
    }
    __syncthreads();
    if (s0 < nq + nkv) {
        for (int x = threadIdx.x; x < nt * half; x += blockDim.x) {
            const int j = x / half, p = x - j * half;
            const int4 tk = tok[j];
            if (tk.y < 0) continue;
            long long pos = (long long)tk.z + tk.y;
            if (a.rope.positions) {
                int ax = a.rope.axis ? a.rope.axis[p] : 0;
                if (ax >= a.rope.n_axes) {
                    set_status(a.status, DF_EINVAL);
                    ax = 0;
                }
                pos = a.rope.positions[(size_t)ax * total + t0 + j];
            }
            const unsigned long long turn = (unsigned long long)pos * freq[p];
            float sn, c;
            sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &sn, &c);
            cs[j][p] = make_float2(c, sn);
        }
    }
    __syncthreads();

    const int tasks = nt * ns;
    for (int base = 0; base < tasks; base += kAppendWarps * U) {
        float x[U][EPL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int task = base + u * kAppendWarps + warp;
            const int j = min(task, tasks - 1) / ns, slot = s0 + min(task, tasks - 1) - j * ns;
            const size_t row = t0 + j;
            if (task >= tasks || tok[j].y < 0) continue;
            const float *src = slot < nq ? a.q + row * a.ldq + slot * D
                               : slot < nq + nkv ? a.k + row * a.ldk + (slot - nq) * D
                                                 : a.v + row * a.ldv + (slot - nq - nkv) * D;
            src += lane * EPL;
            if constexpr (EPL == 2) {
                const float2 f = *reinterpret_cast<const float2 *>(src);
                x[u][0] = f.x, x[u][1] = f.y;
            } else {
#pragma unroll
                for (int e = 0; e < EPL; e += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + e);
                    x[u][e] = f.x, x[u][e + 1] = f.y, x[u][e + 2] = f.z, x[u][e + 3] = f.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int task = base + u * kAppendWarps + warp;
            if (task >= tasks) break;
            const int j = task / ns, slot = s0 + task - j * ns;
            const int4 tk = tok[j];
            if (tk.y < 0) continue;
            const bool is_q = slot < nq, is_v = slot >= nq + nkv;
            const float *nw = is_v ? nullptr : (is_q ? a.q_norm : a.k_norm);
            float y[EPL], err[EPL];
            float r = 1.f, ss = 0.f, w[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) w[e] = 1.f;
            if (nw) {
#pragma unroll
                for (int e = 0; e < EPL; ++e) {
                    ss = fmaf(x[u][e], x[u][e], ss);
                    w[e] = nw[lane * EPL + e];
                }
                ss = warp_sum(ss);
                r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
            }
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                y[e] = x[u][e] * r * w[e];
                err[e] = fabsf(y[e]);
            }
            if (half > 0 && !is_v) {
                const int step = half / EPL, e0 = lane * EPL;
                const int src = e0 < half ? lane + step : (e0 < 2 * half ? lane - step : lane);
                const int p0 = e0 < half ? e0 : e0 - half;
                const float sign = e0 < half ? -1.f : 1.f;
#pragma unroll
                for (int e = 0; e < EPL; ++e) {
                    const float other = __shfl_sync(0xffffffffu, y[e], src);
                    if (e0 < 2 * half) {
                        const float2 c = cs[j][p0 + e];
                        err[e] += fabsf(other);
                        y[e] = y[e] * c.x + sign * other * c.y;
                    }
                }
            }
            if (is_q) {
                float *o = a.q_out + ((size_t)(t0 + j) * nq + slot) * D + lane * EPL;
                if constexpr (EPL == 2) {
                    *reinterpret_cast<float2 *>(o) = make_float2(y[0], y[1]);
                } else {
#pragma unroll
                    for (int e = 0; e < EPL; e += 4)
                        *reinterpret_cast<float4 *>(o + e) =
                            make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                }
                continue;
            }
            const int h = is_v ? slot - nq - nkv : slot - nq;
            const float inv_cs = 1.f / (is_v ? a.c.v_scale : a.c.k_scale);   // a power of two
            bool bad = false;
            float amax = 0.f, emax = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const bool fin = fabsf(y[e]) <= 3.4028234e38f;
                bad |= !fin;
                y[e] = isnan(y[e]) ? 0.f : fminf(fmaxf(y[e] * inv_cs, -3.0e38f), 3.0e38f);
                err[e] = is_v ? 0.f : (fin ? err[e] * kRotErr * inv_cs : 0.f);
                amax = fmaxf(amax, fabsf(y[e]));
                emax = fmaxf(emax, err[e]);
            }
#pragma unroll
            for (int m = LPB / 2; m >= 1; m >>= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
                emax = fmaxf(emax, __shfl_xor_sync(0xffffffffu, emax, m));
            }
            const float sv = amax * (1.f / 6.f), se = fmaf(sv, kDivErr, emax * (1.f / 6.f));
            const uint32_t s2 = f32x2_to_e4m3(sv - se, sv + se);
            // (a sum of squares near the ends of the F32 range has lost its bits)
            bool close = (s2 & 0xff) != (s2 >> 8) || (nw && !(ss >= 1e-24f && ss <= 1e38f));
            uint32_t scale_byte = s2 & 0xff, codes = 0;
            const float s = e4m3_to_f32(scale_byte), inv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
            for (int e = 0; e < EPL; e += 2) {
                const float c0 = y[e] * inv, c1 = y[e + 1] * inv;
                const float m0 = fmaf(fabsf(c0), kDivErr, err[e] * inv);
                const float m1 = fmaf(fabsf(c1), kDivErr, err[e + 1] * inv);
                const uint32_t lo = f32x2_to_e2m1(c0 - m0, c1 - m1);
                const uint32_t hi = f32x2_to_e2m1(c0 + m0, c1 + m1);
                close |= lo != hi;
                codes |= lo << (4 * e);
            }
            if (__any_sync(0xffffffffu, close)) {
                const long long pos0 = (long long)tk.z + tk.y;
                quantise_f64<EPL>(x[u], w, nw != nullptr, a.eps, is_v ? 0 : half, pos0,
                                  a.rope.inv_freq, a.rope.positions ? a.rope.positions + t0 + j : nullptr,
                                  (size_t)total, a.rope.axis, a.rope.n_axes, (double)inv_cs, codes,
                                  scale_byte);
            }
            if (bad) set_status(a.status, DF_EINVAL);
            long long at = tk.z < 0 ? -1 : paged_row(a.c, tk.x, h, (long long)tk.z + tk.y, a.status);
            if (at < 0) continue;
            uint8_t *cp = (is_v ? a.c.v_codes : a.c.k_codes) + at * (D / 2) + lane * (EPL / 2);
            if constexpr (EPL == 2) *cp = (uint8_t)codes;
            else if constexpr (EPL == 4) *reinterpret_cast<uint16_t *>(cp) = (uint16_t)codes;
            else *reinterpret_cast<uint32_t *>(cp) = codes;
            if (lane % LPB == 0)
                (is_v ? a.c.v_scales : a.c.k_scales)[at * (D / 16) + lane / LPB] = (uint8_t)scale_byte;
        }
    }
}

// One thread per 8 values of a cached row: 4 bytes of codes in, 32 bytes out. Bound by the F32
// rows written.
__global__ void kv_gather_kernel(const __grid_constant__ df_paged_kv c, const int32_t *start,
                                 const int32_t *n, int n_max, float *k_out, float *v_out,
                                 int32_t *status) {
    DF_TRACE_KERNEL(TK_KV_GATHER);
    pdl_trigger();
    pdl_wait();
    const int per_row = c.head_dim / 8;
    const size_t rows = (size_t)c.batch * c.n_kv_heads * n_max;
    for (size_t x = (size_t)blockIdx.x * blockDim.x + threadIdx.x; x < rows * per_row;
         x += (size_t)gridDim.x * blockDim.x) {
        const size_t row = x / per_row;
        const int p = (int)(x - row * per_row);
        const int i = (int)(row % n_max), bh = (int)(row / n_max);
        const int h = bh % c.n_kv_heads, b = bh / c.n_kv_heads;
        int nn = n ? n[b] : n_max;
        if (nn < 0 || nn > n_max) {
            set_status(status, DF_ESHAPE);
            nn = min(max(nn, 0), n_max);
        }
        if (i >= nn) continue;
        const long long at = paged_row(c, b, h, (long long)(start ? start[b] : 0) + i, status);
        if (at < 0) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(kv ? c.v_codes : c.k_codes)[at * per_row + p];
            const float s = e4m3_to_f32((kv ? c.v_scales : c.k_scales)[at * (per_row / 2) + p / 2]) *
                            (kv ? c.v_scale : c.k_scale);
            uint32_t r[4];
            e2m1x8_to_f16(w, r);
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v2 = __half22float2(*reinterpret_cast<const __half2 *>(&r[e]));
                f[2 * e] = v2.x * s;
                f[2 * e + 1] = v2.y * s;
            }
            float4 *o = reinterpret_cast<float4 *>((kv ? v_out : k_out) + x * 8);
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

}  // namespace

int launch_kv_append_paged(const KvAppendArgs &a, cudaStream_t s) {
    const long long total = (long long)a.c.batch * a.n_max;
    const int slots = a.nq + 2 * a.c.n_kv_heads;
    // Few tokens: one token and at most 8 head slots a CTA, so that every warp has one row and
    // the call is one round trip long. Many: all slots of four tokens, so that the angles are
    // taken once a token and a warp keeps several rows in flight.
    const bool many = total >= 8LL * sm_count();
    const int tokens = many ? kAppendMaxTokens : 1;
    const int per = many ? slots : (slots < kAppendWarps ? slots : kAppendWarps);
    const dim3 grid((unsigned)((total + tokens - 1) / tokens), (unsigned)((slots + per - 1) / per));
    const dim3 block(32 * kAppendWarps);
    switch (a.c.head_dim) {
        case 64: return launch_k("kv_append_kernel", kv_append_kernel<2>, grid, block, 0, s, a, tokens, per);
        case 128: return launch_k("kv_append_kernel", kv_append_kernel<4>, grid, block, 0, s, a, tokens, per);
        default: return launch_k("kv_append_kernel", kv_append_kernel<8>, grid, block, 0, s, a, tokens, per);
    }
}

int launch_kv_gather_paged(const df_paged_kv &c, const int32_t *start, const int32_t *n, int n_max,
                           float *k_out, float *v_out, int32_t *status, cudaStream_t s) {
    const size_t threads = (size_t)c.batch * c.n_kv_heads * n_max * (c.head_dim / 8);
    const size_t ctas = (threads + 255) / 256;
    const unsigned most = 16u * (unsigned)sm_count();
    return launch_k("kv_gather_kernel", kv_gather_kernel, dim3((unsigned)(ctas < most ? ctas : most)),
                    dim3(256), 0, s, c, start, n, n_max, k_out, v_out, status);
}

}  // namespace df
