// warp_b16.cuh -- a warp's online softmax over 16 KT keys at a time of bf16 K/V staged with the TMA
// 128-byte swizzle, for up to 8 * NT query rows that share one KV head: S^T = K q^T and
// O^T += V^T P^T on warp MMAs, the keys on the M side, q as a bf16 high part plus residual.
// KT chunks of 16 keys are independent up to the row maxima, which are raised only when a logit
// passes them by more than 8 (log2 units, P <= 2^8 in bf16), so that their instructions overlap and
// the reductions across lanes are rare.
#pragma once

#include "xattn.cuh"

namespace orthros {

template <int D, int NT>
struct WarpB16 {
    uint32_t qb[NT][D / 16][2], ql[NT][D / 16][2];  // q^T fragments of row 8 nt + lane / 4: high part, residual
    float o[NT][D / 16][4];                          // O^T: d = 16 mt + lane / 4 (+ 8), rows 2 (lane % 4) + {0, 1}
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void reset()
    {
        const float NEG_INF = -__int_as_float(0x7f800000);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
                o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
            m[nt][0] = m[nt][1] = NEG_INF;
            l[nt][0] = l[nt][1] = 0.f;
        }
    }

    // query rows of x [n][D] with the scale-offset (all three in shared memory); rows from n on are zeros
    __device__ __forceinline__ void load_q(const orthros_bf16 *x, const float *alpha, const float *beta, int n,
                                           float qscale)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = 8 * nt + (lane >> 2), d = row * D + kt * 16 + 2 * (lane & 3) + 8 * hf;
                    uint32_t hi = 0, lo = 0;
                    if (row < n) {
                        const float2 v = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(x + d));
                        const float2 a = *reinterpret_cast<const float2 *>(alpha + d);
                        const float2 b = *reinterpret_cast<const float2 *>(beta + d);
                        split_q_pair(fmaf(v.x, a.x, b.x) * qscale, fmaf(v.y, a.y, b.y) * qscale, hi, lo);
                    }
                    qb[nt][kt][hf] = hi;
                    ql[nt][kt][hf] = lo;
                }
    }

    // Keys at rows r0 .. r0 + 16 KT - 1 of a block of D / 64 slabs (slab bytes apart).  Unless whole, only
    // rows lo .. hi count; V rows that do not must be finite.
    template <int KT>
    __device__ __forceinline__ void step(uint32_t kbase, uint32_t vbase, int slab, int r0, bool whole, int lo, int hi)
    {
        step_where<KT>(kbase, vbase, slab, r0, whole, [=](int x, int, int) { return x >= lo && x <= hi; });
    }

    // The same; unless whole, key x counts for this lane's query row 8 nt + 2 (lane % 4) + i iff counts(x, nt, i).
    template <int KT, class F>
    __device__ __forceinline__ void step_where(uint32_t kbase, uint32_t vbase, int slab, int r0, bool whole, F counts)
    {
        const int lane = threadIdx.x & 31, gq = lane >> 2;
        const float NEG_INF = -__int_as_float(0x7f800000);
        const int ka_row = r0 + (lane & 7) + (((lane >> 3) & 1) << 3), ka_hi = lane >> 4;
        const int va_row = r0 + (lane & 7) + ((lane >> 4) << 3), va_hi = (lane >> 3) & 1;
        float s[KT][NT][4], s2[KT][NT][4];  // high part and residual of q
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[j][nt][e] = s2[j][nt][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                uint32_t a[4];
                ldsm_x4(kbase + (kt / 4) * slab + sw128_offset(ka_row + 16 * j, (kt % 4) * 2 + ka_hi), a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(s[j][nt], a, qb[nt][kt][0], qb[nt][kt][1]);
                    mma_16816(s2[j][nt], a, ql[nt][kt][0], ql[nt][kt][1]);
                }
            }
        // s[j][nt][e]: key 16 j + gq + 8 (e >> 1), row 8 nt + 2 (lane % 4) + (e & 1)
        bool raise = false;
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][nt][e] += s2[j][nt][e];
                    if (!whole) {
                        const int x = r0 + 16 * j + gq + 8 * (e >> 1);
                        if (!counts(x, nt, e & 1))
                            s[j][nt][e] = NEG_INF;
                    }
                    raise |= s[j][nt][e] > m[nt][e & 1] + 8.f;
                }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = NEG_INF;
#pragma unroll
                    for (int j = 0; j < KT; ++j)
                        mx = fmaxf(mx, fmaxf(s[j][nt][i], s[j][nt][2 + i]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float n = fmaxf(m[nt][i], mx);
                    c[i] = n == NEG_INF ? 1.f : fast_exp2(m[nt][i] - n);
                    m[nt][i] = n;
                    l[nt][i] *= c[i];
                }
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    o[nt][mt][0] *= c[0];
                    o[nt][mt][1] *= c[1];
                    o[nt][mt][2] *= c[0];
                    o[nt][mt][3] *= c[1];
                }
            }
        }
        uint32_t pb[KT][NT][2];
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float u0 = m[nt][0] == NEG_INF ? 0.f : m[nt][0], u1 = m[nt][1] == NEG_INF ? 0.f : m[nt][1];
                const float p0 = fast_exp2(s[j][nt][0] - u0), p1 = fast_exp2(s[j][nt][1] - u1);
                const float p2 = fast_exp2(s[j][nt][2] - u0), p3 = fast_exp2(s[j][nt][3] - u1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pb[j][nt][0] = movmatrix_trans(pack_bf16x2(p0, p1));
                pb[j][nt][1] = movmatrix_trans(pack_bf16x2(p2, p3));
            }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                uint32_t a[4];
                ldsm_x4_trans(vbase + (mt / 4) * slab + sw128_offset(va_row + 16 * j, (mt % 4) * 2 + va_hi), a[0], a[1], a[2],
                              a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816(o[nt][mt], a, pb[j][nt][0], pb[j][nt][1]);
            }
    }

    __device__ __forceinline__ void finish_sums()
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
    }
};

}  // namespace orthros
