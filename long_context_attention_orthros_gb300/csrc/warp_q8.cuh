// warp_q8.cuh -- a warp's online softmax over 16 or 32 keys at a time of an 8-bit cache, for up
// to 8 * NT query rows that share one KV head, on warp MMAs in fp16:
//   S^T = K q^T (16 keys x rows),  O^T += V^T P^T.
// Codes turn into fp16 in registers (exactly), so shared memory is read once, 16 bytes a lane:
// the order of d inside an MMA's k (and m) is free as long as both operands agree, and a lane
// takes whole runs of d instead of the pairs the fragment's plain order would ask for.
//   K: lane (gq = lane / 4, t = lane % 4) reads rows gq and gq + 8, bytes 16 t .. 16 t + 15 (and
//      64 bytes on); its word s is the lane's share of MMA s, and q is laid out alike.
//   V: the lane reads d / 8 bytes at gq d / 8 of its four keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; bytes
//      of two keys are paired by a byte permute before they are converted.
// Scales are powers of two.  A query row is scaled to a largest value in [2^14, 2^15), so its
// size does not matter to fp16; the logit is (q . code) 2^(row shift) 2^(key exponent), in fp32.
// Two running maxima a row, in log2 units: m of the logits x, for the sum of weights, and mv of
// x + ve (ve the key's V exponent), for the second product, whose factors are P = 2^(x + ve - mv + 6)
// in fp16: what a key brings to the output, its weight and its V row's size together, decides what
// its P keeps, so neither a large V row of no weight nor small V rows throughout cost bits.  Both are
// raised only when they are passed by more than 8, so that reductions across lanes are rare and
// P <= 2^14; P rounds to a multiple of 2^-24 at worst, 2^-30 of what the weightiest key of the row
// brings (row sums stay in fp32, unrounded).  A V row of zeros has the exponent 0 but brings nothing:
// where it would raise mv it is passed over.
#pragma once

#include "kv_q8.cuh"

namespace orthros {

// byte offset of 16-byte chunk c of row r in a tile of d-byte rows as TMA's 128-byte (d = 128) or
// 64-byte (d = 64) swizzle lays it out
template <int D>
__device__ __forceinline__ uint32_t q8_offset(int r, int c)
{
    return static_cast<uint32_t>(D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, int NT, int CODE>
struct WarpQ8 {
    uint32_t qb[NT][D / 16][2];  // q^T fragments of row 8 nt + lane / 4
    float qf[NT][2];             // 2^shift of rows 8 nt + 2 (lane % 4) + {0, 1}
    float o[NT][D / 16][4];      // O^T: d = (d / 8) (lane / 4) + 2 mt + (e >> 1), row 2 (lane % 4) + (e & 1)
    float m[NT][2], l[NT][2];
    float mv[NT][2];             // o stands for o 2^(mv - 6)

    __device__ __forceinline__ void reset()
    {
        const float NEG_INF = -__int_as_float(0x7f800000);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
                o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
            m[nt][0] = m[nt][1] = mv[nt][0] = mv[nt][1] = NEG_INF;
            l[nt][0] = l[nt][1] = 0.f;
        }
    }

    // query rows of x [n][D] with the scale-offset (all three in shared memory); rows from n on are zeros
    __device__ __forceinline__ void load_q(const orthros_bf16 *x, const float *alpha, const float *beta, int n,
                                           float qscale)
    {
        const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + (lane >> 2);
            float f[D / 16][4], amax = 0.f;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const int d = 16 * (t + 4 * (s >> 2)) + 4 * (s & 3);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[s][i] = 0.f;
                if (row < n) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(x + row * D + d);
                    const float4 al = *reinterpret_cast<const float4 *>(alpha + row * D + d);
                    const float4 be = *reinterpret_cast<const float4 *>(beta + row * D + d);
                    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
                    f[s][0] = fmaf(a.x, al.x, be.x) * qscale;
                    f[s][1] = fmaf(a.y, al.y, be.y) * qscale;
                    f[s][2] = fmaf(b.x, al.z, be.z) * qscale;
                    f[s][3] = fmaf(b.y, al.w, be.w) * qscale;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fabsf(f[s][i]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            int sh = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
            sh = amax == 0.f ? 0 : (sh < -126 ? -126 : sh);
            const float sd = q8_pow2(-sh);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 h = __floats2half2_rn(f[s][2 * i] * sd, f[s][2 * i + 1] * sd);
                    qb[nt][s][i] = *reinterpret_cast<const uint32_t *>(&h);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qf[nt][i] = q8_pow2(__shfl_sync(0xffffffffu, sh, (2 * t + i) * 4));
        }
    }

    // Keys at rows r0 .. r0 + 16 KT - 1 of the staged block (K codes at kb, V codes at vb, both
    // exponents in shared memory).  Unless whole, only rows lo .. hi of the block count; V rows
    // that do not count must hold finite codes.
    template <int KT>
    __device__ __forceinline__ void step(const uint8_t *kb, const uint8_t *vb, const int8_t *ke, const int8_t *ve, int r0,
                                         bool whole, int lo, int hi)
    {
        const int lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
        const float NEG_INF = -__int_as_float(0x7f800000);
        uint4 ka[KT][D / 64], kc[KT][D / 64];
        float kf[KT][2], ve2[KT][2];
#pragma unroll
        for (int j = 0; j < KT; ++j) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                ka[j][c] = *reinterpret_cast<const uint4 *>(kb + q8_offset<D>(r0 + 16 * j + gq, t + 4 * c));
                kc[j][c] = *reinterpret_cast<const uint4 *>(kb + q8_offset<D>(r0 + 16 * j + gq + 8, t + 4 * c));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kf[j][i] = q8_pow2(ke[r0 + 16 * j + gq + 8 * i]);
                ve2[j][i] = static_cast<float>(ve[r0 + 16 * j + gq + 8 * i]);
            }
        }
        float s[KT][NT][4], s2[KT][NT][4];
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[j][nt][e] = s2[j][nt][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                const uint4 ua = ka[j][k >> 2], uc = kc[j][k >> 2];
                const uint32_t wa = (k & 3) == 0 ? ua.x : (k & 3) == 1 ? ua.y : (k & 3) == 2 ? ua.z : ua.w;
                const uint32_t wc = (k & 3) == 0 ? uc.x : (k & 3) == 1 ? uc.y : (k & 3) == 2 ? uc.z : uc.w;
                const uint32_t a[4] = {q8_half2<CODE>(wa, false), q8_half2<CODE>(wc, false), q8_half2<CODE>(wa, true),
                                       q8_half2<CODE>(wc, true)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816_f16((k & 1) ? s2[j][nt] : s[j][nt], a, qb[nt][k][0], qb[nt][k][1]);
            }
        // s[j][nt][e]: key 16 j + gq + 8 (e >> 1), row 8 nt + 2 t + (e & 1)
        bool raise = false;
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][nt][e] = (s[j][nt][e] + s2[j][nt][e]) * qf[nt][e & 1] * kf[j][e >> 1];
                    if (!whole) {
                        const int x = r0 + 16 * j + gq + 8 * (e >> 1);
                        if (x < lo || x > hi)
                            s[j][nt][e] = NEG_INF;
                    }
                    raise |= s[j][nt][e] > m[nt][e & 1] + 8.f || s[j][nt][e] + ve2[j][e >> 1] > mv[nt][e & 1] + 8.f;
                }
        // rare: one of a row's maxima goes up
        if (__any_sync(0xffffffffu, raise)) {
            constexpr uint32_t SIZE = CODE == ORTHROS_KV_E4M3 ? 0x7f7f7f7fu : 0xffffffffu;  // e4m3 has a zero of either sign
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t any = 0;  // of a quarter of the V row, then of all of it
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(vb + q8_offset<D>(r0 + 16 * j + gq + 8 * i, t + 4 * c));
                        any |= (u.x | u.y | u.z | u.w) & SIZE;
                    }
                    any |= __shfl_xor_sync(0xffffffffu, any, 1);
                    any |= __shfl_xor_sync(0xffffffffu, any, 2);
                    if (any == 0)
                        ve2[j][i] = NEG_INF;
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = NEG_INF, mw = NEG_INF;
#pragma unroll
                    for (int j = 0; j < KT; ++j) {
                        mx = fmaxf(mx, fmaxf(s[j][nt][i], s[j][nt][2 + i]));
                        mw = fmaxf(mw, fmaxf(s[j][nt][i] + ve2[j][0], s[j][nt][2 + i] + ve2[j][1]));
                    }
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, off));
                    }
                    const float n = fmaxf(m[nt][i], mx), nv = fmaxf(mv[nt][i], mw);
                    l[nt][i] *= n == NEG_INF ? 1.f : fast_exp2(m[nt][i] - n);
                    c[i] = nv == NEG_INF ? 1.f : fast_exp2(mv[nt][i] - nv);
                    m[nt][i] = n;
                    mv[nt][i] = nv;
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
                float p[4], pv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float mm = m[nt][e & 1], mw = mv[nt][e & 1];
                    p[e] = fast_exp2(s[j][nt][e] - (mm == NEG_INF ? 0.f : mm));
                    pv[e] = fast_exp2(s[j][nt][e] + (ve2[j][e >> 1] - (mw == NEG_INF ? 0.f : mw - 6.f)));
                }
                l[nt][0] += p[0] + p[2];
                l[nt][1] += p[1] + p[3];
                const __half2 h0 = __floats2half2_rn(pv[0], pv[1]);
                const __half2 h1 = __floats2half2_rn(pv[2], pv[3]);
                pb[j][nt][0] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h0));
                pb[j][nt][1] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h1));
            }
        // V: four keys of every 16, D / 8 bytes each
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            uint32_t w[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + 16 * j + 2 * t + (i & 1) + 8 * (i >> 1);
                if constexpr (D == 128) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(vb + q8_offset<D>(r, gq));
                    w[i][0] = u.x;
                    w[i][1] = u.y;
                    w[i][2] = u.z;
                    w[i][3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(vb + q8_offset<D>(r, gq >> 1) + 8 * (gq & 1));
                    w[i][0] = u.x;
                    w[i][1] = u.y;
                }
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t x = __byte_perm(w[0][c], w[1][c], hf ? 0x7362 : 0x5140);
                    const uint32_t y = __byte_perm(w[2][c], w[3][c], hf ? 0x7362 : 0x5140);
                    const uint32_t a[4] = {q8_half2<CODE>(x, false), q8_half2<CODE>(x, true), q8_half2<CODE>(y, false),
                                           q8_half2<CODE>(y, true)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816_f16(o[nt][2 * c + hf], a, pb[j][nt][0], pb[j][nt][1]);
                }
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
