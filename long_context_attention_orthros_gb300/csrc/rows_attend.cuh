// rows_attend.cuh -- softmax attention of a few query rows over keys that come row by row from
// wherever a sequence keeps them: an 8-bit cache, or a shared prefix followed by own rows.
#pragma once

#include "kv_q8.cuh"

namespace orthros {

// rows of one KV head of an 8-bit cache
template <int D, int CODE>
struct RowsQ8 {
    const uint8_t *k, *v;
    const int8_t *ke, *ve;
    long long stride;  // codes between rows
    __device__ __forceinline__ void key8(long long j, int e, float (&f)[8]) const
    {
        const uint2 u = *reinterpret_cast<const uint2 *>(k + j * stride + e);
        const float s = q8_pow2(ke[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = q8_value<CODE>(((i < 4 ? u.x : u.y) >> (8 * (i & 3))) & 0xff) * s;
    }
    __device__ __forceinline__ float value(long long j, int e) const
    {
        return q8_value<CODE>(v[j * stride + e]) * q8_pow2(ve[j]);
    }
};

// bf16 rows of one KV head: the first P from a shared prefix, the others from the sequence's own
template <int D>
struct RowsPrefix {
    const orthros_bf16 *kp, *vp, *k, *v;
    long long stride;
    long long P;
    __device__ __forceinline__ void key8(long long j, int e, float (&f)[8]) const
    {
        const uint4 u = *reinterpret_cast<const uint4 *>((j < P ? kp + j * stride : k + (j - P) * stride) + e);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 g = unpack_bf16x2(w[i]);
            f[2 * i] = g.x;
            f[2 * i + 1] = g.y;
        }
    }
    __device__ __forceinline__ float value(long long j, int e) const
    {
        return __uint_as_float(static_cast<uint32_t>((j < P ? vp + j * stride : v + (j - P) * stride)[e]) << 16);
    }
};

// 128 threads: G query rows q_s[G][D] (scaled into log2 units) over keys lo .. hi (none if
// hi < lo).  Row `fresh` of the keys is not in memory yet: it is taken from knew_s / vnew_s.
// Leaves the unnormalised result in acc (thread t < D holds column t of every row) and the
// rows' maximum and sum in m_s / l_s (-inf and 0 without a key).
template <int D, int G, class Rows>
__device__ void attend_rows(const Rows &rows, const float *q_s, float *logit_s, float *m_s, float *l_s, float *corr_s,
                            const float *knew_s, const float *vnew_s, long long fresh, long long lo, long long hi,
                            float (&acc)[G])
{
    constexpr int NT = 128;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    if (t < G) {
        m_s[t] = NEG_INF;
        l_s[t] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < G; ++r)
        acc[r] = 0.f;
    __syncthreads();
    for (long long c0 = lo; c0 <= hi; c0 += NT) {
        const long long j = c0 + t;
        float s[G];
#pragma unroll
        for (int r = 0; r < G; ++r)
            s[r] = j <= hi ? 0.f : NEG_INF;
        if (j <= hi) {
            for (int e = 0; e < D; e += 8) {
                float f[8];
                if (j == fresh) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = knew_s[e + i];
                } else {
                    rows.key8(j, e, f);
                }
#pragma unroll
                for (int r = 0; r < G; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s[r] = fmaf(q_s[r * D + e + i], f[i], s[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < G; ++r)
            logit_s[r * NT + t] = s[r];
        __syncthreads();
        for (int r = warp; r < G; r += 4) {
            float cm = NEG_INF;
            for (int i = lane; i < NT; i += 32)
                cm = fmaxf(cm, logit_s[r * NT + i]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
            const float mo = m_s[r], mn = fmaxf(mo, cm);
            const float u = mn == NEG_INF ? 0.f : mn;
            float sum = 0.f;
            for (int i = lane; i < NT; i += 32) {
                const float pr = fast_exp2(logit_s[r * NT + i] - u);
                logit_s[r * NT + i] = pr;
                sum += pr;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) {
                const float corr = fast_exp2(mo - u);
                corr_s[r] = corr;
                l_s[r] = l_s[r] * corr + sum;
                m_s[r] = mn;
            }
        }
        __syncthreads();
        if (t < D) {
            const int jn = static_cast<int>(hi - c0 + 1 < NT ? hi - c0 + 1 : NT);
#pragma unroll
            for (int r = 0; r < G; ++r)
                acc[r] *= corr_s[r];
            for (int i = 0; i < jn; ++i) {
                const float v = c0 + i == fresh ? vnew_s[t] : rows.value(c0 + i, t);
#pragma unroll
                for (int r = 0; r < G; ++r)
                    acc[r] = fmaf(logit_s[r * NT + i], v, acc[r]);
            }
        }
        __syncthreads();
    }
}

}  // namespace orthros
