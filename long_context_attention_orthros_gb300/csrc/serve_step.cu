// serve_step.cu -- one decode step over an 8-bit KV cache, or over a prompt prefix that the
// whole batch shares and each sequence's own bf16 cache.  Per sequence with p = cache_len[b]:
//   append k_new / v_new at own row p (as codes in the 8-bit form),
//   o  = Eq. (4) for the new base token over its last `window` rows,
//   oc = Eq. (5) for its output copy over every row (prefix, own rows, the new one),
//   cache_len[b] = p + 1.
// One launch, grid (nsplit + 1, B * Hkv): CTA x < nsplit takes its share of the copy's keys, the
// last one the base token's window and the append; the last of a (b, KV head) to arrive joins
// the copy's partials.
#include "rows_attend.cuh"

namespace orthros {

template <int D, int CODE>
struct RowsOf {
    using type = RowsQ8<D, CODE>;
};
template <int D>
struct RowsOf<D, -1> {
    using type = RowsPrefix<D>;
};

template <int D, int G, int CODE>
__global__ void __launch_bounds__(128) serve_step_kernel(const ServeParams p)
{
    constexpr bool Q8 = CODE >= 0;
    __shared__ float q_s[G * D], logit_s[G * 128], m_s[G], l_s[G], corr_s[G], knew_s[D], vnew_s[D];
    __shared__ int last_s;
    const int x = blockIdx.x, bh = blockIdx.y, b = bh / p.Hkv, g = bh % p.Hkv;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int pcur = p.cache_len[b];
    const bool full = pcur < 0 || pcur >= p.L_max;
    const long long stride = static_cast<long long>(p.Hkv) * D;
    const long long base = (static_cast<long long>(b) * p.L_max * p.Hkv + g) * D;
    const long long last = static_cast<long long>(p.P) + pcur;  // the new token's position
    typename RowsOf<D, CODE>::type rows;
    int8_t *ke = nullptr, *ve = nullptr;
    if constexpr (Q8) {
        ke = p.k_exp + static_cast<long long>(bh) * p.L_max;
        ve = p.v_exp + static_cast<long long>(bh) * p.L_max;
        rows = {static_cast<const uint8_t *>(p.k_cache) + base, static_cast<const uint8_t *>(p.v_cache) + base, ke, ve,
                stride};
    } else {
        rows = {p.k_prefix + g * D, p.v_prefix + g * D, static_cast<const orthros_bf16 *>(p.k_cache) + base,
                static_cast<const orthros_bf16 *>(p.v_cache) + base, stride, p.P};
    }
    // the new row, one warp each for K and V
    if (warp < 2) {
        const orthros_bf16 *src = (warp ? p.v_new : p.k_new) + (static_cast<long long>(b) * p.Hkv + g) * D;
        float *dst = warp ? vnew_s : knew_s;
        constexpr int E = D / 32;
        float f[E], amax = 0.f;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            f[e] = __uint_as_float(static_cast<uint32_t>(src[lane * E + e]) << 16);
            if (fabsf(f[e]) < __int_as_float(0x7f800000))
                amax = fmaxf(amax, fabsf(f[e]));
            else
                bad = true;
        }
        if constexpr (Q8) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int ex = q8_exponent<CODE>(amax);
            uint8_t *out = static_cast<uint8_t *>(warp ? p.v_cache : p.k_cache) + base + pcur * stride;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t c = q8_codes2<CODE>(f[e] * q8_pow2(-ex), f[e + 1] * q8_pow2(-ex));
                dst[lane * E + e] = q8_value<CODE>(c & 0xff) * q8_pow2(ex);
                dst[lane * E + e + 1] = q8_value<CODE>(c >> 8) * q8_pow2(ex);
                if (x == p.nsplit && !full)
                    *reinterpret_cast<uint16_t *>(out + lane * E + e) = static_cast<uint16_t>(c);
            }
            if (x == p.nsplit && !full) {
                if (lane == 0)
                    (warp ? ve : ke)[pcur] = static_cast<int8_t>(ex);
                if (bad)
                    record_error(p.dev_err, ORTHROS_DEVERR_RANGE);
            }
        } else {
            orthros_bf16 *out = static_cast<orthros_bf16 *>(warp ? p.v_cache : p.k_cache) + base + pcur * stride;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                dst[lane * E + e] = f[e];
                if (x == p.nsplit && !full)
                    out[lane * E + e] = src[lane * E + e];
            }
        }
    }
    const bool copy = x < p.nsplit;
    for (int i = t; i < G * D; i += 128) {
        const int h = g * G + i / D, e = i % D;
        const float x0 = __uint_as_float(
            static_cast<uint32_t>((copy ? p.qc_new : p.q_new)[(static_cast<long long>(b) * p.Hq + h) * D + e]) << 16);
        q_s[i] = fmaf(x0, (copy ? p.alpha_c : p.alpha)[h * D + e], (copy ? p.beta_c : p.beta)[h * D + e]) * p.qscale;
    }
    __syncthreads();
    long long lo, hi;
    if (copy) {
        const long long chunk = (last + p.nsplit) / p.nsplit;
        lo = x * chunk;
        hi = lo + chunk - 1 < last ? lo + chunk - 1 : last;
    } else {
        lo = last - p.window + 1 > 0 ? last - p.window + 1 : 0;
        hi = last;
    }
    if (full)
        hi = lo - 1;
    float acc[G];
    attend_rows<D, G>(rows, q_s, logit_s, m_s, l_s, corr_s, knew_s, vnew_s, last, lo, hi, acc);
    if (!copy) {
        if (full && g == 0 && t == 0)
            record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
        if (t < D)
#pragma unroll
            for (int r = 0; r < G; ++r) {
                const float v = l_s[r] > 0.f ? acc[r] / l_s[r] : 0.f;
                p.o[(static_cast<long long>(b) * p.Hq + g * G + r) * D + t] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            }
    } else {
        const long long slot = (static_cast<long long>(bh) * p.n_part + x) * G;
        if (t < D)
#pragma unroll
            for (int r = 0; r < G; ++r)
                p.part_o[(slot + r) * D + t] = acc[r];
        if (t < G)
            p.part_ml[slot + t] = make_float2(m_s[t], l_s[t]);
    }
    __threadfence();
    __syncthreads();
    if (t == 0)
        last_s = atomicAdd(&p.cnt_bh[bh], 1) == p.nsplit ? 1 : 0;
    __syncthreads();
    if (!last_s)
        return;
    __threadfence();
    for (int r = 0; r < G; ++r) {
        float M = NEG_INF, L = 0.f, a = 0.f;
        const long long slot = static_cast<long long>(bh) * p.n_part * G + r;
        for (int q = 0; q < p.n_part; ++q)
            M = fmaxf(M, __ldcg(&p.part_ml[slot + q * G]).x);
        for (int q = 0; q < p.n_part; ++q) {
            const float2 ml = __ldcg(&p.part_ml[slot + q * G]);
            const float w = ml.y > 0.f ? fast_exp2(ml.x - M) : 0.f;
            L += w * ml.y;
            if (t < D && ml.y > 0.f)
                a += w * __ldcg(&p.part_o[(slot + q * G) * D + t]);
        }
        if (t < D)
            p.oc[(static_cast<long long>(b) * p.Hq + g * G + r) * D + t] =
                __bfloat16_as_ushort(__float2bfloat16_rn(L > 0.f ? a / L : 0.f));
    }
    if (t == 0) {
        p.cnt_bh[bh] = 0;
        __threadfence();
        if (atomicAdd(&p.cnt_b[b], 1) == p.Hkv - 1) {
            if (!full)
                p.cache_len[b] = pcur + 1;
            p.cnt_b[b] = 0;
        }
    }
}

static int serve_nsplit(int B, int P, int L_max, int Hkv)
{
    long long ns = 608 / (static_cast<long long>(B) * Hkv);
    const long long by_len = (static_cast<long long>(P) + L_max + 255) / 256;
    ns = ns > by_len ? by_len : ns;
    return static_cast<int>(ns < 1 ? 1 : ns);
}

size_t serve_workspace_bytes(int B, int P, int L_max, int Hq, int Hkv, int D)
{
    const size_t BH = static_cast<size_t>(B) * Hkv, slots = BH * serve_nsplit(B, P, L_max, Hkv) * (Hq / Hkv);
    return (slots * D * sizeof(float) + 255) / 256 * 256 + (slots * sizeof(float2) + 255) / 256 * 256 +
           ((BH + B) * sizeof(int) + 255) / 256 * 256;
}

template <int D, int G>
static cudaError_t launch_serve_t(int code, const ServeParams &p, cudaStream_t stream)
{
    const dim3 grid(p.nsplit + 1, p.B * p.Hkv);
    if (code == ORTHROS_KV_E4M3)
        serve_step_kernel<D, G, ORTHROS_KV_E4M3><<<grid, 128, 0, stream>>>(p);
    else if (code == ORTHROS_KV_INT8)
        serve_step_kernel<D, G, ORTHROS_KV_INT8><<<grid, 128, 0, stream>>>(p);
    else
        serve_step_kernel<D, G, -1><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_serve(int D, int code, ServeParams p, void *workspace, cudaStream_t stream)
{
    const int G = p.Hq / p.Hkv;
    p.nsplit = p.n_part = serve_nsplit(p.B, p.P, p.L_max, p.Hkv);
    const size_t BH = static_cast<size_t>(p.B) * p.Hkv, slots = BH * p.n_part * G;
    const size_t o_bytes = (slots * D * sizeof(float) + 255) / 256 * 256;
    const size_t ml_bytes = (slots * sizeof(float2) + 255) / 256 * 256;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + o_bytes);
    p.cnt_bh = reinterpret_cast<int *>(ws + o_bytes + ml_bytes);
    p.cnt_b = p.cnt_bh + BH;
#define ORTHROS_SERVE_CASE(DD, GG) \
    if (D == DD && G == GG)        \
        return launch_serve_t<DD, GG>(code, p, stream);
    ORTHROS_SERVE_CASE(128, 1)
    ORTHROS_SERVE_CASE(128, 2)
    ORTHROS_SERVE_CASE(128, 4)
    ORTHROS_SERVE_CASE(128, 8)
    ORTHROS_SERVE_CASE(128, 16)
    ORTHROS_SERVE_CASE(64, 1)
    ORTHROS_SERVE_CASE(64, 2)
    ORTHROS_SERVE_CASE(64, 4)
    ORTHROS_SERVE_CASE(64, 8)
    ORTHROS_SERVE_CASE(64, 16)
#undef ORTHROS_SERVE_CASE
    return cudaErrorInvalidValue;
}

}  // namespace orthros
