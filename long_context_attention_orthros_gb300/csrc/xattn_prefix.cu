// xattn_prefix.cu -- output-copy cross-attention, Eq. (5), for a batch whose sequences share a
// prompt prefix: copy i of sequence b attends over the prefix rows 0 .. P-1 and its sequence's
// own rows 0 .. pos.  Grid (split, KV head, copy): a CTA takes the G query rows of one copy over
// its share of the keys; the combine kernel joins the partials.
#include "rows_attend.cuh"

namespace orthros {

template <int D, int G>
__global__ void __launch_bounds__(128) xattn_prefix_kernel(const XattnPrefixParams p)
{
    const XattnParams &x = p.x;
    __shared__ float q_s[G * D], logit_s[G * 128], m_s[G], l_s[G], corr_s[G];
    const int g = blockIdx.x % x.Hkv, split = blockIdx.x / x.Hkv;
    const long long bi = blockIdx.y + static_cast<long long>(blockIdx.z) * 32768;
    if (bi >= static_cast<long long>(x.B) * x.T_out)
        return;
    const int b = static_cast<int>(bi / x.T_out), i = static_cast<int>(bi % x.T_out), t = threadIdx.x;
    const long long stride = static_cast<long long>(x.Hkv) * D;
    const RowsPrefix<D> rows = {p.k_prefix + g * D, p.v_prefix + g * D, p.k + b * p.kv_bstride + g * D,
                                p.v + b * p.kv_bstride + g * D, stride, p.P};
    const int pos = x.pos[bi];
    const bool ok = pos >= 0 && pos < x.T_kv;
    if (!ok && split == 0 && g == 0 && t == 0)
        record_error(x.dev_err, ORTHROS_DEVERR_POSITION);
    for (int e = t; e < G * D; e += 128) {
        const int h = g * G + e / D, c = e % D;
        const float x0 = __uint_as_float(
            static_cast<uint32_t>(x.qc[b * x.qc_bstride + (static_cast<long long>(i) * x.Hq + h) * D + c]) << 16);
        q_s[e] = fmaf(x0, x.alpha_c[h * D + c], x.beta_c[h * D + c]) * x.qscale;
    }
    __syncthreads();
    const long long n = static_cast<long long>(p.P) + pos + 1, chunk = (n + x.splits - 1) / x.splits;
    const long long lo = split * chunk, hi = ok ? (lo + chunk < n ? lo + chunk : n) - 1 : lo - 1;
    float acc[G];
    attend_rows<D, G>(rows, q_s, logit_s, m_s, l_s, corr_s, q_s, q_s, -1, lo, hi, acc);
    const long long slot =
        (static_cast<long long>(split) * x.B * x.Hkv + b * x.Hkv + g) * x.R + static_cast<long long>(i) * G;
    if (t < D)
#pragma unroll
        for (int r = 0; r < G; ++r)
            x.part_o[(slot + r) * D + t] = acc[r];
    if (t < G)
        x.part_ml[slot + t] = make_float2(m_s[t], l_s[t]);
}

static int prefix_splits(int B, int T_out, int P, int T_kv, int Hkv)
{
    long long ns = 608 / (static_cast<long long>(B) * Hkv * T_out);
    const long long by_len = (static_cast<long long>(P) + T_kv + 255) / 256;
    ns = ns > by_len ? by_len : ns;
    return static_cast<int>(ns < 1 ? 1 : ns);
}

size_t xattn_prefix_workspace_bytes(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D)
{
    const size_t slots = static_cast<size_t>(prefix_splits(B, T_out, P, T_kv, Hkv)) * B * T_out * Hq;
    return (slots * D * sizeof(float) + 255) / 256 * 256 + (slots * sizeof(float2) + 255) / 256 * 256;
}

template <int D, int G>
static cudaError_t launch_xattn_prefix_t(const XattnPrefixParams &p, cudaStream_t stream)
{
    const long long n = static_cast<long long>(p.x.B) * p.x.T_out;
    const dim3 grid(p.x.splits * p.x.Hkv, static_cast<unsigned>(n < 32768 ? n : 32768),
                    static_cast<unsigned>((n + 32767) / 32768));
    xattn_prefix_kernel<D, G><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_xattn_prefix(int D, XattnPrefixParams p, void *workspace, cudaStream_t stream)
{
    XattnParams &x = p.x;
    x.G = x.Hq / x.Hkv;
    x.R = x.T_out * x.G;
    x.splits = x.n_part = prefix_splits(x.B, x.T_out, p.P, x.T_kv, x.Hkv);
    const size_t slots = static_cast<size_t>(x.n_part) * x.B * x.T_out * x.Hq;
    x.part_o = static_cast<float *>(workspace);
    x.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + (slots * D * sizeof(float) + 255) / 256 * 256);
    cudaError_t e = cudaErrorInvalidValue;
#define ORTHROS_XP_CASE(DD, GG)     \
    if (D == DD && x.G == GG)       \
        e = launch_xattn_prefix_t<DD, GG>(p, stream);
    ORTHROS_XP_CASE(128, 1)
    ORTHROS_XP_CASE(128, 2)
    ORTHROS_XP_CASE(128, 4)
    ORTHROS_XP_CASE(128, 8)
    ORTHROS_XP_CASE(128, 16)
    ORTHROS_XP_CASE(64, 1)
    ORTHROS_XP_CASE(64, 2)
    ORTHROS_XP_CASE(64, 4)
    ORTHROS_XP_CASE(64, 8)
    ORTHROS_XP_CASE(64, 16)
#undef ORTHROS_XP_CASE
    return e == cudaSuccess ? launch_xattn_combine(D, x, stream) : e;
}

}  // namespace orthros
