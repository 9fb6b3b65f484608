// xattn_prefix.cu -- output-copy cross-attention, Eq. (5), for a batch whose sequences share a
// prompt prefix: copy i of sequence b attends over the prefix rows 0 .. P-1 and its sequence's
// own rows 0 .. pos.  The prefix kernel takes all rows of the batch over the prefix, the split-KV
// kernels of xattn_fwd.cu the copies over their own rows, each writing partials; one combine
// kernel joins both.  One copy a sequence goes through the decode step's kernel behind the prefix
// kernel (serve_step.cu), which joins in the same launch.  Many copies a sequence take prefix and
// own rows in one kernel instead.
#include "serve.cuh"

namespace orthros {

namespace {

struct XpLayout {
    int pre, own;  // partials a row has of each
    size_t part_ml, total;
};

XpLayout xp_layout(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D)
{
    XpLayout l = {0, 0, 0, 256};
    if (prefix_direct_tiles(B, T_out, P, T_kv, Hq, Hkv, D) > 0)
        return l;
    if (T_out == 1) {
        l.total = serve_workspace_bytes(B, P, T_kv, Hq, Hkv, D);
        return l;
    }
    l.pre = prefix_attn_parts(static_cast<long long>(B) * T_out, P, Hq, Hkv);
    l.own = xattn_parts(B, T_out, T_kv, Hq, Hkv);
    const size_t slots = (static_cast<size_t>(l.pre) + l.own) * B * T_out * Hq;
    l.part_ml = (slots * D * sizeof(float) + 255) / 256 * 256;
    l.total = l.part_ml + (slots * sizeof(float2) + 255) / 256 * 256;
    return l;
}

}  // namespace

size_t xattn_prefix_workspace_bytes(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D)
{
    return xp_layout(B, T_out, P, T_kv, Hq, Hkv, D).total;
}

cudaError_t launch_xattn_prefix(int D, const CUtensorMap *m, XattnParams x, int P, void *workspace, cudaStream_t stream)
{
    if (x.T_out == 1)
        return launch_serve_copies(D, m, x, P, workspace, stream);
    const XpLayout l = xp_layout(x.B, x.T_out, P, x.T_kv, x.Hq, x.Hkv, D);
    float *part_o = static_cast<float *>(workspace);
    float2 *part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + l.part_ml);
    PrefixAttnParams a{};
    a.qc = x.qc;
    a.pos = x.pos;
    a.alpha_c = x.alpha_c;
    a.beta_c = x.beta_c;
    a.part_o = part_o;
    a.part_ml = part_ml;
    a.dev_err = x.dev_err;
    a.qc_bstride = x.qc_bstride;
    a.B = x.B;
    a.T_out = x.T_out;
    a.T_kv = x.T_kv;
    a.P = P;
    a.Hq = x.Hq;
    a.Hkv = x.Hkv;
    a.qscale = x.qscale;
    if (prefix_direct_tiles(x.B, x.T_out, P, x.T_kv, x.Hq, x.Hkv, D) > 0) {
        a.oc = x.oc;
        a.oc_bstride = x.oc_bstride;
        return launch_prefix_direct(D, PrefixMaps{m[2], m[3], m[0], m[1]}, a, stream);
    }
    cudaError_t e = launch_prefix_attn(D, m[2], m[3], a, stream);
    if (e != cudaSuccess)
        return e;
    const size_t rows = static_cast<size_t>(x.B) * x.T_out * x.Hq;
    x.part_o = part_o + static_cast<size_t>(l.pre) * rows * D;
    x.part_ml = part_ml + static_cast<size_t>(l.pre) * rows;
    e = launch_xattn_partials(D, m[0], m[1], x, stream);
    if (e != cudaSuccess)
        return e;
    x.G = x.Hq / x.Hkv;
    x.R = x.T_out * x.G;
    x.part_o = part_o;
    x.part_ml = part_ml;
    x.n_part = l.pre + l.own;
    return launch_xattn_combine_prefix(D, x, stream);
}

}  // namespace orthros
