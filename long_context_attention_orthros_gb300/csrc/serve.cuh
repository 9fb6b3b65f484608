// serve.cuh -- launch parameters and host launchers of the serving kernels (the 8-bit KV cache, the shared
// prompt prefix), and the copies between global and shared memory that only they use.
#pragma once

#include "common.cuh"
#include "kernels.cuh"

namespace orthros {

// After a wait has given up: time enough (1 ms) for the copies and MMAs in flight to land before
// their shared or tensor memory is given back.
__device__ ORTHROS_RARE void drain_in_flight()
{
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
}

// untiled bulk copy: addresses and bytes are multiples of 16
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 16 bytes from global to shared memory without a register on the way (both addresses 16-byte aligned)
__device__ __forceinline__ void cp_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// prompt rows written into, or read back from, the 8-bit cache
struct KvQ8Params {
    orthros_bf16 *k, *v;        // [B, T, Hkv, d], batch stride kv_bstride (inputs of the write)
    uint8_t *k8, *v8;           // codes [B, L_max, Hkv, d]
    int8_t *k_exp, *v_exp;      // exponents [B, Hkv, L_max]
    const int32_t *start, *rows;  // [B] or NULL (0 and T)
    long long kv_bstride;
    int32_t *dev_err;
    int B, T, Hkv, L_max;
};
cudaError_t launch_kv_quantize(int D, int code, const KvQ8Params &p, cudaStream_t stream);
cudaError_t launch_kv_dequantize(int D, int code, const KvQ8Params &p, cudaStream_t stream);

// attention of all rows of a batch over one shared prefix [P, Hkv, d]: partials in slots
// (split, b, KV head, copy * G + head).  k, v maps with boxes of 64 x 1 x 64.
struct PrefixAttnParams {
    const orthros_bf16 *qc;  // [B, T_out, Hq, d], batch stride qc_bstride
    const int32_t *pos;      // [B, T_out] own positions (a copy outside [0, T_kv) takes no key), or NULL
    const float *alpha_c, *beta_c;
    float *part_o;
    float2 *part_ml;
    orthros_bf16 *oc;        // launch_prefix_direct: [B, T_out, Hq, d], batch stride oc_bstride
    int32_t *dev_err;
    long long qc_bstride, oc_bstride;
    int B, T_out, T_kv, P, Hq, Hkv;
    int chunk;  // keys of a split, set by the launcher
    float qscale;
    int *clear;  // optional: n_clear ints that the kernel sets to zero before a dependent kernel reads them
    int n_clear;
};
struct PrefixMaps {
    CUtensorMap k, v, ko, vo;  // the prefix's K and V; the sequences' own (launch_prefix_direct)
};
// mode: 0 one tile of 128 rows, 1 two tiles
cudaError_t launch_prefix_tc(int D, int mode, const PrefixMaps &maps, const PrefixAttnParams &p, int splits, int tiles,
                             cudaStream_t stream);
// copies over the prefix and their own rows in one kernel, outputs at p.oc; tiles of a sequence, or 0
// where partials serve better
int prefix_direct_tiles(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D);
cudaError_t launch_prefix_direct(int D, const PrefixMaps &maps, const PrefixAttnParams &p, cudaStream_t stream);
int prefix_attn_parts(long long copies, int P, int Hq, int Hkv);
cudaError_t launch_prefix_attn(int D, const CUtensorMap &k, const CUtensorMap &v, PrefixAttnParams p,
                               cudaStream_t stream);

// one decode step over the 8-bit cache, or over a shared prefix and each sequence's own bf16 cache
struct ServeParams {
    const orthros_bf16 *q_new, *qc_new, *k_new, *v_new;
    void *k_cache, *v_cache;  // bf16, or codes, [B, L_max, Hkv, d]
    int8_t *k_exp, *v_exp;    // [B, Hkv, L_max] (8-bit form)
    int32_t *cache_len;
    const float *alpha, *beta, *alpha_c, *beta_c;
    orthros_bf16 *o, *oc;
    float *part_o;            // [2 * CTAs (+ B * Hkv behind a prefix)][G][D]
    float2 *part_ml;
    int *cnt_seg;             // [CTAs]: parts of the segment that runs out of a CTA, counted in
    int *cnt_all;
    float *pre_o;             // the prefix kernel's partials (prefix form)
    float2 *pre_ml;
    int32_t *dev_err;
    int B, Hq, Hkv, L_max, window;
    int P, n_part;            // prefix rows (0: 8-bit form) and splits
    int join_after;           // partials are joined by a kernel of its own; set by the launchers
    int join_two;             // a row's partials are joined by two half-warps (by sizes: the order of sums is fixed)
    float qscale;
    long long q_bstride, o_bstride;  // elements between sequences of q_new, qc_new and of o, oc; set by the launchers
};
size_t serve_workspace_bytes(int B, int P, int L_max, int Hq, int Hkv, int D);
// code: ORTHROS_KV_E4M3 / ORTHROS_KV_INT8, or -1 for bf16 caches behind a shared prefix; maps: the
// cache's K and V, then the prefix's (boxes of 64 x 1 x 64; the 8-bit cache's d x 1 x 64)
cudaError_t launch_serve(int D, int code, const CUtensorMap *maps, ServeParams p, void *workspace,
                         cudaStream_t stream);

// one copy a sequence (T_out = 1) over a shared prefix and its own rows; maps as above, workspace of
// serve_workspace_bytes(B, P, T_kv, ...), not initialised
cudaError_t launch_serve_copies(int D, const CUtensorMap *maps, const XattnParams &p, int P, void *workspace,
                                cudaStream_t stream);

// output copies over a shared prefix and their own rows; maps: own K and V, the prefix's K and V
size_t xattn_prefix_workspace_bytes(int B, int T_out, int P, int T_kv, int Hq, int Hkv, int D);
cudaError_t launch_xattn_prefix(int D, const CUtensorMap *maps, XattnParams p, int P, void *workspace,
                                cudaStream_t stream);

// the split-KV kernels alone, over own rows behind a prefix: every row's xattn_parts() partials at
// p.part_o / p.part_ml.  V rows behind a CTA's last position may hold anything.
int xattn_parts(int B, int T_out, int T_kv, int Hq, int Hkv);
cudaError_t launch_xattn_partials(int D, const CUtensorMap &k, const CUtensorMap &v, XattnParams p,
                                  cudaStream_t stream);
// launch_xattn_combine for these and the prefix's partials: one whose sum is a NaN reaches the output
cudaError_t launch_xattn_combine_prefix(int D, const XattnParams &p, cudaStream_t stream);

}  // namespace orthros
