// sink_bwd.cu -- gradient of the base stream with attention sinks (row t sees keys j <= t with j > t - window or
// j < sinks), given the forward's log-sum-exp and output.  With x = Q_raw, q = x alpha + beta,
//   p_tj = exp(scale q_t . k_j - lse_t),  D_t = dO_t . o_t,  dS_tj = p_tj (dO_t . v_j - D_t)
//   dq_t = scale sum_j dS_tj k_j,  dq_raw = dq alpha,  dalpha = sum_t x_t dq_t,  dbeta = sum_t dq_t
//   dk_j = scale sum_t dS_tj q_t,  dv_j = sum_t p_tj dO_t
// Everything leaves in fp32 and is computed to match: k, v, x and dO are bf16 and enter the products as they are;
// q, dS and P enter as a bf16 high part plus residual (their product's relative error some 2^-17, where one
// bf16 would give 2^-9); sums, exponents and D are fp32.  Launches:
//   sink_rows_kernel    q's two parts, D and the log-sum-exp in log2 units, one pass over x, o, dO
//   sink_dq_kernel      dq of 64 rows over their band and the sinks, warp MMAs; dalpha, dbeta by atomics
//   sink_dkv_tc_kernel  dk, dv of the window's part (sink_dkv.cu)
//   sink_keys_kernel    the sinks' share of the rows behind their window: every row adds to the same few keys, so
//                       the tokens are split over CTAs, whose partial sums sink_join_kernel adds to dk, dv in order
#include "bwd_util.cuh"
#include "kernels.cuh"
#include "xattn.cuh"

namespace orthros {

namespace {

// ------------------------------------------------------------------ prepared rows

// D / 8 lanes a row, 16 bytes of each of x, o and dO a lane.  The first CTAs also zero dalpha and dbeta.
template <int D>
__global__ void __launch_bounds__(256) sink_rows_kernel(const SinkBwdParams p)
{
    constexpr int LPR = D / 8;
    const long long rows = static_cast<long long>(p.B) * p.T * p.Hq;
    const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x, row = id / LPR;
    const int sub = static_cast<int>(id % LPR);
    for (long long i = id; i < p.Hq * D; i += static_cast<long long>(gridDim.x) * blockDim.x)
        p.dalpha[i] = p.dbeta[i] = 0.f;
    float acc = 0.f;
    if (row < rows) {
        const long long off = row * D + sub * 8;
        const uint4 xa = __ldg(reinterpret_cast<const uint4 *>(p.q + off));
        const uint4 oa = __ldg(reinterpret_cast<const uint4 *>(p.o + off));
        const uint4 ga = __ldg(reinterpret_cast<const uint4 *>(p.dO + off));
        const int col = static_cast<int>(row % p.Hq) * D + sub * 8;
        const uint32_t xw[4] = {xa.x, xa.y, xa.z, xa.w}, ow[4] = {oa.x, oa.y, oa.z, oa.w}, gw[4] = {ga.x, ga.y, ga.z, ga.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(p.alpha + col) + e);
            const float2 b = __ldg(reinterpret_cast<const float2 *>(p.beta + col) + e);
            const float2 x = unpack_bf16x2(xw[e]), u = unpack_bf16x2(ow[e]), v = unpack_bf16x2(gw[e]);
            split_q_pair(fmaf(x.x, a.x, b.x), fmaf(x.y, a.y, b.y), hi[e], lo[e]);
            acc = fmaf(u.x, v.x, fmaf(u.y, v.y, acc));
        }
        *reinterpret_cast<uint4 *>(p.q_hi + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(p.q_lo + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
        acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (row < rows && sub == 0) {
        p.Drow[row] = acc;
        p.lse[row] = p.lse_in[row] * kLog2eF;
    }
}

// ------------------------------------------------------------------ dq

constexpr int DQ_ROWS = 64;  // query rows of a CTA: 64 / G tokens x G heads
constexpr int DQ_KEYS = 64;  // keys of a streamed block
constexpr int DQ_RUN = 32;   // blocks that dq is summed over in the MMA's accumulators (256 steps: some 4e-6)

template <int D, int G>
__global__ void __launch_bounds__(128) sink_dq_kernel(const SinkBwdParams p)
{
    constexpr int TOK = DQ_ROWS / G;
    constexpr int SLAB = DQ_KEYS * 128;   // one 64-column slab of a 64-key block
    constexpr int BLK = (D / 64) * SLAB;  // one K (or V) block
    const int u0 = blockIdx.x * TOK, bh = blockIdx.y;
    const int b = bh / p.Hkv, g = bh % p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    float *red = reinterpret_cast<float *>(smem + 4 * BLK);  // [2][G][D]: dalpha, dbeta
    const uint32_t sbase = smem_u32(smem);

    // this warp's 16 rows: r = 16 warp + 0..15 -> token u0 + r / G, head g G + r % G
    const int gr = lane >> 2, qd = (lane & 3) * 2;
    const int rowA = 16 * warp + gr, rowB = rowA + 8;
    const int tA = u0 + rowA / G, tB = u0 + rowB / G;
    const int hA = g * G + rowA % G, hB = g * G + rowB % G;
    const bool vA = tA < p.T, vB = tB < p.T;
    const int loA = tA - p.window + 1, loB = tB - p.window + 1;
    const int t_lo = u0 + 16 * warp / G, t_hi = min(p.T - 1, u0 + (16 * warp + 15) / G);  // the warp's tokens
    const int wlo = max(0, t_lo - p.window + 1), whi = t_lo < p.T ? t_hi : -1;
    for (int i = threadIdx.x; i < 2 * G * D; i += 128)
        red[i] = 0.f;
    const int cb0 = max(0, u0 - p.window + 1) / DQ_KEYS, cb1 = min(p.T - 1, u0 + TOK - 1) / DQ_KEYS + 1;
    const int far = p.sinks > 0 && cb0 > 0 ? 1 : 0;  // the sinks' block comes first
    const int nblk = cb1 - cb0 + far;

    const long long q_bs = static_cast<long long>(p.T) * p.Hq * D;
    const float c2 = p.scale * kLog2eF;  // logits in log2 units
    WarpRows16<D> st;                    // q fragments and the dQ accumulators
    uint32_t ga[D / 16][4];              // dO fragments (A operand)
#pragma unroll
    for (int kt2 = 0; kt2 < D / 16; ++kt2)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool isB = r & 1;
            const int t = isB ? tB : tA, h = isB ? hB : hA;
            const int dcol = kt2 * 16 + qd + ((r & 2) ? 8 : 0);
            uint32_t hi = 0, lo = 0, gw = 0;
            if (isB ? vB : vA) {
                const long long off = b * q_bs + (static_cast<long long>(t) * p.Hq + h) * D + dcol;
                hi = *reinterpret_cast<const uint32_t *>(p.q_hi + off);
                lo = *reinterpret_cast<const uint32_t *>(p.q_lo + off);
                gw = *reinterpret_cast<const uint32_t *>(p.dO + off);
            }
            st.qa[kt2][r] = hi;
            st.ql[kt2][r] = lo;
            ga[kt2][r] = gw;
        }
    st.reset();
    const int kld_row = (lane & 7) + ((lane >> 4) << 3), kld_hi = (lane >> 3) & 1;
    const int vld_row = (lane & 7) + (((lane >> 3) & 1) << 3), vld_hi = lane >> 4;

    const long long kv_rs = static_cast<long long>(p.Hkv) * D;
    const orthros_bf16 *kb = p.k + static_cast<long long>(b) * p.T * kv_rs + static_cast<long long>(g) * D;
    const orthros_bf16 *vb = p.v + static_cast<long long>(b) * p.T * kv_rs + static_cast<long long>(g) * D;
    // stream the i-th block into ring slot i % 2; behind the sinks their block has zeros
    auto stage = [&](int i) {
        const bool sink = i < far;
        const int key0 = sink ? 0 : (cb0 + i - far) * DQ_KEYS, end = sink ? p.sinks : p.T;
        for (int e = threadIdx.x; e < DQ_KEYS * (D / 8); e += 128) {
            const int r = e / (D / 8), c = (e % (D / 8)) * 8;
            const bool ok = key0 + r < end;
            const long long off = static_cast<long long>(ok ? key0 + r : 0) * kv_rs + c;
            const uint32_t o = sbase + (i & 1) * 2 * BLK + tile_off(r, c, SLAB);
            cp_async16(o, kb + off, ok);
            cp_async16(o + BLK, vb + off, ok);
        }
        cp_async_commit();
    };

    const long long rA = (static_cast<long long>(b) * p.T + tA) * p.Hq + hA;
    const long long rB = (static_cast<long long>(b) * p.T + tB) * p.Hq + hB;
    const float lseA = vA ? p.lse[rA] : 0.f, lseB = vB ? p.lse[rB] : 0.f;
    const float DA = vA ? p.Drow[rA] : 0.f, DB = vB ? p.Drow[rB] : 0.f;
    stage(0);
#pragma unroll 1
    for (int i = 0; i < nblk; ++i) {
        const bool sink = i < far;
        if (i + 1 < nblk) {
            stage(i + 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const uint32_t kbase = sbase + (i & 1) * 2 * BLK, vbase = kbase + BLK;
#pragma unroll 1
        for (int jc = 0; jc < DQ_KEYS; jc += 16) {
            const int kc = (sink ? 0 : (cb0 + i - far) * DQ_KEYS) + jc;
            if (kc > whi || (kc + 15 < wlo && kc >= p.sinks))
                continue;  // warp-uniform: no key of this chunk is seen by the warp's rows
            float s[2][4], dp[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] = dp[n][e] = 0.f;
#pragma unroll
            for (int kt2 = 0; kt2 < D / 16; ++kt2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(kbase + tile_off(jc + kld_row, kt2 * 16 + kld_hi * 8, SLAB), b0, b1, b2, b3);
                mma_16816(s[0], st.qa[kt2], b0, b1);
                mma_16816(s[1], st.qa[kt2], b2, b3);
                mma_16816(s[0], st.ql[kt2], b0, b1);
                mma_16816(s[1], st.ql[kt2], b2, b3);
                ldsm_x4(vbase + tile_off(jc + kld_row, kt2 * 16 + kld_hi * 8, SLAB), b0, b1, b2, b3);
                mma_16816(dp[0], ga[kt2], b0, b1);
                mma_16816(dp[1], ga[kt2], b2, b3);
            }
            float ds[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool isB = e & 2;
                    const int key = kc + n * 8 + qd + (e & 1), t = isB ? tB : tA;
                    const bool seen = key <= t && (key >= (isB ? loB : loA) || key < p.sinks) && (isB ? vB : vA);
                    ds[n][e] = seen ? fast_exp2(s[n][e] * c2 - (isB ? lseB : lseA)) * (dp[n][e] - (isB ? DB : DA)) : 0.f;
                }
            uint32_t dh[4], dl[4];
            split_q_pair(ds[0][0], ds[0][1], dh[0], dl[0]);
            split_q_pair(ds[0][2], ds[0][3], dh[1], dl[1]);
            split_q_pair(ds[1][0], ds[1][1], dh[2], dl[2]);
            split_q_pair(ds[1][2], ds[1][3], dh[3], dl[3]);
#pragma unroll
            for (int dp2 = 0; dp2 < D / 16; ++dp2) {
                uint32_t v0, v1, v2, v3;
                ldsm_x4_trans(kbase + tile_off(jc + vld_row, dp2 * 16 + vld_hi * 8, SLAB), v0, v1, v2, v3);
                mma_16816(st.o[2 * dp2], dh, v0, v1);
                mma_16816(st.o[2 * dp2 + 1], dh, v2, v3);
                mma_16816(st.o[2 * dp2], dl, v0, v1);
                mma_16816(st.o[2 * dp2 + 1], dl, v2, v3);
            }
        }
        __syncthreads();  // the slot is refilled by the next iteration's prefetch
        // the MMA's accumulators are truncated at every step: a long run of keys is summed up in memory
        if (i % DQ_RUN == DQ_RUN - 1 && i < nblk - 1) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half ? vB : vA) {
                    float *to = p.dq + (half ? rB : rA) * D + qd;
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) {
                        float2 y = i < DQ_RUN ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2 *>(to + 8 * e);
                        *reinterpret_cast<float2 *>(to + 8 * e) = make_float2(y.x + st.o[e][2 * half], y.y + st.o[e][2 * half + 1]);
                    }
                }
            st.reset();
        }
    }
    // dq = scale dQ; dq_raw = dq alpha; dalpha += x dq, dbeta += dq
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (!(half ? vB : vA))
            continue;
        const int t = half ? tB : tA, h = half ? hB : hA, hh = h - g * G;
        const long long off = b * q_bs + (static_cast<long long>(t) * p.Hq + h) * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const int dcol = i * 8 + qd;
            float2 y = nblk > DQ_RUN ? *reinterpret_cast<const float2 *>(p.dq + off + dcol) : make_float2(0.f, 0.f);
            const float dq0 = (y.x + st.o[i][2 * half]) * p.scale, dq1 = (y.y + st.o[i][2 * half + 1]) * p.scale;
            const float2 al = __ldg(reinterpret_cast<const float2 *>(p.alpha + h * D + dcol));
            *reinterpret_cast<float2 *>(p.dq + off + dcol) = make_float2(dq0 * al.x, dq1 * al.y);
            const float2 x = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(p.q + off + dcol));
            atomicAdd(&red[hh * D + dcol], x.x * dq0);
            atomicAdd(&red[hh * D + dcol + 1], x.y * dq1);
            atomicAdd(&red[G * D + hh * D + dcol], dq0);
            atomicAdd(&red[G * D + hh * D + dcol + 1], dq1);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += 128) {
        atomicAdd(p.dalpha + g * G * D + i, red[i]);
        atomicAdd(p.dbeta + g * G * D + i, red[G * D + i]);
    }
}

// ------------------------------------------------------------------ the sinks' dk, dv

// Rows t and sinks j <= t - window.  A CTA has one (sequence, query head) and a run of tokens, a warp 16 tokens at a
// time: the (up to 16) sinks on M and the tokens on N for S^T = K q^T and dP^T = V dO^T, whose fragments are then the
// operands of Y = dS^T q and dV = P^T dO (tokens on K).  Operands come straight from global memory, 16 bytes a
// lane, with the head dimension in the order in which they lie there.  More than 16 sinks: blockIdx.z.
constexpr int SK_M = 16;

template <int D>
__global__ void __launch_bounds__(128, 2) sink_keys_kernel(const SinkBwdParams p, int chunks, int count)
{
    constexpr int KK = D / 32;  // runs of 32 values: a lane has 8 of each row
    __shared__ __align__(16) uint4 ka_s[D / 16][32], va_s[D / 16][32];  // K, V as A fragments
    __shared__ __align__(16) float red[SK_M][2 * D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, rq = lane >> 2;
    const int chunk = blockIdx.x, bh = blockIdx.y, b = bh / p.Hq, h = bh % p.Hq, g = h / (p.Hq / p.Hkv);
    const int s0 = SK_M * blockIdx.z, ns = min(SK_M, count - s0);
    const int T = p.T;

    auto pair = [&](const orthros_bf16 *src, int j, int d) -> uint32_t {  // two values of a sink (zero behind the last)
        return j < ns ? *reinterpret_cast<const uint32_t *>(src + ((static_cast<long long>(b) * T + s0 + j) * p.Hkv + g) * D + d)
                      : 0u;
    };
    for (int x = threadIdx.x; x < D / 16 * 32; x += 128) {
        const int kt = x / 32, l = x % 32, d = 32 * (kt / 2) + 8 * (l & 3) + 4 * (kt & 1), j = l >> 2;
        ka_s[kt][l] = make_uint4(pair(p.k, j, d), pair(p.k, j + 8, d), pair(p.k, j, d + 2), pair(p.k, j + 8, d + 2));
        va_s[kt][l] = make_uint4(pair(p.v, j, d), pair(p.v, j + 8, d), pair(p.v, j, d + 2), pair(p.v, j + 8, d + 2));
    }
    __syncthreads();

    const int per = ((T + chunks - 1) / chunks + 63) / 64 * 64;
    const int t_begin = chunk * per, t_end = min(T, t_begin + per);
    const float c2 = p.scale * kLog2eF;
    float y[D / 8][4], dv[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[i][e] = dv[i][e] = 0.f;
    const long long stride = static_cast<long long>(p.Hq) * D;  // between tokens
    const long long row0 = static_cast<long long>(b) * T * p.Hq + h;
    for (int t0 = t_begin + 16 * warp; t0 < t_end; t0 += 64) {
        if (t0 + 15 - p.window < s0)
            continue;  // no row of these sees a sink behind its window
        uint4 Q[2][KK], L[2][KK], O[2][KK];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int t = t0 + rq + 8 * r;
                const long long off = row0 * D + t * stride + 32 * kk + 8 * c;
                const bool in = t < t_end;
                Q[r][kk] = in ? __ldg(reinterpret_cast<const uint4 *>(p.q_hi + off)) : make_uint4(0, 0, 0, 0);
                L[r][kk] = in ? __ldg(reinterpret_cast<const uint4 *>(p.q_lo + off)) : make_uint4(0, 0, 0, 0);
                O[r][kk] = in ? __ldg(reinterpret_cast<const uint4 *>(p.dO + off)) : make_uint4(0, 0, 0, 0);
            }
        float s[2][4], dp[2][4], lse[2][2], Dr[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[r][e] = dp[r][e] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = t0 + 8 * r + 2 * c + i;
                lse[r][i] = t < t_end ? p.lse[row0 + static_cast<long long>(t) * p.Hq] : 0.f;
                Dr[r][i] = t < t_end ? p.Drow[row0 + static_cast<long long>(t) * p.Hq] : 0.f;
            }
        }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const uint4 k0 = ka_s[2 * kk][lane], k1 = ka_s[2 * kk + 1][lane];
            const uint4 v0 = va_s[2 * kk][lane], v1 = va_s[2 * kk + 1][lane];
            const uint32_t ka0[4] = {k0.x, k0.y, k0.z, k0.w}, ka1[4] = {k1.x, k1.y, k1.z, k1.w};
            const uint32_t va0[4] = {v0.x, v0.y, v0.z, v0.w}, va1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mma_16816(s[r], ka0, Q[r][kk].x, Q[r][kk].y);
                mma_16816(s[r], ka1, Q[r][kk].z, Q[r][kk].w);
                mma_16816(s[r], ka0, L[r][kk].x, L[r][kk].y);
                mma_16816(s[r], ka1, L[r][kk].z, L[r][kk].w);
                mma_16816(dp[r], va0, O[r][kk].x, O[r][kk].y);
                mma_16816(dp[r], va1, O[r][kk].z, O[r][kk].w);
            }
        }
        uint32_t ph[4], pl[4], sh[4], sl[4];  // P and dS with the sinks on M, tokens on K
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int j = rq + 8 * hf;
                float pr[2], ds[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = t0 + 8 * r + 2 * c + i;
                    const bool seen = j < ns && t < t_end && s0 + j <= t - p.window;
                    const float e = fast_exp2(s[r][2 * hf + i] * c2 - lse[r][i]);
                    pr[i] = seen ? e : 0.f;
                    ds[i] = seen ? e * (dp[r][2 * hf + i] - Dr[r][i]) : 0.f;
                }
                split_q_pair(pr[0], pr[1], ph[2 * r + hf], pl[2 * r + hf]);
                split_q_pair(ds[0], ds[1], sh[2 * r + hf], sl[2 * r + hf]);
            }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                auto word = [e](uint4 u) { return e == 0 ? u.x : e == 1 ? u.y : e == 2 ? u.z : u.w; };
                const uint32_t x0 = movmatrix_trans(word(Q[0][kk])), x1 = movmatrix_trans(word(Q[1][kk]));
                mma_16816(y[4 * kk + e], sh, x0, x1);
                mma_16816(y[4 * kk + e], sl, x0, x1);
                mma_16816(y[4 * kk + e], sh, movmatrix_trans(word(L[0][kk])), movmatrix_trans(word(L[1][kk])));
                const uint32_t g0 = movmatrix_trans(word(O[0][kk])), g1 = movmatrix_trans(word(O[1][kk]));
                mma_16816(dv[4 * kk + e], ph, g0, g1);
                mma_16816(dv[4 * kk + e], pl, g0, g1);
            }
    }
    // the four warps' sums, added up in order
    for (int w = 0; w < 4; ++w) {
        if (warp == w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float *row = red[rq + 8 * hf];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const int d = 32 * (i / 4) + 8 * c + 2 * (i % 4);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        row[d + e] = (w ? row[d + e] : 0.f) + y[i][2 * hf + e];
                        row[D + d + e] = (w ? row[D + d + e] : 0.f) + dv[i][2 * hf + e];
                    }
                }
            }
        __syncthreads();
    }
    float *out = p.part + ((static_cast<long long>(blockIdx.z) * p.B * p.Hq + bh) * chunks + chunk) * SK_M * 2 * D;
    for (int x = threadIdx.x; x < SK_M * 2 * D; x += 128)
        out[x] = red[x / (2 * D)][x % (2 * D)];
}

// one CTA a sink of a (sequence, KV head), a thread a column of dk and of dv
template <int D>
__global__ void __launch_bounds__(2 * D) sink_join_kernel(const SinkBwdParams p, int chunks)
{
    const int j = blockIdx.x, bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv, G = p.Hq / p.Hkv, d = threadIdx.x;
    const float *src = p.part + (((static_cast<long long>(j / SK_M) * p.B + b) * p.Hq + g * G) * chunks * SK_M + j % SK_M) * 2 * D + d;
    float sum = 0.f;
#pragma unroll 8
    for (int i = 0; i < G * chunks; ++i)  // the heads' chunks follow one another
        sum += src[static_cast<long long>(i) * SK_M * 2 * D];
    const long long at = ((static_cast<long long>(b) * p.T + j) * p.Hkv + g) * D;
    if (d < D)
        p.dk[at + d] += p.scale * sum;
    else
        p.dv[at + d - D] += sum;
}

// ------------------------------------------------------------------ host side

// four waves of two CTAs on each of 152 SMs, from 64 tokens a CTA to 4096 (64 a warp's step: the accumulators are
// truncated at each)
int sink_chunks(int B, int T, int Hq)
{
    const int most = (T + 63) / 64, least = (T + 4095) / 4096, want = 1216 / (B * Hq);
    return want < least ? least : (want < most ? want : most);
}

template <int D, int G>
cudaError_t launch_dq(const SinkBwdParams &p, cudaStream_t stream)
{
    const int smem = 4 * (D / 64) * DQ_KEYS * 128 + 2 * G * D * 4 + 1024;
    auto kern = sink_dq_kernel<D, G>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    constexpr int TOK = DQ_ROWS / G;
    kern<<<dim3((p.T + TOK - 1) / TOK, p.B * p.Hkv), 128, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_t(const SinkBwdMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    const long long lanes = static_cast<long long>(p.B) * p.T * p.Hq * (D / 8);
    sink_rows_kernel<D><<<static_cast<unsigned>((lanes + 255) / 256), 256, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    switch (p.Hq / p.Hkv) {
    case 1: e = launch_dq<D, 1>(p, stream); break;
    case 2: e = launch_dq<D, 2>(p, stream); break;
    case 4: e = launch_dq<D, 4>(p, stream); break;
    case 8: e = launch_dq<D, 8>(p, stream); break;
    case 16: e = launch_dq<D, 16>(p, stream); break;
    default: e = cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || (e = launch_sink_dkv(D, maps, p, stream)) != cudaSuccess)
        return e;
    const int count = p.sinks < p.T - p.window ? p.sinks : p.T - p.window;  // sinks that some row sees behind its window
    if (count <= 0)
        return cudaSuccess;
    const int chunks = sink_chunks(p.B, p.T, p.Hq);
    sink_keys_kernel<D><<<dim3(chunks, p.B * p.Hq, (count + SK_M - 1) / SK_M), 128, 0, stream>>>(p, chunks, count);
    sink_join_kernel<D><<<dim3(count, p.B * p.Hkv), 2 * D, 0, stream>>>(p, chunks);
    return cudaGetLastError();
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t sink_bwd_workspace_bytes(int B, int T, int Hq, int D)
{
    const size_t rows = static_cast<size_t>(B) * T * Hq;
    return 2 * up256(2 * rows * D) + 2 * up256(4 * rows) +
           2 * static_cast<size_t>(B) * Hq * sink_chunks(B, T, Hq) * SK_M * 2 * D * sizeof(float);
}

void sink_bwd_workspace(SinkBwdParams &p, int D, void *workspace)
{
    const size_t rows = static_cast<size_t>(p.B) * p.T * p.Hq;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q_hi = reinterpret_cast<uint16_t *>(ws);
    p.q_lo = reinterpret_cast<uint16_t *>(ws += up256(2 * rows * D));
    p.lse = reinterpret_cast<float *>(ws += up256(2 * rows * D));
    p.Drow = reinterpret_cast<float *>(ws += up256(4 * rows));
    p.part = reinterpret_cast<float *>(ws + up256(4 * rows));
}

cudaError_t launch_sink_bwd(int D, const SinkBwdMaps &maps, const SinkBwdParams &p, cudaStream_t stream)
{
    return D == 128 ? launch_t<128>(maps, p, stream) : launch_t<64>(maps, p, stream);
}

}  // namespace orthros
