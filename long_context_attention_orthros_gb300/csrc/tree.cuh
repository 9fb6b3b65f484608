// tree.cuh -- a tree of drafted tokens over a KV cache: launch parameters, the paths of its nodes, and the
// list of key blocks that the kernels share out.
//
// Node i of a sequence hangs below node parent[i] < i, or below the last cached row (-1), and stands at
// position cache_len + depth.  Query rows of one KV head are node * G + head.  A segment is one (sequence,
// KV head, stream, tile of rows); its keys come in blocks of 64: for the copies every cached row, for the
// base tokens the block of the sinks (where the window does not reach back to it) and the blocks of the
// window of the shallowest node, and for both one block with the tree's own rows.  Segments laid end to
// end form one list of W places that all CTAs share alike, as in the decode step over a block list.
#pragma once

#include "serve.cuh"

namespace orthros {

constexpr int TREE_KB = 64;       // keys of a block
constexpr int TREE_MAX_NODES = 64;
constexpr int TREE_MAX_SINKS = 32;

struct TreeParams {
    const orthros_bf16 *q_new, *qc_new;  // [B, N, Hq, d]
    const int32_t *parent;               // [B, N]
    const int32_t *nodes;                // [B] or NULL (N)
    const int32_t *cache_len;            // [B]
    const float *alpha, *beta, *alpha_c, *beta_c;
    orthros_bf16 *o, *oc;  // [B, N, Hq, d]
    float *part_o;         // [2 * CTAs][TR][D]
    float2 *part_ml;       // [2 * CTAs][TR]
    int32_t *dev_err;
    int B, N, Hq, Hkv, L_max, window, sinks;
    float qscale;
};
struct TreeMaps {
    CUtensorMap k, v, kt, vt;  // the cache; the tree's own rows (boxes of 64 x 1 x 64)
};

size_t tree_workspace_bytes(int B, int N, int L_max, int Hq, int Hkv, int D);
cudaError_t launch_tree(int D, const TreeMaps &maps, TreeParams p, void *workspace, cudaStream_t stream);

// the tensor-memory kernel; tr: rows of a tile, 128 or 256
constexpr int TREE_TC_CTAS = 152;  // one on each of 152 SMs
constexpr int TREE_TC_COST = 10;   // what a segment costs it beside its blocks
cudaError_t launch_tree_tc(int D, int tr, const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream);

struct TreeAcceptParams {
    const orthros_bf16 *k_new, *v_new;  // [B, N, Hkv, d]
    const int32_t *parent, *node;       // [B, N], [B]
    const int32_t *nodes;               // [B] or NULL (N)
    orthros_bf16 *k_cache, *v_cache;    // [B, L_max, Hkv, d]
    int32_t *cache_len, *path;          // [B], [B, N]
    int32_t *dev_err;
    int B, N, L_max, row;  // row: Hkv * d values
};
cudaError_t launch_tree_accept(const TreeAcceptParams &p, cudaStream_t stream);

// ------------------------------------------------------------------ paths

// The paths of up to 64 nodes, two a lane (lane and lane + 32), as sets of nodes: bit j of a node's set is
// node j on its path, itself included.  Whole warp; log2(n) rounds of path doubling.
struct TreePaths {
    unsigned long long m[2];  // of nodes lane, lane + 32
    unsigned long long bad;   // nodes below which a parent is not an earlier node (all lanes)

    __device__ __forceinline__ unsigned long long of(int node) const  // any lane's node; whole warp
    {
        const unsigned long long a = __shfl_sync(0xffffffffu, m[0], node & 31);
        const unsigned long long b = __shfl_sync(0xffffffffu, m[1], node & 31);
        return node & 32 ? b : a;
    }
};

__device__ __forceinline__ TreePaths tree_paths(const int32_t *parent, int n)
{
    const int lane = threadIdx.x & 31;
    TreePaths t;
    int up[2];
    bool wrong[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        up[h] = i < n ? __ldg(parent + i) : -1;
        wrong[h] = up[h] < -1 || up[h] >= i;
        if (wrong[h])
            up[h] = -1;
        t.m[h] = 1ull << i;
    }
    const unsigned long long roots = __ballot_sync(0xffffffffu, wrong[0]) |
                                     static_cast<unsigned long long>(__ballot_sync(0xffffffffu, wrong[1])) << 32;
    for (int s = 1; s < n; s <<= 1) {
        unsigned long long more[2];
        int next[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = up[h] < 0 ? 0 : up[h];
            more[h] = t.of(j);
            const int a = __shfl_sync(0xffffffffu, up[0], j & 31), b = __shfl_sync(0xffffffffu, up[1], j & 31);
            next[h] = j & 32 ? b : a;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (up[h] >= 0) {
                t.m[h] |= more[h];
                up[h] = next[h];
            }
    }
    t.bad = __ballot_sync(0xffffffffu, (t.m[0] & roots) != 0) |
            static_cast<unsigned long long>(__ballot_sync(0xffffffffu, (t.m[1] & roots) != 0)) << 32;
    return t;
}

// ------------------------------------------------------------------ the list

// what a sequence's length and number of nodes make of it
struct TreeSeq {
    int len, n;      // cached rows, live nodes
    int full;        // a length or a number of nodes out of range: its rows (all N, where the number is) become zeros
    int tiles;       // of query rows
    int nc, nb;      // blocks of a copy's segment, of a base segment: the tree's block is the last of each
    int sink;        // a base segment begins with the sinks' block (block 0 of the cache)
    int wb0;         // first block of the window
};

template <int TR>  // rows of a tile
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b)
{
    TreeSeq s;
    s.len = __ldcg(p.cache_len + b);
    s.n = p.nodes != nullptr ? __ldcg(p.nodes + b) : p.N;
    const bool sized = s.n >= 0 && s.n <= p.N;
    s.n = sized ? s.n : p.N;
    s.full = s.len < 0 || s.len > p.L_max || !sized;
    s.len = s.full ? 0 : s.len;
    s.tiles = (s.n * (p.Hq / p.Hkv) + TR - 1) / TR;
    s.tiles = s.full ? max(s.tiles, 1) : s.tiles;  // a tree without nodes has a tile all the same, which reports the length
    const int blocks = (s.len + TREE_KB - 1) / TREE_KB;
    const int lo = s.len - p.window + 1;  // first row of the window of a node at depth 0 (window >= 1: no overflow)
    s.wb0 = lo > 0 ? lo / TREE_KB : 0;
    s.wb0 = s.wb0 > blocks ? blocks : s.wb0;
    s.sink = p.sinks > 0 && s.wb0 > 0;
    s.nc = blocks + 1;
    s.nb = s.sink + blocks - s.wb0 + 1;
    return s;
}

// COST: what a segment costs beside its blocks, in blocks: every segment begins with so many empty places
template <int TR, int COST>
struct TreeCursor {
    int b, g, base, tile, r;  // place r of the segment; block r - COST
    TreeSeq s;
    __device__ __forceinline__ int blocks() const { return base ? s.nb : s.nc; }
    __device__ __forceinline__ int places() const { return COST + blocks(); }
    __device__ __forceinline__ long long seq_places(int Hkv) const
    {
        return static_cast<long long>(s.nc + s.nb + 2 * COST) * s.tiles * Hkv;
    }
    // the caller knows that there is one
    __device__ __forceinline__ void next_segment(const TreeParams &p)
    {
        r = 0;
        if (++tile < s.tiles)
            return;
        tile = 0;
        if (!base) {
            base = 1;
            return;
        }
        base = 0;
        if (++g < p.Hkv)
            return;
        g = 0;
        do
            s = tree_seq<TR>(p, ++b);
        while (s.tiles == 0 && b + 1 < p.B);
    }
    // first cached row of block i of the segment; -1: the tree's own rows
    __device__ __forceinline__ int first_row(int i) const
    {
        if (i == blocks() - 1)
            return -1;
        if (!base)
            return i * TREE_KB;
        return s.sink && i == 0 ? 0 : (s.wb0 + i - s.sink) * TREE_KB;
    }
};

template <int TR, int COST>
struct TreeShare {
    long long W, n, it0, it1;  // places, CTAs that have some, this one's
    TreeCursor<TR, COST> cur;
};

// Whole warp: CTA c of at most n takes places it0 .. it1 - 1, and its cursor stands at it0.
template <int TR, int COST>
__device__ __forceinline__ TreeShare<TR, COST> tree_share(const TreeParams &p, long long c, long long n)
{
    const int lane = threadIdx.x & 31;
    TreeShare<TR, COST> sh;
    TreeCursor<TR, COST> cur{};
    long long W = 0;
    for (int b = lane; b < p.B; b += 32) {
        cur.s = tree_seq<TR>(p, b);
        W += cur.seq_places(p.Hkv);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        W += __shfl_xor_sync(0xffffffffu, W, off);
    sh.W = W;
    sh.n = n < W ? n : W;
    sh.it0 = c < sh.n ? c * W / sh.n : W;
    sh.it1 = c < sh.n ? (c + 1) * W / sh.n : W;
    sh.cur = TreeCursor<TR, COST>{};
    if (sh.it0 >= sh.it1)
        return sh;
    long long it = sh.it0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        long long w = 0;
        if (b0 + lane < p.B) {
            cur.s = tree_seq<TR>(p, b0 + lane);
            w = cur.seq_places(p.Hkv);
        }
        long long inc = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off)
                inc += y;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, inc > it);
        if (here != 0) {
            const int f = __ffs(here) - 1;
            it -= __shfl_sync(0xffffffffu, inc - w, f);
            sh.cur.b = b0 + f;
            break;
        }
        it -= __shfl_sync(0xffffffffu, inc, 31);
    }
    sh.cur.s = tree_seq<TR>(p, sh.cur.b);
    const int pc = sh.cur.s.nc + COST, pb = sh.cur.s.nb + COST, tiles = sh.cur.s.tiles;
    const long long per = static_cast<long long>(pc + pb) * tiles;
    sh.cur.g = static_cast<int>(it / per);
    long long r = it % per;
    sh.cur.base = r >= static_cast<long long>(pc) * tiles;
    r -= sh.cur.base ? static_cast<long long>(pc) * tiles : 0;
    sh.cur.tile = static_cast<int>(r / (sh.cur.base ? pb : pc));
    sh.cur.r = static_cast<int>(r % (sh.cur.base ? pb : pc));
    return sh;
}

}  // namespace orthros
