// tree_tc.cu -- both streams of a tree of drafted tokens over a KV cache on the 5th-generation tensor cores: the
// form of tree_step.cu for more query rows a KV head than its warp MMAs keep up with (rows_tc.cuh).
//
// A CTA takes its share of the list of key blocks (tree.cuh); a piece is its blocks of one segment.  A piece that is
// its whole segment leaves as bf16, another as one partial (max, sum, o), which tree_join_kernel joins.  One tile of
// 128 rows goes as KEYS2, more as ROWS2.  A segment costs its start and end, some 7 us, as much as 10 blocks: with 5
// counted 16 nodes over 2 x 131072 rows took 188 us, with 10 185, with 14 185.
#include "rows_tc.cuh"
#include "tree_rows.cuh"

namespace orthros {

namespace {

template <int D, int TR>
struct TreeJob {
    using Params = TreeParams;
    using Maps = TreeMaps;
    struct Where {
        long long it, it1, W, n;  // the next place, the share's end, places and CTAs
    };
    struct Piece {
        TreeCursor<TR, TREE_TC_COST> cur;  // its segment; the place behind it
        int first, m;                      // its blocks: first .. first + m - 1
        int plain0, plain1;
        int alone;                         // the whole segment
        long long slot;                    // of its partial
    };
    struct See : TreeRow {
        bool none;
    };

    static __device__ __forceinline__ void share(const Params &p, Piece &seed, Where &where)
    {
        const TreeShare<TR, TREE_TC_COST> sh = tree_share<TR, TREE_TC_COST>(p, blockIdx.x, gridDim.x);
        if ((threadIdx.x & 31) == 0) {
            where = {sh.it0, sh.it1, sh.W, sh.n};
            seed.cur = sh.cur;
        }
    }
    static __device__ __forceinline__ void next(const Params &p, const Piece &from, Piece &to, Where &where)
    {
        to.cur = from.cur;
        int m = 0;
        long long it = where.it;
        while (m == 0 && it < where.it1) {  // a share may begin or end with a segment's empty places
            if (to.cur.r == to.cur.places())
                to.cur.next_segment(p);
            const int at = to.cur.r, all = to.cur.places();
            const long long left = where.it1 - it;
            const int places = static_cast<int>(all - at < left ? all - at : left);
            const int first = max(at - TREE_TC_COST, 0);
            m = max(at + places - TREE_TC_COST - first, 0);
            const long long s0 = it - at + TREE_TC_COST, s1 = it - at + all;
            const long long c0 = ((s0 + 1) * where.n - 1) / where.W, c1 = (s1 * where.n - 1) / where.W;
            to.first = first;
            to.alone = c0 == c1;
            to.plain0 = 0;  // a copy's blocks of cached rows
            to.plain1 = to.cur.base || to.cur.s.full ? 0 : min(m, max(to.cur.s.len / TREE_KB - first, 0));
            to.slot = 2 * static_cast<long long>(blockIdx.x) + (blockIdx.x == c0 ? 1 : 0);
            it += places;
            to.cur.r = at + places;
        }
        where.it = it;
        to.m = m;
    }
    static __device__ __forceinline__ void place(const Piece &c, int &g, int &b)
    {
        g = c.cur.g;
        b = c.cur.b;
    }
    static __device__ __forceinline__ int row_of(const Params &, const Piece &c, int x) { return c.cur.first_row(c.first + x); }
    static __device__ __forceinline__ int keys(const Params &p) { return p.L_max; }
    static __device__ __forceinline__ const CUtensorMap *map(const Maps &m, bool v, int j0)
    {
        return j0 == -1 ? (v ? &m.vt : &m.kt) : (v ? &m.v : &m.k);
    }
    static __device__ __forceinline__ void span(const Params &p, const Piece &c, int j0, int &end, int &lo, int &first)
    {
        end = j0 >= 0 ? c.cur.s.len - j0 : c.cur.s.n;
        tree_span(p, c.cur.s, c.cur.base, lo, first);
    }
    static __device__ __forceinline__ const orthros_bf16 *query(const Params &p, const Piece &c, int r)
    {
        const int G = p.Hq / p.Hkv, row = c.cur.tile * TR + r, node = row / G;
        if (node >= c.cur.s.n)
            return nullptr;
        return (c.cur.base ? p.q_new : p.qc_new) +
               ((static_cast<long long>(c.cur.b) * p.N + node) * p.Hq + c.cur.g * G + row % G) * D;
    }
    static __device__ __forceinline__ void vectors(const Params &p, const Piece &c, const float *&alpha, const float *&beta)
    {
        alpha = c.cur.base ? p.alpha : p.alpha_c;
        beta = c.cur.base ? p.beta : p.beta_c;
    }
    static __device__ __forceinline__ See see(const Params &p, const Piece &c, int r)
    {
        const int node = (c.cur.tile * TR + r) / (p.Hq / p.Hkv);
        const TreePaths paths = tree_paths(p.parent + static_cast<long long>(c.cur.b) * p.N, c.cur.s.n);
        See s;
        static_cast<TreeRow &>(s) = tree_row(p, c.cur.s, paths, c.cur.base, node);
        s.none = c.cur.s.full || ((paths.bad >> (node & 63)) & 1);
        if (r == 0 && !c.cur.base && c.cur.g == 0 && c.cur.tile == 0) {
            const int len = __ldcg(p.cache_len + c.cur.b);
            if (len < 0 || len > p.L_max)
                record_error(p.dev_err, ORTHROS_DEVERR_CACHE_FULL);
            else if (c.cur.s.full || paths.bad != 0)
                record_error(p.dev_err, ORTHROS_DEVERR_POSITION);
        }
        return s;
    }
    static __device__ __forceinline__ unsigned long long mask(const Params &, const Piece &c, const See &s, int j0)
    {
        if (j0 < 0)
            return s.mask;
        // lo - j0 does not overflow: both lie in [0, 2^31)
        return bits_below(c.cur.s.len - j0) & (~bits_below(s.lo - j0) | bits_below(s.first - j0));
    }
    static __device__ __forceinline__ RowOut out(const Params &p, const Piece &c, const See &s, int r)
    {
        const int G = p.Hq / p.Hkv, row = c.cur.tile * TR + r, node = row / G;
        RowOut o = {nullptr, nullptr, nullptr, nullptr, s.none};
        if (node >= c.cur.s.n)
            return o;
        if (c.alone) {
            o.row = (c.cur.base ? p.o : p.oc) +
                    ((static_cast<long long>(c.cur.b) * p.N + node) * p.Hq + c.cur.g * G + row % G) * D;
        } else {
            o.part = p.part_o + (c.slot * TR + r) * D;
            o.ml = p.part_ml + c.slot * TR + r;
        }
        return o;
    }
};

}  // namespace

cudaError_t launch_tree_tc(int D, int tr, const TreeMaps &maps, const TreeParams &p, int ctas, cudaStream_t stream)
{
    if (D == 128)
        return tr == 128 ? launch_rows_tc<128, false, TreeJob>(maps, p, ctas, stream)
                         : launch_rows_tc<128, true, TreeJob>(maps, p, ctas, stream);
    return tr == 128 ? launch_rows_tc<64, false, TreeJob>(maps, p, ctas, stream)
                     : launch_rows_tc<64, true, TreeJob>(maps, p, ctas, stream);
}

}  // namespace orthros
