// tree_rows.cuh -- what one query row of a drafted tree sees, and where its results go.
#pragma once

#include "tree.cuh"

namespace orthros {

struct TreeRow {
    unsigned long long mask;  // the tree's nodes that it sees
    int lo, first;            // cached row j counts iff j >= lo or j < first (and j < len)
};

// Row `node` of a tree with paths t; a row that is not live, or hangs below a bad parent, sees nothing.  Whole warp.
__device__ __forceinline__ TreeRow tree_row(const TreeParams &p, const TreeSeq &s, const TreePaths &t, int base, int node)
{
    TreeRow r;
    r.mask = t.of(node < 0 || node > 63 ? 0 : node);
    r.lo = 0x7fffffff;
    r.first = 0;
    if (node < 0 || node >= s.n || s.full || ((t.bad >> node) & 1)) {
        r.mask = 0;
        return r;
    }
    r.lo = 0;
    if (base) {
        // ancestors come before their descendants: the path in order of depth is its set in order of bits
        const int count = __popcll(r.mask), far = count - p.window, kept = p.sinks - s.len;
        const int lo = s.len + count - p.window;  // len + depth - window + 1
        r.lo = lo > 0 ? lo : 0;
        r.first = p.sinks;
        if (far > 0) {
            unsigned long long near = r.mask, past = r.mask;
            for (int k = 0; k < far; ++k)
                near &= near - 1;
            for (int k = 0; k < kept && past != 0; ++k)
                past &= past - 1;
            r.mask = near | (r.mask & ~past);
        }
    }
    return r;
}

// rows of the cache whose V counts for some row of a segment: j >= lo or j < first (and j < len)
__device__ __forceinline__ void tree_span(const TreeParams &p, const TreeSeq &s, int base, int &lo, int &first)
{
    lo = base && s.len - p.window + 1 > 0 ? s.len - p.window + 1 : 0;
    first = base ? p.sinks : 0;
}

}  // namespace orthros
