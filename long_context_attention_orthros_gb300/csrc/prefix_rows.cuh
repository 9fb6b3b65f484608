// prefix_rows.cuh -- where the query rows of a batch over a shared prefix come from and where their
// partials go: row = copy * G + head within one KV head, copies counted through the batch.
#pragma once

#include "kernels.cuh"

namespace orthros {

struct PrefixRow {
    const orthros_bf16 *q;  // NULL: no such row, or a copy whose position is out of range
    long long slot;         // of the first part; -1: no such row
    int head;
};

template <int G>
__device__ __forceinline__ PrefixRow prefix_row(const PrefixAttnParams &p, long long row, int g, int D)
{
    PrefixRow r = {nullptr, -1, g * G};
    const long long bi = row / G;
    if (bi >= static_cast<long long>(p.B) * p.T_out)
        return r;
    const int b = static_cast<int>(bi / p.T_out), i = static_cast<int>(bi % p.T_out), h = static_cast<int>(row % G);
    r.head = g * G + h;
    r.slot = (static_cast<long long>(b) * p.Hkv + g) * p.T_out * G + static_cast<long long>(i) * G + h;
    if (p.pos == nullptr || (p.pos[bi] >= 0 && p.pos[bi] < p.T_kv))
        r.q = p.qc + b * p.qc_bstride + (static_cast<long long>(i) * p.Hq + r.head) * D;
    return r;
}

}  // namespace orthros
