// prefix_rows.cuh -- where the query rows of a batch over a shared prefix come from and where their
// partials go: row = copy * G + head within one KV head, copies counted through the batch.
#pragma once

#include "serve.cuh"

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
    // in 32 bits (the launcher refuses more rows): a thread does this for dozens of rows
    const uint32_t row32 = static_cast<uint32_t>(row), bi = row32 / G, h = row32 % G;
    if (bi >= static_cast<uint32_t>(p.B) * static_cast<uint32_t>(p.T_out))
        return r;
    const uint32_t b = p.T_out == 1 ? bi : bi / static_cast<uint32_t>(p.T_out), i = bi - b * p.T_out;
    r.head = g * G + static_cast<int>(h);
    r.slot = (static_cast<long long>(b) * p.Hkv + g) * p.T_out * G + static_cast<long long>(i) * G + h;
    if (p.pos == nullptr || (p.pos[bi] >= 0 && p.pos[bi] < p.T_kv))
        r.q = p.qc + b * p.qc_bstride + (static_cast<long long>(i) * p.Hq + r.head) * D;
    return r;
}

}  // namespace orthros
