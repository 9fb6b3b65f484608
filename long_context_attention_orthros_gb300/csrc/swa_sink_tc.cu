// swa_sink_tc.cu -- the tensor-memory kernel of the base stream (swa_tc.cuh) with attention sinks: where a tile's band
// and the sinks' block fit tensor memory (4 x 16384 tokens of 32/8 heads, d = 128, window 128: 285 us, by
// swa_wide.cu's tiles 783).  2 x 131072 tokens take 1093 us, 4.9 of 6.7 TB/s (950 without sinks); a tile's chain bounds it.
#include "swa_tc.cuh"

namespace orthros {

bool swa_sink_tc_supported(int D, int G, int window) { return swa_tc_fits<true>(D, G, window); }

cudaError_t launch_swa_sink_tc(int D, int G, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                               const SwaParams &p, int num_sms, cudaStream_t stream)
{
    return launch_swa_tc_any<true>(D, G, q, k, v, p, num_sms, stream);
}

}  // namespace orthros
