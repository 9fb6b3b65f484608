// swa_sink_tc.cu -- the tensor-memory kernel of the base stream (swa_tc.cuh) with attention sinks.
#include "swa_tc.cuh"

namespace orthros {

bool swa_sink_tc_supported(int D, int G, int window) { return swa_tc_fits<true>(D, G, window); }

cudaError_t launch_swa_sink_tc(int D, int G, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                               const SwaParams &p, int num_sms, cudaStream_t stream)
{
    return launch_swa_tc_any<true>(D, G, q, k, v, p, num_sms, stream);
}

}  // namespace orthros
