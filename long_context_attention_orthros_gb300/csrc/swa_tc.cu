// swa_tc.cu -- the tensor-memory kernel of base-stream sliding-window attention, Eq. (4)
// (swa_tc.cuh), without sinks.
#include "swa_tc.cuh"

namespace orthros {

bool swa_tc_supported(int D, int G, int window) { return swa_tc_fits<false>(D, G, window); }

cudaError_t launch_swa_tc(int D, int G, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                          const CUtensorMap &o, const SwaParams &p, int num_sms, cudaStream_t stream)
{
    (void)o;  // rows are stored straight from registers (p.o)
    return launch_swa_tc_any<false>(D, G, q, k, v, p, num_sms, stream);
}

}  // namespace orthros
