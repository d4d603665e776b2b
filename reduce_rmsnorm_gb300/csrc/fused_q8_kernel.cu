// The fused step with its output in e4m3 with scales: the instances of
// fused_forms.cuh whose rows end in 8 bits.
#define TW_FUSED_Q8 1
#include "fused_forms.cuh"

namespace tw {

int launch_fused_q8(const FusedArgs& a, cudaStream_t stream, int sm_budget) {
  return launch_forms(a, stream, sm_budget, nullptr);
}

int read_fused_q8_error(int reset, unsigned* code) { return read_ring_error(reset, code); }

}  // namespace tw
