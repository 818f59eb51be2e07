// The pass over the own rows of a decoding step, 8-bit caches.
#include "fa_serve_own.cuh"

namespace fa {

cudaError_t launch_own_e4m3(const ServeArgs& a, int D, bool q_f16, int sms, bool after, cudaStream_t s) {
  return launch_own_k<kE4m3>(a, D, q_f16, sms, after, s);
}

}  // namespace fa
