// The pass over the own rows of a decoding step, 16-bit caches.
#include "fa_serve_own.cuh"

namespace fa {

cudaError_t launch_own_16(const ServeArgs& a, int D, bool f16, int sms, bool after, cudaStream_t s) {
  return f16 ? launch_own_k<kF16>(a, D, true, sms, after, s) : launch_own_k<kBf16>(a, D, false, sms, after, s);
}

}  // namespace fa
