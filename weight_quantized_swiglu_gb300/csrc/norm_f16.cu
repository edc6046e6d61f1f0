// norm_f16.cu -- the norms before and after a block (norm.cuh), z and y fp16.
#include "norm.cuh"

namespace qmlp {

cudaError_t launch_norm_f16(const NormArgs& a, bool r_f32, bool backward, cudaStream_t s) {
    return r_f32 ? launch_tr<__half, float>(a, backward, s) : launch_tr<__half, __half>(a, backward, s);
}

QMLP_BOUNDS_UNIT(norm_f16)

}  // namespace qmlp
