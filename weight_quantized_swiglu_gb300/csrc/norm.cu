// norm.cu -- the norms before and after a block (norm.cuh), z and y bf16.
#include "norm.cuh"

namespace qmlp {

cudaError_t launch_norm(const NormArgs& a, bool t_f16, bool r_f32, bool backward, cudaStream_t s) {
    if (t_f16) return launch_norm_f16(a, r_f32, backward, s);
    return r_f32 ? launch_tr<__nv_bfloat16, float>(a, backward, s)
                 : launch_tr<__nv_bfloat16, __nv_bfloat16>(a, backward, s);
}

QMLP_BOUNDS_UNIT(norm)

}  // namespace qmlp
