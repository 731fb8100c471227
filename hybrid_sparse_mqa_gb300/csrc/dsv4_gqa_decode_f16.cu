// dsv4_gqa_decode_f16.cu - the one-token attention kernel for caches of f16
// rows (dsv4_gqa_decode.cuh).
#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {
int launch_decode_f16(const DecodeParams& p, int head_dim, int nt, void* stream) {
    return launch_decode_kind<DSV4_GQA_F16, DSV4_GQA_F16>(p, head_dim, nt, stream);
}
}  // namespace gqa
}  // namespace dsv4
