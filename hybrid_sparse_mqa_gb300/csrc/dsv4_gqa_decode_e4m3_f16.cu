// dsv4_gqa_decode_e4m3_f16.cu - the one-token attention kernel for caches of e4m3
// rows beside f16 queries (dsv4_gqa_decode.cuh).
#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {
int launch_decode_e4m3_f16(const DecodeParams& p, int head_dim, int nt, void* stream) {
    return launch_decode_kind<DSV4_GQA_E4M3, DSV4_GQA_F16>(p, head_dim, nt, stream);
}
}  // namespace gqa
}  // namespace dsv4
