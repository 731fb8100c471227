// dsv4_gqa_decode_e2m1_f16.cu - the one-token attention kernel for caches of 4-bit
// codes and f16 queries (lists: dsv4_gqa_decode4.cuh, a cluster per segment:
// dsv4_gqa_decode.cuh).
#include "dsv4_gqa_decode4.cuh"

namespace dsv4 {
namespace gqa {
int launch_decode_e2m1_f16(const DecodeParams& p, int head_dim, int nt, void* stream) {
    return launch_decode4<DSV4_GQA_F16>(p, head_dim, nt, stream);
}
}  // namespace gqa
}  // namespace dsv4
