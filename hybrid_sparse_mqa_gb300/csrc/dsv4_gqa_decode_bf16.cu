// dsv4_gqa_decode_bf16.cu - the one-token attention kernel for caches of bf16
// rows (dsv4_gqa_decode.cuh).
#include "dsv4_gqa_decode.cuh"

namespace dsv4 {
namespace gqa {
int launch_decode_bf16(const DecodeParams& p, int head_dim, int nt, void* stream) {
    return launch_decode_kind<DSV4_GQA_BF16, DSV4_GQA_BF16>(p, head_dim, nt, stream);
}
}  // namespace gqa
}  // namespace dsv4
