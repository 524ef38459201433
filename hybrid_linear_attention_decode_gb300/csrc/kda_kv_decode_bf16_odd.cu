// kda_kv_decode_bf16_odd.cu -- the attention kernels of kda_kv_decode.cuh for bf16, head_dim no multiple of 64.
#include "kda_kv_decode.cuh"

namespace kda {
namespace kv {

int launch_decode_bf16_odd(const DecodeP &p, cudaStream_t st) {
    return launch_decode_of<false, false>(p, st);
}

}  // namespace kv
}  // namespace kda
