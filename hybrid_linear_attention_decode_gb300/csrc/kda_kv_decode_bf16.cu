// kda_kv_decode_bf16.cu -- the attention kernels of kda_kv_decode.cuh for bf16, head_dim a multiple of 64.
#include "kda_kv_decode.cuh"

namespace kda {
namespace kv {

int launch_decode_bf16(const DecodeP &p, cudaStream_t st) {
    return launch_decode_of<false, true>(p, st);
}

}  // namespace kv
}  // namespace kda
