// Attention over a cache of int8 codes.
#include "kv8_attn.cuh"

namespace qg {

cudaError_t launch_kv8_attn_int8(const Kv8AttnParams &p, cudaStream_t st) { return launch_code<QGEMV_CODE_INT8>(p, st); }

}  // namespace qg
