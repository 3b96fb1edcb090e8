// Attention over a cache of e4m3 codes.
#include "kv8_attn.cuh"

namespace qg {

cudaError_t launch_kv8_attn_e4m3(const Kv8AttnParams &p, cudaStream_t st) { return launch_code<QGEMV_CODE_E4M3>(p, st); }

}  // namespace qg
