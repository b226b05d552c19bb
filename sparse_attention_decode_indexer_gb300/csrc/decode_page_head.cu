// decode_page_head.cu -- the decode attention of the page_head formats (e4m3 or
// int8 codes, one fp32 scale per page and KV head for K and for V).
#include "decode_kernel.cuh"

namespace ssa {

int decode_max_ctas_page_head(const Dims& d, int num_sms) {
  return num_sms * (d.kind == SSA_KV_INT8_PAGE_HEAD ? ctas_per_sm<SSA_KV_INT8_PAGE_HEAD>(d.P)
                                                    : ctas_per_sm<SSA_KV_E4M3_PAGE_HEAD>(d.P));
}

cudaError_t launch_decode_page_head(const DecodeArgs& a, cudaStream_t s) {
  DecodeParams p = decode_params(a);
  switch (a.d->kind) {
    case SSA_KV_E4M3_PAGE_HEAD: return launch_decode_k<SSA_KV_E4M3_PAGE_HEAD>(a, p, decode_mode(a), s);
    case SSA_KV_INT8_PAGE_HEAD: return launch_decode_k<SSA_KV_INT8_PAGE_HEAD>(a, p, decode_mode(a), s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ssa
