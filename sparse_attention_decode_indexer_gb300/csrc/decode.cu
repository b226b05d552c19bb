// decode.cu -- the decode attention of the bf16 and per-token fp8 formats, and
// the choice of the format (the page_head formats live in a translation unit
// of their own so that the two compile in parallel).
#include "decode_kernel.cuh"

namespace ssa {

int decode_max_ctas(const Dims& d, int num_sms) {
  switch (d.kind) {
    case SSA_KV_BF16: return num_sms * ctas_per_sm<SSA_KV_BF16>(d.P);
    case SSA_KV_FP8_E4M3: return num_sms * ctas_per_sm<SSA_KV_FP8_E4M3>(d.P);
    default: return decode_max_ctas_page_head(d, num_sms);
  }
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s) {
  const int kind = a.d->kind;
  if (kind != SSA_KV_BF16 && kind != SSA_KV_FP8_E4M3) return launch_decode_page_head(a, s);
  DecodeParams p = decode_params(a);
  return kind == SSA_KV_BF16 ? launch_decode_k<SSA_KV_BF16>(a, p, decode_mode(a), s)
                             : launch_decode_k<SSA_KV_FP8_E4M3>(a, p, decode_mode(a), s);
}

}  // namespace ssa
