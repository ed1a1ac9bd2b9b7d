// Attention of a decode step through a sliding window: attn_kernel<kWin> (lq_attn_decode.cuh), compiled by itself so that
// the two halves of the kernel's variants compile side by side.

#include "lq_attn_decode.cuh"

namespace lq {

lq_status run_attn_window(lq_handle h, AttnParams& P, int bits, int D, bool bf16, Scratch s) { return run_shape<true>(h, P, bits, D, bf16, s); }

}  // namespace lq
