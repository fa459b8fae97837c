// decay_attn_bf16.hip -- bf16 variants of the decay attention kernel (decay_attn.hpp).
#include "decay_attn.hpp"

namespace ssm {
hipError_t launch_decay_attn_bf16(const DaArgs &a, int da_padded, bool dots, bool state_only, hipStream_t s) {
  return launch_da_type<bf16>(a, da_padded, dots, state_only, s);
}
}  // namespace ssm
