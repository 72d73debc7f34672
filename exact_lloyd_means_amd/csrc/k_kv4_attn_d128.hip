// k_kv4_attn_d128.hip -- cache attention for heads of 128 dimensions.
#include "k_kv4_attn.inl"

namespace fk {

hipError_t launch_kv4_attn_d128(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s) {
    return attn_d<128>(a, p, dtype, s);
}

}  // namespace fk
