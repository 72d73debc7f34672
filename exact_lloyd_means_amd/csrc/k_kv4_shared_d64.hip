// Attention of shared prefixes, head dimension 64.
#include "k_kv4_shared.inl"

namespace fk {
hipError_t launch_kv4_shared_d64(const AttnArgs& a, const SharedArgs& s, const SharedPlan& p, int dtype,
                                 hipStream_t st) {
    return shared_d<64>(a, s, p, dtype, st);
}
}  // namespace fk
