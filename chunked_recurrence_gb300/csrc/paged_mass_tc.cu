#include "paged_attn.cuh"
#include "paged_mass.cuh"
namespace gdn {
bool paged_mass_tc_supported(const gdn_cache_shape &, const void *, const void *) { return false; }
size_t paged_mass_tc_workspace(const gdn_cache_shape &) { return 0; }
gdn_status paged_mass_tc(MassArgs &, const gdn_cache_shape &, int32_t, uint32_t, void *, cudaStream_t) {
  return GDN_ERR_UNSUPPORTED;
}
}  // namespace gdn
