#include "qg_attn.cuh"
namespace qg {
bool attn_wide_supported(int) { return false; }
qg_status attn_wide_launch(const AttnArgs &, bool, cudaStream_t) { return QG_EUNSUPPORTED; }
unsigned int read_status_attn_tc(bool) { return 0; }
}  // namespace qg
