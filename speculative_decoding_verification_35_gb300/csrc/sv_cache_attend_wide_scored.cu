// spec_cache_attend_scored for chunks of more than 64 rows.
#include "sv_cache_attend_wide.cuh"

namespace sv {
namespace cache {

template cudaError_t launch_wide<true>(const Params&, int, int, int, cudaStream_t);

}  // namespace cache
}  // namespace sv
