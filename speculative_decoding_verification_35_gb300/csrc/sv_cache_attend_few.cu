// spec_cache_attend for chunks of up to 64 rows.
#include "sv_cache_attend_few.cuh"

namespace sv {
namespace cache {

template cudaError_t launch_few<false>(Params&, int, int, int, cudaStream_t);

}  // namespace cache
}  // namespace sv
