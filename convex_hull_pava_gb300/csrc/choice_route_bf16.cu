// A router's choice of experts by scores of __nv_bfloat16.
#include "choice_route.cuh"

namespace isodev {

template cudaError_t route_rows<__nv_bfloat16>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);

}  // namespace isodev
