// A router's choice of experts by scores of __half.
#include "choice_route.cuh"

namespace isodev {

template cudaError_t route_rows<__half>(const RouteArgs&, int64_t*, int32_t*, float*, cudaStream_t);

}  // namespace isodev
