// ops_api.h — host pieces of the operators' C entries shared with api.cu.
#pragma once

#include "ops.cuh"

namespace moe {

moe_status check_route_desc(const moe_route_desc *d);
RouteArgs route_args(const moe_route_desc &d);  // without the buffers

}  // namespace moe
