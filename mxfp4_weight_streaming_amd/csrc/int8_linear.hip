// int8_linear.hip -- the int8 product.
#include "int8_launch.hpp"
#include "moe_internal.hpp"

namespace moe {

hipError_t launch_int8_linear(const Int8Args& a, hipStream_t s) { return launch_int8(a, NoAdapters{}, s); }

}  // namespace moe
