// int8_lora.hip -- the int8 product with the tokens' adapters: their u first, then
// the product, which adds B u before its one rounding.
#include "int8_launch.hpp"
#include "moe_internal.hpp"

namespace moe {

hipError_t launch_int8_linear_lora(const Int8Args& p, const LoraArgs& a, hipStream_t s)
{
    const hipError_t e = launch_lora_shrink(a, s);
    return e == hipSuccess ? launch_int8(p, a, s) : e;
}

}  // namespace moe
