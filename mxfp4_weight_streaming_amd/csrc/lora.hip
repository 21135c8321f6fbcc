// lora.hip -- host launchers of the kernels in lora_kernels.hpp, alone and behind
// the int8 product.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beside_choice.hpp"
#include "lora_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

namespace {

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;   // of a launch

int rank_tiles(int r) { return r > 16 ? 2 : 1; }   // of 16, that a workgroup takes

int64_t shrink_grid(const LoraArgs& a, const LoraPlan& p)
{
    return ceil_div(a.M, 16) * ceil_div(a.r, 16 * rank_tiles(a.r)) * p.shrink_slots;
}

int64_t expand_grid(const LoraArgs& a, const LoraPlan& p)
{
    return ceil_div(a.M, 16) * ceil_div(a.N, 256) * p.expand_slots;
}

// Whether the launches are possible: known before the first of them.
bool fits(const LoraArgs& a)
{
    const LoraPlan p = lora_plan(a.M, a.N, a.K, a.r);
    if (p.few) return a.M * ceil_div(a.N, 256) * 256 <= kMaxThreads;
    return shrink_grid(a, p) * 512 <= kMaxThreads && expand_grid(a, p) * 256 <= kMaxThreads;
}

template <bool BASE32, bool F32, int RK, bool SHORT = false>
hipError_t expand_tiles(LoraArgs a, const LoraPlan& p, hipStream_t s)
{
    a.slots = p.expand_slots;
    const int64_t grid = expand_grid(a, p);
    const auto kernel = lora_expand_kernel<BASE32, F32, RK, SHORT>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <bool BASE32, bool F32>
hipError_t expand(const LoraArgs& a, const LoraPlan& p, hipStream_t s)
{
    if (a.r < 8) return expand_tiles<BASE32, F32, 1, true>(a, p, s);
    if (a.r <= 32) return expand_tiles<BASE32, F32, 1>(a, p, s);
    return a.r <= 64 ? expand_tiles<BASE32, F32, 2>(a, p, s) : expand_tiles<BASE32, F32, 4>(a, p, s);
}

template <bool BASE32, bool F32, bool FUSED>
hipError_t few(LoraArgs a, const LoraPlan& p, hipStream_t s)
{
    a.near = p.near;
    // (FUSED calls have 16 ranks at most)
    const auto kernel = a.r <= 8    ? lora_few_kernel<BASE32, F32, FUSED, 1>
                        : a.r <= 16 ? lora_few_kernel<BASE32, F32, FUSED, 2>
                        : a.r <= 32 ? lora_few_kernel<BASE32, F32, false, 4>
                        : a.r <= 64 ? lora_few_kernel<BASE32, F32, false, 8>
                                    : lora_few_kernel<BASE32, F32, false, 16>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(a.M * ceil_div(a.N, 256))), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t shrink(LoraArgs a, const LoraPlan& p, hipStream_t s)
{
    if (p.few) {
        const auto kernel = a.K < 8 ? lora_shrink_few_kernel<true> : lora_shrink_few_kernel<false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.M * ceil_div(a.r, 16))), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    a.slots = p.shrink_slots;
    const int64_t grid = shrink_grid(a, p);
    hipLaunchKernelGGL((rank_tiles(a.r) == 2 ? lora_shrink_kernel<2> : lora_shrink_kernel<1>), dim3((unsigned)grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

// The rows of a that stand among `M` of a call.
template <bool BASE32, bool F32>
hipError_t add(const LoraArgs& a, int64_t M, hipStream_t s)
{
    LoraPlan p = lora_plan(a.M, a.N, a.K, a.r);
    // (a row's sums have one order wherever it stands among them)
    p.few = lora_plan(M, a.N, a.K, a.r).few;
    p.fused = p.few && p.fused;
    if (p.fused) return few<BASE32, F32, true>(a, p, s);
    const hipError_t e = shrink(a, p, s);
    if (e != hipSuccess) return e;
    return p.few ? few<BASE32, F32, false>(a, p, s) : expand<BASE32, F32>(a, p, s);
}

}  // namespace

size_t lora_add_workspace(int64_t M, int r) { return align256((size_t)M * lora_padded(r) * 4); }

size_t lora_product_workspace(int64_t M, int64_t N, int r)
{
    return lora_add_workspace(M, r) + (size_t)std::min<int64_t>(M, lora_product_rows(N)) * N * 4;
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s)
{
    if (!fits(a)) return hipErrorInvalidConfiguration;
    return a.out_type == kTypeF32 ? add<true, true>(a, a.M, s) : add<false, false>(a, a.M, s);
}

// The product in fp32 first, into out where that is fp32 and else into the
// workspace, 256 MB at a time; then the adapters on top of it.
hipError_t launch_int8_linear_lora(const Int8Args& p, const LoraArgs& a, hipStream_t s)
{
    if (!fits(a)) return hipErrorInvalidConfiguration;   // (what fits here is fewer tiles than a product may have)
    const bool f32 = a.out_type == kTypeF32;
    const int64_t step = f32 ? a.M : lora_product_rows(a.N);
    for (int64_t m = 0; m < a.M; m += step) {
        Int8Args g = p;
        LoraArgs l = a;
        g.M = l.M = std::min(step, a.M - m);
        g.a += (size_t)m * p.K;
        g.a_scale += m;
        l.x += (size_t)m * a.K;
        l.ids += m;
        if (f32) {
            l.base = l.out;
        } else {
            g.out = reinterpret_cast<uint8_t*>(a.u) + lora_add_workspace(a.M, a.r);
            l.base = g.out;
            l.out = static_cast<uint16_t*>(a.out) + (size_t)m * a.N;
        }
        g.out_type = kTypeF32;
        hipError_t e = launch_int8_linear(g, s);
        if (e != hipSuccess) return e;
        e = f32 ? add<true, true>(l, a.M, s) : add<true, false>(l, a.M, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
