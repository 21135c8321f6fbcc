// lora_kernels.hpp -- low-rank adapters of many requests (gfx950): token m has
// adapter i = ids[m], and
//   u[m] = scale[i] A[i] x[m]             (r values, fp32; kept with zeros behind
//                                          them up to a multiple of 32, rp)
//   out[m] = round(base[m] + B[i] u[m])   base alone where i is no adapter
//
// Tokens are taken as they stand, 16 at a time, which is a matrix instruction's
// width: a request's tokens follow one another, so 16 of them have few adapters.
// Each adapter among them is multiplied by all 16, and each token takes its own
// adapter's result, so nothing of another adapter, infinities and NaN included,
// reaches it.  Where tiles are few, their adapters are dealt to several
// workgroups (slots).
//
// v_mfma_f32_16x16x32_bf16: lane l gives row l % 16, values 8 (l / 16).. of both
// operands, and gets rows 4 (l / 16) + 0..3 of the first and row l % 16 of the
// second, the token.  u goes into the second product as three bf16 numbers that
// add up to the fp32 one (8 bits each), so it is not rounded.
#pragma once

#include "around_common.hpp"
#include "beside_choice.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_half __attribute__((aligned(2)));    // at any bf16
typedef u32x2 u32x2_half __attribute__((aligned(2)));
typedef f32x4 f32x4_word __attribute__((aligned(4)));    // at any fp32
typedef u32x4 u32x4_word __attribute__((aligned(4)));

// The adapter of token m, or -1; -2 for what is no token.
__device__ __forceinline__ int adapter_of(const LoraArgs& g, int64_t m)
{
    if (m >= g.M) return -2;
    const int i = g.ids[m];
    return i >= 0 && i < g.L ? i : -1;
}

// Calls f(adapter, mask of the tokens that have it) for each adapter among the
// wave's 16 tokens (-1, none, too) that falls to `slot` of `slots` (a power of
// two).
template <typename F>
__device__ __forceinline__ void each_adapter(int id, uint32_t slot, int slots, F f)
{
    uint32_t todo = (uint32_t)__ballot(id >= -1) & 0xFFFFu;
    for (uint32_t d = 0; todo != 0; ++d) {
        const int i = __builtin_amdgcn_readlane(id, (int)__builtin_ctz(todo));
        const uint32_t mask = (uint32_t)__ballot(id == i) & 0xFFFFu;
        todo &= ~mask;
        if ((d & (uint32_t)(slots - 1)) == slot) f(i, mask);
    }
}

// Workgroups are dealt to the 8 XCDs in turn, each with a cache of its own: the
// tile of workgroup b of n, so that an XCD has consecutive tiles, which share
// tokens and their adapter's rows.
__device__ __forceinline__ uint32_t tile_of(uint32_t b, uint32_t n)
{
    const uint32_t xcd = b & 7;
    return n / 8 * xcd + min(xcd, n & 7) + (b >> 3);
}

// Values k .. k + 7 of a row of n, and zeros behind it: a part of them comes from
// the row's last 8, shifted down; rows shorter than 8 are read value by value.
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t* row, int k, int n)
{
    if (n >= 8) {
        const int at = min(k, n - 8), by = k - at;       // values to drop
        const u32x4 v = *reinterpret_cast<const u32x4_half*>(row + at);
        const uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
        const int bits = (by & 3) * 16;
        const uint64_t a = by & 4 ? hi : lo, b = by & 4 ? 0 : hi;
        const uint64_t x = by >= 8 ? 0 : bits == 0 ? a : a >> bits | b << (64 - bits), y = by >= 8 ? 0 : b >> bits;
        return u32x4{(uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32)};
    }
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint32_t v = row[min(k + i, n - 1)];
        d[i >> 1] |= (k + i < n ? v : 0) << (16 * (i & 1));
    }
    return u32x4{d[0], d[1], d[2], d[3]};
}

// The same in the form that costs nothing before the values are there: where 8
// would pass the row's end they are its last 8, of which the other factor counts
// each once (drop_first, place_of).  SHORT: a row of less than 8.
template <bool SHORT>
__device__ __forceinline__ u32x4 load_last8(const uint16_t* row, int k, int n)
{
    if constexpr (SHORT) return load_bf16x8(row, k, n);
    return *reinterpret_cast<const u32x4_half*>(row + min(k, n - 8));
}

// 0 for the first n values (any n of 8 or more: all).
__device__ __forceinline__ u32x4 drop_first(u32x4 v, int n)
{
    const uint64_t lo = n >= 4 ? 0 : ~0ull << (16 * n), hi = n >= 8 ? 0 : n > 4 ? ~0ull << (16 * (n & 3)) : ~0ull;
    return u32x4{v.x & (uint32_t)lo, v.y & (uint32_t)(lo >> 32), v.z & (uint32_t)hi, v.w & (uint32_t)(hi >> 32)};
}

// Where rank k stands in a row of u: r = 8 c + d ranks have the last d at the end
// of their 8, behind zeros, as B's last 8 are read.
__device__ __forceinline__ int u_gap(int r) { return r > 8 && (r & 7) != 0 ? 8 - (r & 7) : 0; }
__device__ __forceinline__ int place_of(int k, int r) { return k + (k >= (r & ~7) ? u_gap(r) : 0); }

// acc + the sum of 8 products, one after another in fp32.
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float acc)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        acc = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), acc);
        acc = fmaf(__uint_as_float(a[e] & 0xFFFF0000u), __uint_as_float(b[e] & 0xFFFF0000u), acc);
    }
    return acc;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two fp32 values as three pairs of bf16 that add up to them: each takes the 8
// leading bits of what is left (cut off, as rounding could pass the largest
// number).  An infinity or a NaN is the first alone.
struct Split3 {
    uint32_t v[3];
};

__device__ __forceinline__ Split3 split_pair(float a, float b)
{
    Split3 s;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const uint32_t lo = __float_as_uint(a) & 0xFFFF0000u, hi = __float_as_uint(b) & 0xFFFF0000u;
        s.v[p] = lo >> 16 | hi;
        a -= __uint_as_float(lo);
        b -= __uint_as_float(hi);
        a = a == a ? a : 0.0f;
        b = b == b ? b : 0.0f;
    }
    return s;
}

// u of ranks k .. k + 3 of a token to their places, zeros where there is none; the
// 16 behind a last tile that ends in the middle of 32 are cleared with it.
__device__ __forceinline__ void store_u(const LoraArgs& g, int64_t m, int k, f32x4 u)
{
    if (k >= g.rp) return;
    float* row = g.u + (size_t)m * g.rp;
    const int last = g.r & ~7, gap = u_gap(g.r);
    if (gap != 0 && k >= last && k < last + 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (k + e < g.r) row[k + e + gap] = u[e];
        if (k == last)
            for (int e = 0; e < gap; ++e) row[last + e] = 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = k + e < g.r ? u[e] : 0.0f;
        *reinterpret_cast<f32x4*>(row + k) = u;
    }
    if (k / 16 * 16 + 16 >= g.r && k + 16 < g.rp) *reinterpret_cast<f32x4*>(row + k + 16) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// ---------------------------------------------------------------------------
// u of 16 tokens and RR x 16 rows of A: 8 waves share K, 64 values at a time,
// and their sums meet in LDS.  A matrix operand wants 16 rows side by side in
// neighbouring lanes, which as loads are 16 lines of memory at 16 bytes each (a
// lane a clock: 2,048 tokens of rank 64 16 us); here 8 lanes read a row's 128
// bytes, and the operands are read back from the wave's own 2 KB of LDS a tile
// (chunk c of row r at c ^ r % 8, so that neither side has bank conflicts): 8 us,
// bound by latencies: ids, then A, then the waves' sums, with one workgroup a
// compute unit, and by the tiles that two adapters share (3 us).  Rank 16: 5 us.
// ---------------------------------------------------------------------------
template <int RR>
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs g)
{
    constexpr int W = 8, U = 5;                          // waves, and chunks of 64 whose loads are in flight
    __shared__ u32x4 stage[W][1 + RR][16 * 8];
    __shared__ f32x4 part[W][RR][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, quarter = lane >> 4, load_row = lane >> 3, chunk = lane & 7;
    const uint32_t ranks = (g.r + 16 * RR - 1) / (16 * RR), tiles = (uint32_t)((g.M + 15) / 16) * ranks;
    const uint32_t slot = blockIdx.x / tiles, tile = tile_of(blockIdx.x - slot * tiles, tiles);   // (most slots are idle, and come last)
    const int64_t m0 = (int64_t)(tile / ranks) * 16;
    const int r0 = (int)(tile % ranks) * 16 * RR;
    const int id = adapter_of(g, m0 + row);
    // (addresses as a uniform part and 32 bits of a lane's own: 64 bits each would
    // take the registers that the loads in flight need)
    const uint16_t* x = g.x + (size_t)m0 * g.K;
    uint32_t xo[2], ao[RR][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        xo[h] = (uint32_t)min((int64_t)(h * 8 + load_row), g.M - 1 - m0) * (uint32_t)g.K;
#pragma unroll
        for (int q = 0; q < RR; ++q) ao[q][h] = (uint32_t)min(q * 16 + h * 8 + load_row, g.r - 1 - r0) * (uint32_t)g.K;
    }
    const int chunks = g.K / 64, s0 = chunks * wave / W, s1 = chunks * (wave + 1) / W;
    // x's values are asked for before the adapter is known, and where they are
    // all a wave needs they serve every adapter of the tile.
    u32x4 xv[U][2];
    int held = s0;
    auto load_x = [&](int s) {
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                xv[j][h] = *reinterpret_cast<const u32x4_half*>(x + min(s + j, s1 - 1) * 64 + (xo[h] + chunk * 8));
        held = s;
    };
    if (s0 < s1) load_x(s0);
    __builtin_amdgcn_sched_barrier(0);
    each_adapter(id, slot, g.slots, [&](int i, uint32_t mask) {
        if (i < 0) return;
        const uint16_t* a = g.a + ((size_t)i * g.r + r0) * g.K;
        f32x4 acc[RR] = {};
        auto multiply = [&](const u32x4 (&xj)[2], const u32x4 (&aj)[RR][2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = (h * 8 + load_row) * 8 + (chunk ^ (load_row & 7));
                stage[wave][0][at] = xj[h];
#pragma unroll
                for (int q = 0; q < RR; ++q) stage[wave][1 + q][at] = aj[q][h];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = row * 8 + ((h * 4 + quarter) ^ (row & 7));
                const u32x4 b = stage[wave][0][at];
#pragma unroll
                for (int q = 0; q < RR; ++q) acc[q] = mfma(stage[wave][1 + q][at], b, acc[q]);
            }
        };
        for (int s = s0; s < s1; s += U) {
            if (s != held) load_x(s);
            u32x4 av[U][RR][2];
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int q = 0; q < RR; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        av[j][q][h] = *reinterpret_cast<const u32x4_half*>(a + min(s + j, s1 - 1) * 64 + (ao[q][h] + chunk * 8));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s + j < s1) multiply(xv[j], av[j]);
        }
        if (wave == W - 1 && chunks * 64 < g.K) {
            u32x4 xj[2], aj[RR][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                xj[h] = load_bf16x8(x + xo[h], chunks * 64 + chunk * 8, g.K);
#pragma unroll
                for (int q = 0; q < RR; ++q) aj[q][h] = load_bf16x8(a + ao[q][h], chunks * 64 + chunk * 8, g.K);
            }
            multiply(xj, aj);
        }
#pragma unroll
        for (int q = 0; q < RR; ++q) part[wave][q][lane] = acc[q];
        __syncthreads();
        if (wave < RR && (mask >> row & 1)) {
            f32x4 sum = part[0][wave][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += part[w][wave][lane];
            const float scale = g.scale != nullptr ? g.scale[i] : 1.0f;
            store_u(g, m0 + row, r0 + wave * 16 + quarter * 4, sum * scale);
        }
        __syncthreads();
    });
}

// ---------------------------------------------------------------------------
// u of one token and 16 rows of A, for few tokens: a wave takes 4 rows of A,
// all lanes along them, so that few tokens of many adapters read each adapter
// once and nothing else; all loads of 2,560 values are in flight at once.  64
// tokens of rank 16, K 2,560: 2.7 us, a launch and one round of latency.
// ---------------------------------------------------------------------------
constexpr int kDotRows = 4, kDotLoads = kLoraStep / 512;   // rows, and loads of each in flight

struct DotLoads {
    u32x4 x[kDotLoads], a[kDotRows][kDotLoads];
};

// Rows r0 .. r0 + 3 of adapter i and token m, from value k0.
template <bool SHORT>
__device__ __forceinline__ void dot_load(const LoraArgs& g, int i, int64_t m, int r0, int k0, DotLoads& v)
{
    const uint16_t* x = g.x + (size_t)m * g.K;
    const uint16_t* a = g.a + (size_t)i * g.r * g.K;
#pragma unroll
    for (int c = 0; c < kDotLoads; ++c) {
        const int k = k0 + (c * 64 + (threadIdx.x & 63)) * 8;
        v.x[c] = load_last8<SHORT>(x, k, g.K);
#pragma unroll
        for (int q = 0; q < kDotRows; ++q) v.a[q][c] = load_last8<SHORT>(a + (size_t)min(r0 + q, g.r - 1) * g.K, k, g.K);
    }
    __builtin_amdgcn_sched_barrier(0);                   // (left alone, some are asked for one by one, where they are used)
}

template <bool SHORT>
__device__ __forceinline__ void dot_add(const LoraArgs& g, int k0, DotLoads& v, float (&acc)[kDotRows])
{
    if (!SHORT && k0 + kLoraStep > g.K)
#pragma unroll
        for (int c = 0; c < kDotLoads; ++c)
            v.x[c] = drop_first(v.x[c], max(k0 + (c * 64 + (int)(threadIdx.x & 63)) * 8 - (g.K - 8), 0));
#pragma unroll
    for (int q = 0; q < kDotRows; ++q)
#pragma unroll
        for (int c = 0; c < kDotLoads; ++c) acc[q] = dot8(v.a[q][c], v.x[c], acc[q]);
}

__device__ __forceinline__ f32x4 dot_sum(const LoraArgs& g, int i, const float (&acc)[kDotRows])
{
    const float scale = g.scale != nullptr ? g.scale[i] : 1.0f;
    f32x4 u;
#pragma unroll
    for (int q = 0; q < kDotRows; ++q) u[q] = wave_sum(acc[q]) * scale;
    return u;
}

template <bool SHORT>
__device__ __forceinline__ f32x4 dot_rows(const LoraArgs& g, int i, int64_t m, int r0)
{
    float acc[kDotRows] = {};
    for (int k0 = 0; k0 < g.K; k0 += kLoraStep) {
        DotLoads v;
        dot_load<SHORT>(g, i, m, r0, k0, v);
        dot_add<SHORT>(g, k0, v, acc);
    }
    return dot_sum(g, i, acc);
}

template <bool SHORT>
__global__ __launch_bounds__(256) void lora_shrink_few_kernel(LoraArgs g)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), ranks = (g.r + 15) / 16;
    const int64_t m = blockIdx.x / ranks;
    const int i = adapter_of(g, m), r0 = (int)(blockIdx.x % ranks) * 16 + wave * 4;
    if (i < 0) return;
    f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r0 < g.r) u = dot_rows<SHORT>(g, i, m, r0);
    if ((threadIdx.x & 63) == 0) store_u(g, m, r0, u);
}

// ---------------------------------------------------------------------------
// out of 16 tokens and 256 channels, 64 a wave.  u's three parts stand in LDS;
// they are the first operand and B's rows the second, row q of tile j being
// channel 4 q + j, so that a lane gets 4 consecutive channels of 4 tokens, and 16
// lanes a token's 64: base and out are read and written 128 bytes (bf16) a row.
// B's rows are loaded by 4 lanes each, 64 bytes, and dealt to the operand's lanes
// through LDS (loaded in the operand's order, a lane a clock, 2,048 tokens of
// rank 128 took 2 us more).  RK: steps of 32 ranks; SHORT: less than 8 ranks.
// 2,048 tokens and 2,560 channels of bf16: rank 16 9.5 us, rank 64 11; 21 MB of
// base and out are 4.5 us at a copy's rate, and the rest latencies (ids, B, LDS)
// of 5 workgroups a compute unit, 4 at a time.  Two to eight tiles of tokens in
// turn, B's rows kept, were no faster.
// ---------------------------------------------------------------------------
template <bool F32>
struct Row4 {
    uint32_t d[F32 ? 4 : 2];
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (F32) return __uint_as_float(d[i]);
        return __uint_as_float(i & 1 ? d[i >> 1] & 0xFFFF0000u : d[i >> 1] << 16);
    }
};

// 4 consecutive values from `at`, of which n (may be 0 or less) are the row's.
template <bool F32>
__device__ __forceinline__ Row4<F32> load_row4(const void* p, size_t at, int n)
{
    Row4<F32> v = {};
    if (n >= 4) {
        if constexpr (F32) {
            const u32x4 d = *reinterpret_cast<const u32x4_word*>(static_cast<const float*>(p) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) v.d[i] = d[i];
        } else {
            const u32x2 d = *reinterpret_cast<const u32x2_half*>(static_cast<const uint16_t*>(p) + at);
            v.d[0] = d.x;
            v.d[1] = d.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) {
                if constexpr (F32) v.d[i] = static_cast<const uint32_t*>(p)[at + i];
                else v.d[i >> 1] |= (uint32_t) static_cast<const uint16_t*>(p)[at + i] << (16 * (i & 1));
            }
    }
    return v;
}

template <bool F32>
__device__ __forceinline__ Row4<F32> round_row4(const float (&v)[4])
{
    Row4<F32> r;
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i)
        r.d[i] = F32 ? __float_as_uint(v[i]) : f32_to_bf16_bits(v[2 * i]) | f32_to_bf16_bits(v[2 * i + 1]) << 16;
    return r;
}

template <bool F32>
__device__ __forceinline__ void store_row4(void* p, size_t at, int n, const Row4<F32>& v)
{
    if (n >= 4) {
        if constexpr (F32) *reinterpret_cast<u32x4_word*>(static_cast<float*>(p) + at) = u32x4{v.d[0], v.d[1], v.d[2], v.d[3]};
        else *reinterpret_cast<u32x2_half*>(static_cast<uint16_t*>(p) + at) = u32x2{v.d[0], v.d[1]};
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) {
                if constexpr (F32) static_cast<uint32_t*>(p)[at + i] = v.d[i];
                else static_cast<uint16_t*>(p)[at + i] = (uint16_t)(v.d[i >> 1] >> (16 * (i & 1)));
            }
    }
}

// Where 16 bytes c of a row of 4 RK of them stand, so that the lanes that LDS
// serves together, 16 rows' operands, meet no bank twice.
template <int RK>
__device__ __forceinline__ int swizzled(int row, int c)
{
    return row * 4 * RK + (c ^ (RK == 1 ? row >> 1 & 3 : RK == 2 ? row & 7 : row));
}

template <bool BASE32, bool F32, int RK, bool SHORT>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs g)
{
    __shared__ u32x4 stage[4][4 * RK][64], us[3][16 * 4 * RK];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, quarter = lane >> 4;
    const uint32_t tn = (uint32_t)((g.N + 255) / 256), tiles = (uint32_t)((g.M + 15) / 16) * tn;
    const uint32_t slot = blockIdx.x / tiles, tile = tile_of(blockIdx.x - slot * tiles, tiles);
    const int64_t m0 = (int64_t)(tile / tn) * 16, n0 = (int64_t)(tile % tn) * 256 + wave * 64, n = n0 + row * 4;
    const int left = (int)max((int64_t)0, min((int64_t)4, g.N - n));
    const int id = adapter_of(g, m0 + row);
    if (slot > 0) {
        bool any = false;
        each_adapter(id, slot, g.slots, [&](int, uint32_t) { any = true; });
        if (!any) return;
    }
    // What a tile reads is asked for at once: u, base (all of it before the first
    // store, which could change it for all the compiler knows, base may be out),
    // and B's rows for the first token's adapter.
    constexpr int UQ = (RK + 1) / 2;                     // quads of u a thread
    const int quads = g.rp / 4;
    f32x4 uq[UQ];
#pragma unroll
    for (int i = 0; i < UQ; ++i) {
        const int q = min((int)threadIdx.x + 256 * i, 16 * quads - 1), t = q / quads;
        uq[i] = *reinterpret_cast<const f32x4*>(g.u + (size_t)min(m0 + t, g.M - 1) * g.rp + 4 * (q - t * quads));
    }
    Row4<BASE32> base[4] = {};
    if (g.base != nullptr)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            base[e] = load_row4<BASE32>(g.base, (size_t)min(m0 + quarter * 4 + e, g.M - 1) * g.N + n, left);
    u32x4 bv[4][RK];
    auto load_b = [&](int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t* b = g.b + ((size_t)i * g.N + min(n0 + (lane >> 2) * 4 + j, g.N - 1)) * g.r;
#pragma unroll
            for (int k = 0; k < RK; ++k) bv[j][k] = load_last8<SHORT>(b, 32 * k + (lane & 3) * 8, g.r);
        }
    };
    int held = slot == 0 ? __builtin_amdgcn_readlane(id, 0) : -1;
    if (held >= 0) load_b(held);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < UQ; ++i) {
        const int q = threadIdx.x + 256 * i, t = q / quads, c = q - t * quads;
        if (q >= 16 * quads) break;
        const Split3 lo = split_pair(uq[i][0], uq[i][1]), hi = split_pair(uq[i][2], uq[i][3]);
#pragma unroll
        for (int p = 0; p < 3; ++p) reinterpret_cast<u32x2*>(&us[p][swizzled<RK>(t, c >> 1)])[c & 1] = u32x2{lo.v[p], hi.v[p]};
    }
    lds_barrier();
    float o[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[e][j] = base[e].get(j);
    uint32_t own = 0, bare = 0;
    each_adapter(id, slot, g.slots, [&](int i, uint32_t mask) {
        own |= mask;
        if (i < 0) {
            bare = mask;
            return;
        }
        if (i != held) load_b(held = i);
        f32x4 acc[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < RK; ++k) stage[wave][j * RK + k][swizzled<1>(lane >> 2, lane & 3)] = bv[j][k];
#pragma unroll
        for (int k = 0; k < RK; ++k) {
            if (k * 32 >= g.rp) break;                   // (ranks 65 to 96)
            u32x4 bw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) bw[j] = stage[wave][j * RK + k][swizzled<1>(row, quarter)];
#pragma unroll
            for (int p = 2; p >= 0; --p) {
                // (a token of another adapter has its own u here, and drops the result)
                const u32x4 uv = us[p][swizzled<RK>(row, 4 * k + quarter)];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = mfma(uv, bw[j], acc[j]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[e][j] = mask >> (quarter * 4 + e) & 1 ? o[e][j] + acc[j][e] : o[e][j];
    });
    Row4<F32> v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = round_row4<F32>(o[e]);
    // (a token without an adapter keeps base's bits: nothing was added to them, and
    // bf16's are the upper halves that they were, where rounding would change a
    // signalling NaN)
    if constexpr (!BASE32 && !F32)
        if (bare != 0)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t same = __float_as_uint(o[e][2 * i]) >> 16 | (__float_as_uint(o[e][2 * i + 1]) & 0xFFFF0000u);
                    v[e].d[i] = bare >> (quarter * 4 + e) & 1 ? same : v[e].d[i];
                }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (own >> (quarter * 4 + e) & 1) store_row4<F32>(g.out, (size_t)(m0 + quarter * 4 + e) * g.N + n, left, v[e]);
}

// ---------------------------------------------------------------------------
// out of one token and 256 channels, 64 a wave: for few tokens, whose lanes a
// tile of 16 would leave idle.  L lanes share a row of B, 8 values each, so that
// a wave's load is one piece of memory (a thread a row is 64 pieces: 63 tokens of
// rank 118 and 11,708 channels 48 us, now 17); L loads give each lane one
// channel, number (64 / L) (lane % L) + lane / L.  A row's last values are read
// with those before them, which count once.  Workgroups of the same channels
// follow one another, on one XCD where B is large (near).  FUSED: every workgroup
// computes its token's u itself, which saves a launch: one token of rank 16, 2,560
// to 2,560, 3.6 us, of which a launch is 1.6 and the rest ids, A and x, and the
// sums' reduction.  There a token's workgroups follow one another on an XCD, so
// that A comes from its L2 after the first (in turn over all XCDs, by number, 51
// tokens took 7.1 us where 48 took 4.7, now 4.6, and 25 of K 8,192 13.1, now 7.7).  Four tokens and 157,184
// channels, 25.5 MB: 7.3 us with the launch before it, 3.5 TB/s.
// ---------------------------------------------------------------------------
template <bool BASE32, bool F32, bool FUSED, int L>
__global__ __launch_bounds__(256) void lora_few_kernel(LoraArgs g)
{
    __shared__ float us[kMaxLoraRank];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = lane % L, group = lane / L;
    const uint32_t M = (uint32_t)g.M, tn = (uint32_t)((g.N + 255) / 256);
    const uint32_t tile = FUSED || g.near ? tile_of(blockIdx.x, gridDim.x) : blockIdx.x;
    const int64_t m = FUSED ? tile / tn : tile % M;
    const int64_t n0 = (int64_t)(FUSED ? tile % tn : tile / M) * 256 + wave * 64, n = n0 + part * (64 / L) + group;
    const int i = __builtin_amdgcn_readfirstlane(adapter_of(g, m));
    const size_t at = (size_t)m * g.N + min(n, g.N - 1);
    // (asked for in any case, so that it is not waited for behind a branch)
    const void* src = g.base != nullptr ? g.base : BASE32 == F32 ? g.out : g.ids;
    const size_t from = g.base != nullptr || BASE32 == F32 ? at : 0;
    const uint32_t base = BASE32 ? static_cast<const uint32_t*>(src)[from] : static_cast<const uint16_t*>(src)[from];
    float d = 0.0f;
    if (i >= 0) {
        const int first = min(part * 8, max(g.r - 8, 0));   // the lane's ranks are first .. first + 7
        u32x4 bv[L];
#pragma unroll
        for (int s = 0; s < L; ++s) {
            const uint16_t* b = g.b + ((size_t)i * g.N + min(n0 + s * (64 / L) + group, g.N - 1)) * g.r;
            bv[s] = L > 1 ? *reinterpret_cast<const u32x4_half*>(b + first) : load_bf16x8(b, 0, g.r);
        }
        if constexpr (FUSED) {                           // (K is 8 or more)
            const int r0 = wave * 4;                     // (and r is 16 at most)
            f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
            if (g.K <= kLoraStep) {                      // all at once: a loop would first wait for what is in flight
                DotLoads v;
                float acc[kDotRows] = {};
                dot_load<false>(g, i, m, r0, 0, v);
                dot_add<false>(g, 0, v, acc);
                u = dot_sum(g, i, acc);
            } else {
                u = dot_rows<false>(g, i, m, r0);
            }
            if (lane < 4 && r0 + lane < g.r) us[r0 + lane] = lane == 0 ? u[0] : lane == 1 ? u[1] : lane == 2 ? u[2] : u[3];
        } else {
            for (int q = threadIdx.x; q < g.r; q += 256) us[q] = g.u[m * g.rp + place_of(q, g.r)];
        }
        __syncthreads();
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = us[first + e];                     // (first + 7 < 128, the array's size)
            asm("" : "+v"(v));                           // (a load for a select alone becomes a branch)
            u[e] = first + e >= part * 8 && first + e < g.r ? v : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < L; ++s) {
            float v = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v = fmaf(u[e], __uint_as_float(e & 1 ? bv[s][e >> 1] & 0xFFFF0000u : bv[s][e >> 1] << 16), v);
            v = group_sum<L>(v);
            d = part == s ? v : d;
        }
    }
    if (n >= g.N) return;
    // (a token without an adapter keeps base's bits: -0 + 0 would be +0)
    const uint32_t bits = g.base == nullptr ? 0 : base;
    const float b = BASE32 ? __uint_as_float(bits) : bf16_bits_to_f32(bits), o = i >= 0 ? b + d : b;
    if constexpr (F32) static_cast<float*>(g.out)[at] = o;
    else static_cast<uint16_t*>(g.out)[at] = (uint16_t)(BASE32 || i >= 0 ? f32_to_bf16_bits(o) : bits);
}

}  // namespace moe
