// int8_kernels.hpp -- the int8 matrix product (gfx950):
//   out[m,n] = (sum_k a[m,k] w[n,k]) * a_scale[m] * w_scale[n]
// summed exactly in int32, so no order of the sum changes the result.
#pragma once

#include "around_common.hpp"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
// at any address
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ float int8_scaled(int32_t acc, float a_scale, float w_scale)
{
    return ((float)acc * a_scale) * w_scale;
}

// 16 codes at p, of which the first n (1..16) are the row's; the rest 0.  A
// whole load at any address where it stays below `end`, else byte by byte.
__device__ __forceinline__ u32x4 int8_load_part(const uint8_t* p, int n, const uint8_t* end)
{
    uint32_t d[4] = {0, 0, 0, 0};
    if (p + 16 <= end) {
        const u32x4 v = *reinterpret_cast<const u32x4_any*>(p);
        const uint32_t s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int left = n - 4 * i;                  // codes of this dword
            d[i] = left >= 4 ? s[i] : left > 0 ? s[i] & ((1u << (8 * left)) - 1u) : 0u;
        }
    } else {
        uint64_t lo = 0, hi = 0;                         // once a matrix at most: its last bytes
#pragma unroll 1
        for (int i = n - 1; i >= 0; --i) {
            hi = hi << 8 | lo >> 56;
            lo = lo << 8 | p[i];
        }
        return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    return u32x4{d[0], d[1], d[2], d[3]};
}

// ---------------------------------------------------------------------------
// GEMV for up to MT tokens.  L lanes share a channel, lane li taking the
// 16-code chunks li, li + L, ...; a wave holds R x 64 / L channels, a
// workgroup of 4 waves 4 times that, and strides over blocks of as many.  A
// step is U chunks a lane; the next step's codes are in flight while one is
// computed.  The token rows are staged once per workgroup in LDS, padded with
// zeros to whole steps, so past a row's end any codes will do: they meet zeros.
// Products by v_dot4_i32_i8.  Bound by the codes' read from HBM: 157,184 x 2,560
// at 1 token 60.2 us (6.7 TB/s), at 4 tokens 65-68 us.
// ---------------------------------------------------------------------------
// Sum over aligned groups of L lanes, in every lane of the group.
template <int L>
__device__ __forceinline__ int32_t group_sum_i32(int32_t v)
{
    static_assert(L == 16 || L == 64, "one DPP row or the wave");
    v += (int32_t)dpp_u32<kDppXor1>((uint32_t)v);
    v += (int32_t)dpp_u32<kDppXor2>((uint32_t)v);
    v += (int32_t)dpp_u32<kDppHalfMirror>((uint32_t)v);
    v += (int32_t)dpp_u32<kDppMirror>((uint32_t)v);
    if constexpr (L == 64)
        v = (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
            (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
    return v;
}

__device__ __forceinline__ int32_t dot16(u32x4 a, u32x4 b, int32_t acc)
{
    acc = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, acc, false);
    acc = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, acc, false);
    acc = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, acc, false);
    return __builtin_amdgcn_sdot4((int)a.w, (int)b.w, acc, false);
}

template <int MT, int U, int L, int R>
__global__ __launch_bounds__(256) void int8_gemv_kernel(Int8Args g)
{
    extern __shared__ u32x4 xs[];                        // [token][padded chunk]
    constexpr int CH = 4 * R * (64 / L);                 // channels a workgroup holds
    const int M = (int)g.M, K = g.K, chunks = (K + 15) / 16;
    const int steps = (chunks + L * U - 1) / (L * U), padded = steps * L * U;
    const bool whole = K % 16 == 0;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, li = lane % L, grp = lane / L;
    const uint8_t* w_end = g.w + (size_t)g.N * K;
    const int64_t blocks = (g.N + CH - 1) / CH;
    auto channel = [&](int64_t b, int r) { return (b * 4 + wave) * (CH / 4) + r * (64 / L) + grp; };
    struct Codes {
        u32x4 w[R][U];
    };
    auto load = [&](int64_t b, int s, Codes& c) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint8_t* row = g.w + (size_t)min(channel(b, r), g.N - 1) * K;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint8_t* p = row + min((s * U + i) * L + li, chunks - 1) * 16;
                if (whole) c.w[r][i] = load_stream(reinterpret_cast<const u32x4*>(p));
                else if (p + 16 <= w_end) c.w[r][i] = *reinterpret_cast<const u32x4_any*>(p);
                else c.w[r][i] = int8_load_part(p, (int)(w_end - p), w_end);
            }
        }
    };
    int64_t b = blockIdx.x;
    Codes now, next;
    load(b, 0, now);                                     // the grid is at most `blocks`
    {
        const uint8_t* a_end = g.a + (size_t)M * K;
        for (int t = 0; t < M; ++t)
            for (int c = threadIdx.x; c < padded; c += 256) {
                const uint8_t* p = g.a + (size_t)t * K + c * 16;
                u32x4 v = {0, 0, 0, 0};
                if (c < chunks) v = whole ? *reinterpret_cast<const u32x4*>(p) : int8_load_part(p, min(16, K - c * 16), a_end);
                xs[t * padded + c] = v;
            }
    }
    lds_barrier();
    int32_t acc[R][MT] = {};
    int s = 0;
    while (true) {
        int64_t nb = b;
        int ns = s + 1;
        if (ns == steps) {
            ns = 0;
            nb = b + gridDim.x;
        }
        if (nb < blocks) load(nb, ns, next);
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t)
                if (t < M) {
                    const u32x4 x = xs[t * padded + (s * U + i) * L + li];
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][t] = dot16(now.w[r][i], x, acc[r][t]);
                }
        if (ns == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t n = channel(b, r);
                const float ws = g.w_scale[min(n, g.N - 1)];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (t >= M) continue;
                    const int32_t sum = group_sum_i32<L>(acc[r][t]);
                    acc[r][t] = 0;
                    if (li == 0 && n < g.N) {
                        const float v = int8_scaled(sum, g.a_scale[t], ws);
                        if (g.out_type == kTypeF32) static_cast<float*>(g.out)[(size_t)t * g.N + n] = v;
                        else static_cast<uint16_t*>(g.out)[(size_t)t * g.N + n] = (uint16_t)f32_to_bf16_bits(v);
                    }
                }
            }
            if (nb >= blocks) return;
        }
        now = next;
        b = nb;
        s = ns;
    }
}

// ---------------------------------------------------------------------------
// Tiled product on the matrix cores.  A workgroup of WM x WN waves computes
// BM tokens x BN channels, a wave FM x FN tiles of 16 x 16, in steps of BK
// codes of K.  LDS holds a ring of S steps: while one is computed the loads of
// the next S - 1 are in flight, so a step does not wait for memory unless S - 1
// steps of work are shorter than a load.
//
// LDS rows are BK codes, CR = BK / 16 chunks of 16.  Chunk c of row r stands at
// position c ^ swizzle(r), chosen so that the 8 chunks of any 8 rows in turn
// lie in 8 different groups of 4 banks: neither an operand read (16 rows, one
// chunk of each) nor a load's write (whole rows) has a bank conflict.
//
// v_mfma_i32_16x16x64_i8: lane l gives row l % 16, codes 16 (l / 16).. of both
// operands, and gets rows 4 (l / 16) + 0..3 of the first and row l % 16 of the
// second.  The channels are the first operand, so a lane holds 4 consecutive
// channels of one token: one 16-byte store in fp32.
//
// What bounds it, from stamps of the phases (256 x 256 tiles): at 4096 x 4096 x
// 2560, one tile a compute unit, 46-50 us of which 2.6 us until the first step
// has landed, 36 us in the steps (20.7 us of them the matrix cores' own time at
// the ~2.1 GHz they run at; reads from LDS take nearly as long and overlap
// partly) and 8 us in the scales and stores.  At 10240 codes of K the same
// product runs at 2.1-2.3 POP/s.  Small products are a chain of latencies: 77 x
// 2560 x 768, 4.0 us, has 1.0 us to the first step, 1.3 us of steps and 0.9 us
// of scales and stores.
// ---------------------------------------------------------------------------
template <int BK>
__device__ __forceinline__ int int8_swizzle(int r)
{
    static_assert(BK == 64 || BK == 128, "rows of 4 or 8 chunks");
    return BK == 128 ? r & 7 : (r >> 1) & 3;
}

__device__ __forceinline__ void load_to_lds(const uint8_t* src, u32x4* dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Waits until at most N of this wave's vector-memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "a 6-bit counter");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4 | 15 << 8);
}

// Waits for all but the last `steps` steps' loads, of NL each (0 <= steps <= MAX).
template <int NL, int MAX>
__device__ __forceinline__ void wait_steps(int steps)
{
    if constexpr (MAX > 0) {
        if (steps >= MAX) return wait_vm<NL * MAX>();
        return wait_steps<NL, MAX - 1>(steps);
    } else {
        wait_vm<0>();
    }
}

template <int N>
struct Count {
    static constexpr int value = N;
};

template <int BM, int BN, int WM, int WN, int BK, int S, int EU, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN, EU) void int8_tile_kernel(Int8Args g)
{
    constexpr int T = 64 * WM * WN, FM = BM / (16 * WM), FN = BN / (16 * WN), CR = BK / 16;
    constexpr int ROWS = BM + BN, NL = ROWS * CR / T;    // rows in LDS, chunks a thread loads a step
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && ROWS * CR % T == 0 && BM % (T / CR) == 0, "tile shape");
    static_assert(T / CR % 8 == 0, "a thread's rows have one swizzle");
    extern __shared__ u32x4 lds[];                       // [S][ROWS * CR]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    // Workgroups are dealt to the 8 XCDs in turn, each with a cache of its own:
    // the tiles are split into xm x (8 / xm) interleaved parts, one an XCD,
    // chosen by the host so that an XCD reads few rows.  Within a part the token
    // tiles of a channel tile follow one another, so its channels come from
    // memory once.
    const uint32_t mt = (uint32_t)((g.M + BM - 1) / BM), nt = (uint32_t)((g.N + BN - 1) / BN);
    const uint32_t xm = g.xm, xn = 8 / xm, mx = (mt + xm - 1) / xm;
    const uint32_t nx = (blockIdx.x >> 3) / mx, mi = ((blockIdx.x >> 3) - nx * mx) * xm + (blockIdx.x & 7) % xm;
    const uint32_t ni = nx * xn + (blockIdx.x & 7) / xm;
    if (mi >= mt || ni >= nt) return;
    const int64_t m0 = (int64_t)mi * BM, n0 = (int64_t)ni * BN;
    const int K = g.K;

    // Thread's chunk j: row (tid + j T) / CR of the tile (tokens, then channels;
    // rows behind the last are the last again and their results dropped), at
    // LDS position tid + j T; the position's chunk is found by the swizzle.
    // Offsets from the tile's first row: at most 256 rows of 131071 codes.
    const uint8_t* const a0 = g.a + (size_t)m0 * K;
    const uint8_t* const w0 = g.w + (size_t)n0 * K;
    uint32_t off[NL];
    const int r0 = tid / CR, chunk = (tid % CR) ^ int8_swizzle<BK>(r0);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const int r = r0 + j * (T / CR);
        const int last = (int)min((int64_t)(r < BM ? BM : BN), r < BM ? g.M - m0 : g.N - n0) - 1;
        off[j] = (uint32_t)min(r < BM ? r : r - BM, last) * (uint32_t)K + chunk * 16;
    }
    auto base = [&](int j) { return j * (T / CR) < BM ? a0 : w0; };
    auto buf = [&](int i) { return lds + i * (ROWS * CR); };

    i32x4 acc[FN][FM] = {};
    struct Frags {
        i32x4 op[FN + FM];                               // operands of 64 codes: channels, then tokens
    };
    const int row = lane & 15;
    auto read = [&](Frags& f, const u32x4* b, int kk, int i) {
        const int c = (kk * 4 + (lane >> 4)) ^ int8_swizzle<BK>(row);
        const int r = i < FN ? BM + (wn * FN + i) * 16 : (wm * FM + i - FN) * 16;
        f.op[i] = __builtin_bit_cast(i32x4, b[(r + row) * CR + c]);
    };
    auto multiply = [&](const Frags& f, int q) {
        const int j = q / FM, i = q % FM;
        acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.op[j], f.op[FN + i], acc[j][i], 0, 0, 0);
    };

    // DIRECT (K a multiple of 16: rows of whole, aligned chunks): whole steps
    // go from memory straight to LDS.  Otherwise, and for the part step at the
    // end, through registers.
    const int steps = (K + BK - 1) / BK, straight = DIRECT ? K / BK : 0;
    if constexpr (DIRECT) {
        constexpr int P = BK / 64;                       // phases a step
        constexpr int Q = FM * FN, NR = FM + FN;         // products and operand reads a phase
        constexpr int H1 = P == 2 ? NL / 2 : NL;         // loads in a step's last phase; the rest in the next's first
        auto fetch = [&](int step, int slot, int j) {
            load_to_lds(base(j) + (size_t)step * BK + off[j], buf(slot) + j * T + wave * 64);
        };
        // A phase multiplies the operands that the phase before it read, and
        // reads the next phase's.  Where those belong to the next step, that
        // step has to have landed, here and (behind the barrier) from every
        // wave, and this step has been read by every wave, so its place is free
        // for the step S ahead, whose loads are spread over this phase and the
        // next step's first.  Reads and loads are issued between the products,
        // so that the matrix cores work while their queues fill.  The reads are
        // waited for by hand at the start of a phase: left to itself the
        // compiler waits for the reads that the phase has just issued as well.
        auto phase = [&](const Frags& now, Frags& next, const u32x4* from, int kk, int step, int slot, auto first, auto last) {
            constexpr int F0 = decltype(first)::value, F1 = decltype(last)::value, ALL = NR + F1 - F0;
            const bool more = step < straight;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int i = q * ALL / Q; i < (q + 1) * ALL / Q; ++i) {
                    if (i < NR) read(next, from, kk, i);
                    else if (more) fetch(step, slot, F0 + i - NR);
                }
                multiply(now, q);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0): `next` is here
        };
        if (straight > 0) {
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (i < straight)
#pragma unroll
                    for (int j = 0; j < (i < S - 1 ? NL : H1); ++j) fetch(i, i, j);
            if (straight >= S) wait_vm<NL * (S - 2) + H1>();
            else wait_steps<NL, S - 2>(straight - 1);
            __builtin_amdgcn_s_barrier();
            Frags f0, f1;
#pragma unroll
            for (int i = 0; i < NR; ++i) read(f0, buf(0), 0, i);
            __builtin_amdgcn_s_waitcnt(0xC07F);
            int at = 0, before = S - 1;                  // ring positions of this step and the one before it
            auto step_on = [&](int s, const Frags& now, Frags& next) {
                const int after = at + 1 == S ? 0 : at + 1;
                wait_steps<NL, S - 2>(max(straight - 2 - s, 0));
                __builtin_amdgcn_s_barrier();
                // (behind the last step: reads of whatever stands there, unused)
                phase(now, next, buf(after), 0, s + S, at, Count<0>{}, Count<H1>{});
                before = at;
                at = after;
            };
            if constexpr (P == 2) {
                for (int s = 0; s < straight; ++s) {
                    phase(f0, f1, buf(at), 1, s + S - 1, before, Count<H1>{}, Count<NL>{});
                    step_on(s, f1, f0);
                }
            } else {
                for (int s = 0; s < straight; s += 2) {
                    step_on(s, f0, f1);
                    if (s + 1 < straight) step_on(s + 1, f1, f0);
                }
            }
        }
        __syncthreads();
    }
    if (straight < steps) {
        const uint8_t* a_end = g.a + (size_t)g.M * K;
        const uint8_t* w_end = g.w + (size_t)g.N * K;
        u32x4 v[NL];
        auto load_part = [&](int s) {                    // any alignment, zeros behind the row's end
            const int k = s * BK + chunk * 16;
            if ((s + 1) * BK <= K) {
#pragma unroll
                for (int j = 0; j < NL; ++j) v[j] = *reinterpret_cast<const u32x4_any*>(base(j) + s * BK + off[j]);
                return;
            }
#pragma unroll
            for (int j = 0; j < NL; ++j)
                v[j] = k < K ? int8_load_part(base(j) + s * BK + off[j], min(16, K - k), j * (T / CR) < BM ? a_end : w_end)
                             : u32x4{0, 0, 0, 0};
        };
        auto put = [&](u32x4* b) {
#pragma unroll
            for (int j = 0; j < NL; ++j) b[tid + j * T] = v[j];
        };
        load_part(straight);
        put(buf(0));
        __syncthreads();
        for (int s = straight; s < steps; ++s) {
            if (s + 1 < steps) load_part(s + 1);
#pragma unroll
            for (int kk = 0; kk < BK / 64; ++kk) {
                Frags f;
#pragma unroll
                for (int i = 0; i < FM + FN; ++i) read(f, buf((s - straight) & 1), kk, i);
#pragma unroll
                for (int q = 0; q < FM * FN; ++q) multiply(f, q);
            }
            if (s + 1 < steps) put(buf((s + 1 - straight) & 1));
            __syncthreads();
        }
    }

    // every scale is loaded before the first store: a store may change what a
    // later load reads, for all the compiler knows, so loads among the stores
    // would wait one by one
    float as[FM], ws[FN][4];
#pragma unroll
    for (int i = 0; i < FM; ++i) as[i] = g.a_scale[min(m0 + (wm * FM + i) * 16 + row, g.M - 1)];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) ws[j][r] = g.w_scale[min(n0 + (wn * FN + j) * 16 + (lane >> 4) * 4 + r, g.N - 1)];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + (wm * FM + i) * 16 + row;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t n = n0 + (wn * FN + j) * 16 + (lane >> 4) * 4;
            if (n >= g.N) continue;
            float o[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = int8_scaled(acc[j][i][r], as[i], ws[j][r]);
            const size_t p = (size_t)m * g.N + n;
            const bool all = n + 4 <= g.N;               // a row may start at any address
            if (g.out_type == kTypeF32) {
                float* out = static_cast<float*>(g.out) + p;
                if (all) *reinterpret_cast<f32x4_any*>(out) = f32x4_any{o[0], o[1], o[2], o[3]};
                else
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        if (n + r < g.N) out[r] = o[r];
            } else {
                uint16_t* out = static_cast<uint16_t*>(g.out) + p;
                if (all)
                    *reinterpret_cast<u32x2_any*>(out) = u32x2_any{f32_to_bf16_bits(o[0]) | f32_to_bf16_bits(o[1]) << 16,
                                                                  f32_to_bf16_bits(o[2]) | f32_to_bf16_bits(o[3]) << 16};
                else
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        if (n + r < g.N) out[r] = (uint16_t)f32_to_bf16_bits(o[r]);
            }
        }
    }
}

}  // namespace moe
