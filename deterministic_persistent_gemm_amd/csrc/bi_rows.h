// bi_rows.h -- rows of a matrix held in the registers of a team of threads, and
// reductions over them: the layer norm and the 8-bit quantisation.
#pragma once

#include <type_traits>

#include "bi_tile.h"

namespace bi {

// P chunks of eight values as they lie in memory.
template <bool BF, int P>
struct RowRaw {
    static constexpr int V = BF ? 1 : 2;
    u32x4 v[P * V];

    // thread t of T: chunks t, t + T, ...
    template <int T>
    __device__ __forceinline__ void load(const void* x, int64_t at, int t, int chunks)
    {
        const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const unsigned char*>(x) + at * (BF ? 2 : 4));
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[i * V + j] = p[min(i * T + t, chunks - 1) * V + j];
    }
    __device__ __forceinline__ float at(int i, int j) const     // value j of chunk i
    {
        if constexpr (BF) {
            const uint32_t u = v[i][j >> 1];
            return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
        } else {
            return __uint_as_float(v[2 * i + (j >> 2)][j & 3]);
        }
    }
    __device__ __forceinline__ void set(int i, const float (&f)[8])    // chunk i, rounded to nearest even
    {
        if constexpr (BF) {
            v[i] = u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
        } else {
            v[2 * i] = __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]});
            v[2 * i + 1] = __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]});
        }
    }
    template <int T>
    __device__ __forceinline__ void store(void* y, int64_t at, int t, int chunks) const
    {
        u32x4* p = reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(y) + at * (BF ? 2 : 4));
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (i * T + t < chunks) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    p[(i * T + t) * V + j] = v[i * V + j];
            }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < P * V; ++i)
            v[i] = u32x4{0u, 0u, 0u, 0u};
    }
};

// The sum over a wave, in every lane: a butterfly within each row of 16 lanes, then
// the four rows in pairs.
__device__ __forceinline__ float wave_sum(float v)
{
    auto moved = [](float f, auto ctrl) __attribute__((always_inline)) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(f), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v += moved(v, std::integral_constant<int, 0xB1>{});         // lanes 1 apart
    v += moved(v, std::integral_constant<int, 0x4E>{});         // 2 apart
    v += moved(v, std::integral_constant<int, 0x141>{});        // the other four of eight
    v += moved(v, std::integral_constant<int, 0x140>{});        // the other eight of sixteen
    auto row = [&](int r) __attribute__((always_inline)) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * r)); };
    return (row(0) + row(1)) + (row(2) + row(3));
}

// The largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto moved = [](uint32_t f, auto ctrl) __attribute__((always_inline)) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)f, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    v = max(v, moved(v, std::integral_constant<int, 0xB1>{}));
    v = max(v, moved(v, std::integral_constant<int, 0x4E>{}));
    v = max(v, moved(v, std::integral_constant<int, 0x141>{}));
    v = max(v, moved(v, std::integral_constant<int, 0x140>{}));
    auto row = [&](int r) __attribute__((always_inline)) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r); };
    return max(max(row(0), row(1)), max(row(2), row(3)));
}

}  // namespace bi
