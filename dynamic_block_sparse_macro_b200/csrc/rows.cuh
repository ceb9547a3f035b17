// Shared device helpers of the row operators (block norms, head rotation,
// expert sort): packs of consecutive elements moved with one wide access, and
// sums over the threads that share a row.
#pragma once

#include "common.cuh"

namespace prism {
namespace rows {

constexpr int kSMs = 148;            // B200: the launch rules are fixed, so workspace sizes are host-only

// The bits in which any of some byte addresses, strides and widths differ from a multiple of 2^k tell the widest
// access that all rows allow.
struct Bits {
    uint64_t m = 0;
    Bits& operator<<(const void* p) { m |= (uint64_t)(uintptr_t)p; return *this; }
    Bits& bytes(int64_t n) { m |= (uint64_t)n; return *this; }
    bool multiple_of(int b) const { return m % b == 0; }
};
inline bool on(const void* p, int b) { return p != nullptr && (uintptr_t)p % b == 0; }
inline bool opt_on(const void* p, int b) { return (uintptr_t)p % b == 0; }

// N consecutive elements of T as they lie in memory
template <typename T, int N> struct Pack {
    static constexpr int kBytes = (int)sizeof(T) * N;
    uint32_t w[(kBytes + 3) / 4];
};

// Data that is read once: no line is kept in L1 (the vectors shared by all rows stay there).
// Not the read-only path: an output may be the input itself.
template <typename T, int N> __device__ __forceinline__ void load(Pack<T, N>& p, const T* src) {
    constexpr int B = Pack<T, N>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(p.w[4 * i]), "=r"(p.w[4 * i + 1]), "=r"(p.w[4 * i + 2]), "=r"(p.w[4 * i + 3])
                         : "l"((const char*)src + 16 * i) : "memory");
    } else if constexpr (B == 8) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(p.w[0]), "=r"(p.w[1]) : "l"(src) : "memory");
    } else if constexpr (B == 4) {
        asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(p.w[0]) : "l"(src) : "memory");
    } else {
        uint16_t v;
        asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(src) : "memory");
        p.w[0] = v;
    }
}

template <typename T, int N> __device__ __forceinline__ void store(T* dst, const Pack<T, N>& p) {
    constexpr int B = Pack<T, N>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};"
                         ::"l"((char*)dst + 16 * i), "r"(p.w[4 * i]), "r"(p.w[4 * i + 1]), "r"(p.w[4 * i + 2]),
                         "r"(p.w[4 * i + 3]) : "memory");
    } else if constexpr (B == 8) {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(dst), "r"(p.w[0]), "r"(p.w[1]) : "memory");
    } else if constexpr (B == 4) {
        asm volatile("st.global.u32 [%0], %1;" ::"l"(dst), "r"(p.w[0]) : "memory");
    } else {
        asm volatile("st.global.u16 [%0], %1;" ::"l"(dst), "h"((uint16_t)p.w[0]) : "memory");
    }
}

template <int N> __device__ __forceinline__ void unpack(const Pack<float, N>& p, float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(p.w[i]);
}
template <int N> __device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, N>& p, float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(i & 1 ? p.w[i / 2] & 0xffff0000u : p.w[i / 2] << 16);
}
template <int N> __device__ __forceinline__ void pack(Pack<float, N>& p, const float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) p.w[i] = __float_as_uint(f[i]);
}
// the one rounding to bf16 of a result held in fp32, to nearest even
template <int N> __device__ __forceinline__ void pack(Pack<__nv_bfloat16, N>& p, const float* f) {
    if constexpr (N == 1) {
        p.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            p.w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
}

// The threads that share a row: a whole number of warps, threadIdx.x within
// the team and threadIdx.y its number in the CTA.  A sum over several warps
// goes through shared memory with one named barrier (id team + 1): two
// buffers alternate, and a thread can write a buffer again only after the
// barrier of the sum in between, which every thread reaches after it has read.
struct Team {
    float4* buf;       // [2][32] of this team
    int threads, id, flip;

    __device__ __forceinline__ void init(float4* smem) {
        threads = blockDim.x;
        id = threadIdx.y;
        buf = smem + id * 64;
        flip = 0;
    }
    // sums of up to four values over the team, in a fixed order
    template <int N> __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N <= 4, "four values");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (threads == 32) return;
        float* p = reinterpret_cast<float*>(buf + flip * 32);
        flip ^= 1;
        const int l = threadIdx.x & 31;
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) p[4 * (threadIdx.x >> 5) + i] = v[i];
        }
        // a row that ends inside a warp can leave the warp's lanes apart here: all of them, the storing one too,
        // meet before the barrier counts the warp
        __syncwarp();
        asm volatile("barrier.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
        const bool in = l < (threads >> 5);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(in ? p[4 * l + i] : 0.f);
    }
    __device__ __forceinline__ float sum1(float a) {
        float v[1] = {a};
        sum(v);
        return v[0];
    }
};

}  // namespace rows
}  // namespace prism
