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

// s / c, where 1 / c is at hand: one correction makes it exact where the quotient is
__device__ __forceinline__ float mean_of(float s, float c, float inv_c) {
    const float m = s * inv_c;
    return fmaf(fmaf(-m, c, s), inv_c, m);
}

// The threads that share a row: 8, 16 or 32 lanes (MAXT = 32; threadIdx.x within the team, threadIdx.y its number
// in the CTA), or a whole CTA of up to MAXT threads, a multiple of 32.  A sum over a CTA's warps goes through shared
// memory with one barrier: two buffers alternate, and a thread can write a buffer again only after the barrier of
// the sum in between, which every thread reaches after it has read.  (Teams of several warps in one CTA, each with a
// named barrier, took 30% longer.)
template <int MAXT> struct Team {
    static constexpr int W = MAXT <= 256 ? 8 : MAXT <= 512 ? 16 : 32;   // warps of a team at most
    static constexpr int kBufs = MAXT == 32 ? 1 : 2 * W;
    float4* buf;       // [2][W]
    uint32_t mask;     // of the team's lanes in a warp
    int flip;

    __device__ __forceinline__ void init(float4* smem) {
        buf = smem;
        flip = 0;
        mask = 0xffffffffu;
        if (MAXT == 32 && blockDim.x < 32) {
            const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
            mask = ((1u << blockDim.x) - 1) << (lane & ~(blockDim.x - 1));
        }
    }
    // sums of up to four values over the team, in a fixed order
    template <int N> __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N <= 4, "four values");
        if constexpr (MAXT == 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (o < blockDim.x) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(mask, v[i], o);
                }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
            float4* b = buf + flip * W;
            flip ^= 1;
            const int l = threadIdx.x & 31, i = l & (W - 1);
            if (l == 0)
                b[threadIdx.x >> 5] = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.f, N > 2 ? v[N > 2 ? 2 : 0] : 0.f,
                                                  N > 3 ? v[N > 3 ? 3 : 0] : 0.f);
            __syncthreads();
            const float4 q = i < (blockDim.x >> 5) ? b[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = q.x;
            if constexpr (N > 1) v[1] = q.y;
            if constexpr (N > 2) v[2] = q.z;
            if constexpr (N > 3) v[3] = q.w;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        }
    }
    __device__ __forceinline__ float sum1(float a) {
        float v[1] = {a};
        sum(v);
        return v[0];
    }
};

}  // namespace rows
}  // namespace prism
