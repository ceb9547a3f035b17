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

inline int esize(int dtype) { return dtype == PRISM_BF16 ? 2 : 4; }
// the row stride in elements (0: dense); false when rows would overlap
inline bool ld_of(int64_t ld, int64_t C, int64_t* out) {
    *out = ld == 0 ? C : ld;
    return *out >= C;
}

// Whether the runtime took the call that has just been made (r: its own answer).  A refusal is this call's to report:
// nothing further is launched, and it is not left behind for the next call's check.
inline bool taken(cudaError_t r) { return r == cudaSuccess || (cudaGetLastError(), false); }
inline bool launched() { return cudaGetLastError() == cudaSuccess; }

// A kernel that finishes another one's work is launched while that one runs and waits for it where it first needs
// its results, so that its start is not waited for.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... A>
inline bool launch_after(void (*kernel)(A...), dim3 grid, dim3 block, int cluster_y, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = (unsigned)cluster_y;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster_y > 1 ? 2 : 1;
    return taken(cudaLaunchKernelEx(&cfg, kernel, args...));
}

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

// Two fp32 values in one 64-bit register: sm_100a adds, multiplies and fuses both with one instruction.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 both(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum(F2 a) {
    const float2 f = both(a);
    return f.x + f.y;
}
__device__ __forceinline__ void unpack2(const Pack<float, 8>& p, F2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(p.w[2 * i]), __uint_as_float(p.w[2 * i + 1]));
}
__device__ __forceinline__ void unpack2(const Pack<__nv_bfloat16, 8>& p, F2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(p.w[i] << 16), __uint_as_float(p.w[i] & 0xffff0000u));
}

// A row's elements on their way from HBM: each thread copies what it will itself read into its own part of
// shared memory, rows ahead of their use, without registers and without a barrier (it waits for its own copies).
// Memory is laid out in planes of one access a thread, so that a warp's accesses are contiguous.
template <int B> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    static_assert(B == 4 || B == 8 || B == 16, "an access of cp.async");
    if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if constexpr (B == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int E> struct Lane {
    static constexpr int U = 8 / E;                                     // units of E channels: eight channels a thread
    static constexpr bool kAsync = sizeof(T) * E >= 4;
    static constexpr int B = sizeof(T) * E < 16 ? (int)sizeof(T) * E : 16, P = (int)sizeof(T) * E / B;
    static constexpr int kBytes = 8 * (int)sizeof(T);                   // of a thread and row
    // unit u of thread t in a team of `team` threads covers channels (u * team + t) * E + [0, E)
    static __device__ __forceinline__ void fetch(uint32_t s, int threads, int tid, const T* row, int t, int team, int C) {
        if constexpr (kAsync) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * team + t) * E;
                if (c < C) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        cp_async<B>(s + (uint32_t)(((u * P + p) * threads + tid) * B), row + c + p * (B / (int)sizeof(T)));
                }
            }
        }
    }
    // places that no copy writes (past the row's end, or `all`) hold 0
    static __device__ __forceinline__ void clear(char* s, int threads, int tid, int t, int team, int C, bool all) {
        if (!all && ((U - 1) * team + t) * E < C) return;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (all || (u * team + t) * E >= C) {
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int i = 0; i < B; i += 4)
                        *reinterpret_cast<uint32_t*>(s + ((u * P + p) * threads + tid) * B + i) = 0u;
            }
    }
    // the thread's eight channels in fp32
    static __device__ __forceinline__ void read(F2 (&f)[4], const char* s, int threads, int tid) {
        Pack<T, 8> v;
#pragma unroll
        for (int i = 0; i < U * P; ++i) {
            const char* a = s + (i * threads + tid) * B;
            if constexpr (B == 16) {
                const uint4 q = *reinterpret_cast<const uint4*>(a);
                v.w[4 * i] = q.x; v.w[4 * i + 1] = q.y; v.w[4 * i + 2] = q.z; v.w[4 * i + 3] = q.w;
            } else if constexpr (B == 8) {
                const uint2 q = *reinterpret_cast<const uint2*>(a);
                v.w[2 * i] = q.x; v.w[2 * i + 1] = q.y;
            } else if constexpr (B == 4) {
                v.w[i] = *reinterpret_cast<const uint32_t*>(a);
            }
        }
        unpack2(v, f);
    }
};

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
    static constexpr int kFloats = MAXT == 32 ? 1 : 2 * 4 * W;
    float* buf;        // [2][4][W]
    uint32_t mask;     // of the team's lanes in a warp
    int flip;

    // by all threads of the CTA
    __device__ __forceinline__ void init(float* smem) {
        buf = smem;
        flip = 0;
        mask = 0xffffffffu;
        if (MAXT == 32 && blockDim.x < 32) {
            const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
            mask = ((1u << blockDim.x) - 1) << (lane & ~(blockDim.x - 1));
        }
        if (MAXT > 32) {                                 // the places of warps that the CTA does not have count as 0
            for (int i = threadIdx.x; i < kFloats; i += blockDim.x) smem[i] = 0.f;
            __syncthreads();
        }
    }
    // Sums of up to four values over the team, in a fixed order.  A warp's lanes share the values out among them:
    // with four, the halves of the warp swap two each, the quarters one, and three steps finish each lane's value
    // (6 exchanges instead of 20); the warps' sums meet in the same way.
    template <int N> __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N >= 1 && N <= 4, "up to four values");
        if (MAXT == 32 && blockDim.x < 32) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                if (o < blockDim.x) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(mask, v[i], o);
                }
        } else {
            constexpr int NP = N <= 2 ? N : 4, L = 32 / NP;
            const int l = threadIdx.x & 31;
            float a[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) a[i] = i < N ? v[i] : 0.f;
            int o = 16;
#pragma unroll
            for (int c = NP / 2; c > 0; c >>= 1, o >>= 1) {
                const bool hi = l & o;
#pragma unroll
                for (int i = 0; i < c; ++i) {
                    const float give = hi ? a[i] : a[i + c], keep = hi ? a[i + c] : a[i];
                    a[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            float k = a[0];
#pragma unroll
            for (; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
            // lane l has value l / L
            if constexpr (MAXT == 32) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = NP == 1 ? k : __shfl_sync(0xffffffffu, k, i * L);
                return;
            }
            float* b = buf + flip * 4 * W;
            flip ^= 1;
            if (l % L == 0) b[l / L * W + (threadIdx.x >> 5)] = k;
            __syncthreads();
            constexpr int PARTS = L < W ? L : W, PER = W / PARTS;       // lanes a value, warps a lane
            const float* q = b + (l % NP) * W + (l / NP % PARTS) * PER;
            k = q[0];
#pragma unroll
            for (int i = 1; i < PER; ++i) k += q[i];
#pragma unroll
            for (int p = NP; p < NP * PARTS; p <<= 1) k += __shfl_xor_sync(0xffffffffu, k, p);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = NP == 1 ? k : __shfl_sync(0xffffffffu, k, i);
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
