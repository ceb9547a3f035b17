// The norms around a transformer block, fused with its gate and residual scale.
//
//   z = res_scale x + gate_g ∘ N_post(h) ∘ w_post          (z = x without a branch h)
//   y = N(z) ∘ w ∘ (1 + scale_g) + b ∘ (1 + scale_g) + shift_g
//
// N(v) = (v - m) r with m = 0 (rms) or the mean (layer) and r = (mean (v-m)² + eps)^-1/2.
// With a = w (1 + scale_g), c = dy ∘ a and n = N(z), the gradients are
//
//   dz' = dz + r (c - [mean c] - n mean(c ∘ n))             (mean c: layer only)
//   dx  = res_scale dz'
//   dn  = dz' ∘ gate_g ∘ w_post,  nh = N_post(h),  dh = r_h (dn - [mean dn] - nh mean(dn ∘ nh))
//   A_g = sum_r dy ∘ n,  D_g = sum_r dy,  B_g = sum_r dz' ∘ nh    over the rows of group g
//   dscale_g = w ∘ A_g + b ∘ D_g,  dshift_g = D_g,  dgate_g = w_post ∘ B_g
//   dw = sum_g (1 + scale_g) ∘ A_g,  db = sum_g (1 + scale_g) ∘ D_g,  dw_post = sum_g gate_g ∘ B_g
//
// Everything between a load and a store is fp32: statistics, means and column sums too.  A result
// that is stored as bf16 is rounded once, at its store; y comes from the unrounded z.
//
// Bound by HBM: every row is read and written once.  A row's threads hold eight channels each, a few lanes, a warp or a
// CTA of up to 1024 threads, and keep the vectors of the row's group in registers from row to row.  What is past the
// row's end enters no sum.  Of what decides the speed:
//   - few spills or none: the f32 / bf16 forward at 131072 x 2048 took 705 us with 88 bytes of them and takes 501 without (498
//     at the measured copy rate); with more CTAs an SM (64 registers, 112 bytes) 747;
//   - fp32 pairs in one instruction: the backward of 61440 x 2048 339 -> 248 us, rows copied three ahead included; with
//     one barrier a row less 243 (233);
//   - the widest teams have an SM to themselves and leave it idle at each of a row's barriers: backwards more than 384
//     threads (f32 stream and branch: 320), forwards with a branch more than 512 (narrow accesses: 384), without one more
//     than 768 (narrow accesses as with a branch); see fwd_ctas and bwd_ctas.  8191 x 5120 with two rms norms 98 us (78),
//     13269 x 8192 276 (202).  Clusters of CTAs of 256 threads in their place wait longer for one another: 13269 x 4096
//     149 us instead of 128, with the cluster's barrier 229.
//   - rows of odd width move element by element: 40000 x 1001 bf16 218 us backwards, x 1000 93.
#pragma once

#include <initializer_list>

#include "rows.cuh"

namespace prism {
namespace bn {

using namespace rows;

constexpr int kMaxChannels = 8192;

struct FwdArgs {
    const void *x, *h;
    const float *gate, *w_post, *w, *b, *scale, *shift;
    void *z, *y;
    int64_t R, rpg, ld_x, ld_h, ld_z, ld_y, ld_gate, ld_scale, ld_shift;
    int C, norm, post;
    float eps, res;
};

struct BwdArgs {
    const void *z, *h, *dz, *dy;
    const float *gate, *w_post, *w, *b, *scale;
    void *dx, *dh;
    float *dgate, *dscale, *dshift;    // [groups][C], where whole groups are a segment's; else null
    float* part;                       // [segments][3][C] column sums; null: not wanted
    int64_t R, rpg, groups, segs;
    int64_t ld_z, ld_h, ld_dz, ld_dy, ld_dx, ld_dh, ld_gate, ld_scale;
    // segments a group; 0: a segment has whole groups, writes their gradients itself and leaves the sums over its
    // groups that dw, db and dw_post are made of
    int C, norm, post, per_group;
    float eps, res;
};

template <int E> __device__ __forceinline__ void load_vec(float* f, const float* p) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
    } else if constexpr (E == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(p));
        f[0] = v.x; f[1] = v.y;
    } else {
        f[0] = __ldg(p);
    }
}
// what the same thread has written: not through the read-only path
template <int E> __device__ __forceinline__ void load_own(float* f, const float* p) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            float4 v;
            asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p + 4 * i) : "memory");
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = *(const volatile float*)(p + i);
    }
}
template <int E> __device__ __forceinline__ void store_vec(float* p, const float* f) {
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else if constexpr (E == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
        p[0] = f[0];
    }
}

// Rows on their way to a team's threads: through shared memory, D rows ahead (Lane), or, for elements of two bytes
// that lie on no wider boundary, through registers, one row ahead.
extern __shared__ __align__(16) char g_ring[];

// A thread's eight channels, of the packs that hold them, in fp32.
template <typename T, int E> __device__ __forceinline__ void unpack_units(const Pack<T, E> (&p)[8 / E], F2 (&f)[4]) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8 / E; ++u) unpack<E>(p[u], v + u * E);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(v[2 * i], v[2 * i + 1]);
}
template <typename T, int E> __device__ __forceinline__ void clear_units(Pack<T, E> (&p)[8 / E]) {
#pragma unroll
    for (int u = 0; u < 8 / E; ++u)
#pragma unroll
        for (int i = 0; i < (int)(sizeof(p[u].w) / 4); ++i) p[u].w[i] = 0u;
}
// and stored, where they are the row's
template <typename T, int E> __device__ __forceinline__ void put_units(T* row, const F2 (&v)[4], int t, int team, int C) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = both(v[i]);
        o[2 * i] = f.x;
        o[2 * i + 1] = f.y;
    }
#pragma unroll
    for (int u = 0; u < 8 / E; ++u) {
        const int c = (u * team + t) * E;
        if (c < C) {
            Pack<T, E> p;
            pack<E>(p, o + u * E);
            store(row + c, p);
        }
    }
}

// D > 0: D rows ahead through shared memory (teams of more than 256 threads), else one through registers.
template <typename TX, typename TH, int E, int MAXT, bool HAS_H, int CTAS, int D>
__global__ void __launch_bounds__(MAXT == 32 ? 256 : MAXT, CTAS) k_block_norm_fwd(const FwdArgs a) {
    constexpr int U = 8 / E;
    constexpr bool RING = D > 0;
    using LX = Lane<TX, E>;
    using LH = Lane<TH, E>;
    __shared__ float sums[Team<MAXT>::kFloats];
    Team<MAXT> team;
    team.init(sums);
    const int t = threadIdx.x, T = blockDim.x, C = a.C;
    // of a CTA-wide team the compiler sees that its row is the same for all threads
    const int64_t nteams = MAXT == 32 ? (int64_t)gridDim.x * blockDim.y : gridDim.x;
    const int64_t me = MAXT == 32 ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    // All teams move over the rows together where groups are long, else each over rows of its own, whose vectors it
    // then loads once a group.
    const bool together = a.rpg >= 4 * nteams;
    const int64_t r0 = together ? me : a.R * me / nteams, r1 = together ? a.R : a.R * (me + 1) / nteams;
    const int64_t step = together ? nteams : 1;
    if (r0 >= r1) return;
    const float fc = (float)C, inv_c = 1.f / fc;
    const TX* x = (const TX*)a.x;
    const TH* h = (const TH*)a.h;
    auto in = [&](int i) { return ((i / E) * T + t) * E < C; };          // whether channel i of the thread's eight is the row's
    auto pair = [&](float m, int i) { return f2(in(2 * i) ? m : 0.f, in(2 * i + 1) ? m : 0.f); };

    const uint32_t ring = RING ? (uint32_t)__cvta_generic_to_shared(g_ring) : 0u;
    const int o_h = LX::kBytes * T, stage_bytes = o_h + (HAS_H ? LH::kBytes * T : 0);
    Pack<TX, E> rx[RING ? 1 : U];
    Pack<TH, E> rh[RING ? 1 : U];
    if constexpr (RING) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            LX::clear(g_ring + i * stage_bytes, T, t, t, T, C, false);
            if constexpr (HAS_H) LH::clear(g_ring + i * stage_bytes + o_h, T, t, t, T, C, false);
        }
    } else {
        clear_units<TX, E>(rx);
        clear_units<TH, E>(rh);
    }
    auto fetch = [&](int64_t r, int stage) {
        if constexpr (RING) {
            if (r < r1) {
                LX::fetch(ring + stage * stage_bytes, T, t, x + r * a.ld_x, t, T, C);
                if constexpr (HAS_H) LH::fetch(ring + stage * stage_bytes + o_h, T, t, h + r * a.ld_h, t, T, C);
            }
            cp_commit();
        } else if (r < r1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                if (c < C) {
                    load(rx[u], x + r * a.ld_x + c);
                    if (HAS_H) load(rh[u], h + r * a.ld_h + c);
                }
            }
        }
    };
#pragma unroll
    for (int i = 0; i < (RING ? D : 1); ++i) fetch(r0 + i * step, i);

    F2 mul[4], add[4], gate[HAS_H ? 4 : 1];
    auto vectors = [&](int64_t g) {
        float m[8], n[8], q[HAS_H ? 8 : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * E;
            float s[E];
#pragma unroll
            for (int e = 0; e < E; ++e) { m[u * E + e] = 1.f; n[u * E + e] = 0.f; }
            if constexpr (HAS_H) {
#pragma unroll
                for (int e = 0; e < E; ++e) q[u * E + e] = 1.f;
            }
            if (c >= C) continue;
            if (a.norm != PRISM_NORM_NONE) {
                if (a.w) load_vec<E>(m + u * E, a.w + c);
                if (a.b) load_vec<E>(n + u * E, a.b + c);
                if (a.scale) {
                    load_vec<E>(s, a.scale + g * a.ld_scale + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) { m[u * E + e] *= 1.f + s[e]; n[u * E + e] *= 1.f + s[e]; }
                }
                if (a.shift) {
                    load_vec<E>(s, a.shift + g * a.ld_shift + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) n[u * E + e] += s[e];
                }
            }
            if constexpr (HAS_H) {
                if (a.gate) load_vec<E>(q + u * E, a.gate + g * a.ld_gate + c);
                if (a.w_post) {
                    load_vec<E>(s, a.w_post + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) q[u * E + e] *= s[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mul[i] = f2(m[2 * i], m[2 * i + 1]);
            add[i] = f2(n[2 * i], n[2 * i + 1]);
            if constexpr (HAS_H) gate[i] = f2(in(2 * i) ? q[2 * i] : 0.f, in(2 * i + 1) ? q[2 * i + 1] : 0.f);
        }
    };
    int64_t g = r0 / a.rpg, next = (g + 1) * a.rpg;
    vectors(g);

    int stage = 0;
    int64_t r = r0;
    if constexpr (RING && D >= 2 && !HAS_H) {
        if (a.norm == PRISM_NORM_LAYER) {
            // A row's second sum goes together with the next row's first one, one barrier a row less: 13269 x 5416
            // 82 -> 72 us.  (With a branch, whose rows are then summed up twice, 4096 wide 84 -> 88.)
            auto stream = [&](F2 (&v)[4], int st) { LX::read(v, g_ring + st * stage_bytes, T, t); };
            auto total = [&](const F2 (&v)[4]) { return sum((v[0] + v[1]) + (v[2] + v[3])); };
            while (r < r1) {
                if (r >= next) {
                    vectors(++g);
                    next += a.rpg;
                }
                const int64_t end = next < r1 ? next : r1;
                F2 v[4];
                cp_wait<D - 1>();
                stream(v, stage);
                float m = team.sum1(total(v));
                for (; r < end; r += step) {
                    const int after = stage + 1 == D ? 0 : stage + 1;
                    stream(v, stage);
                    m = -mean_of(m, fc, inv_c);
                    F2 q;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = v[i] + pair(m, i);
                        q = i ? fma(v[i], v[i], q) : v[i] * v[i];
                    }
                    float two[2] = {sum(q), 0.f};
                    if (r + step < end) {
                        F2 ahead[4];
                        cp_wait<D - 2>();
                        stream(ahead, after);
                        two[1] = total(ahead);
                    }
                    team.sum(two);
                    const F2 rs = f2(rsqrtf(two[0] * inv_c + a.eps));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = fma(v[i] * rs, mul[i], add[i]);
                    put_units<TH, E>((TH*)a.y + r * a.ld_y, v, t, T, C);
                    fetch(r + D * step, stage);
                    stage = after;
                    m = two[1];
                }
            }
        }
    }
    for (; r < r1; r += step) {
        F2 v[4], hv[HAS_H ? 4 : 1];
        if constexpr (RING) {
            cp_wait<D - 1>();
            LX::read(v, g_ring + stage * stage_bytes, T, t);
            if constexpr (HAS_H) LH::read(hv, g_ring + stage * stage_bytes + o_h, T, t);
        } else {
            unpack_units<TX, E>(rx, v);
            if constexpr (HAS_H) unpack_units<TH, E>(rh, hv);
            fetch(r + step, 0);
        }
        if (r >= next) {                  // steps are shorter than groups
            vectors(++g);
            next += a.rpg;
        }

        // 1/std of the row held in f; f becomes f - mean (layer)
        auto stats = [&](F2 (&f)[4], int kind) {
            if (kind == PRISM_NORM_LAYER) {
                const float m = -mean_of(team.sum1(sum((f[0] + f[1]) + (f[2] + f[3]))), fc, inv_c);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = f[i] + pair(m, i);
            }
            F2 q = f[0] * f[0];
#pragma unroll
            for (int i = 1; i < 4; ++i) q = fma(f[i], f[i], q);
            return rsqrtf(team.sum1(sum(q)) * inv_c + a.eps);
        };

        if constexpr (HAS_H) {
            if (a.post != PRISM_NORM_NONE) {
                const F2 rh_ = f2(stats(hv, a.post));
#pragma unroll
                for (int i = 0; i < 4; ++i) hv[i] = hv[i] * rh_;
            }
            const F2 res = f2(a.res);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fma(res, v[i], gate[i] * hv[i]);
            put_units<TX, E>((TX*)a.z + r * a.ld_z, v, t, T, C);
        }
        if (a.norm != PRISM_NORM_NONE) {
            const F2 rs = f2(stats(v, a.norm));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fma(v[i] * rs, mul[i], add[i]);
            put_units<TH, E>((TH*)a.y + r * a.ld_y, v, t, T, C);
        }
        if constexpr (RING) {             // the row's own values have been used: their place is free
            fetch(r + D * step, stage);
            stage = stage + 1 == D ? 0 : stage + 1;
        }
    }
    if constexpr (RING) cp_wait<0>();
}

constexpr bool vec_shared(int maxt, bool f32) { return maxt > 640 || (maxt == 384 && !f32); }
constexpr int kTeamSums = 256 * 8 * 3 * (int)sizeof(float);       // of the teams of a CTA that are each within a warp

// What the backward's branch is: none, one that goes to the sum as it is, or one with a norm of its own.
enum Branch { kNoBranch = 0, kPlain = 1, kNormed = 2 };

template <typename TX, typename TH, int E, int MAXT, int BR, int CTAS, int D>
__global__ void __launch_bounds__(MAXT == 32 ? 256 : MAXT, CTAS) k_block_norm_bwd(const BwdArgs a) {
    constexpr int U = 8 / E;
    constexpr bool HAS_H = BR != kNoBranch;
    constexpr bool RING = Lane<TX, E>::kAsync && Lane<TH, E>::kAsync;
    using LX = Lane<TX, E>;
    using LH = Lane<TH, E>;
    __shared__ float sums[Team<MAXT>::kFloats];
    Team<MAXT> team;
    team.init(sums);
    const int t = threadIdx.x, T = blockDim.x, C = a.C;
    // A segment is a CTA's.  Segment s of a group takes its rows s, s + per_group, ... (teams within a warp: in runs of
    // a row a team), so that all teams move over the rows together.  Where groups are many and short a segment is a
    // team's and has a run of them.
    const bool whole = a.per_group == 0;
    const int64_t seg = MAXT == 32 && whole ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (seg >= a.segs) return;
    int64_t g, r0, r1, step = 1;
    if (!whole) {
        const int teams = MAXT == 32 ? blockDim.y : 1, me = MAXT == 32 ? threadIdx.y : 0;
        g = seg / a.per_group;
        r0 = g * a.rpg + (seg - g * a.per_group) * teams + me;
        r1 = (g + 1) * a.rpg;
        step = (int64_t)a.per_group * teams;
    } else {
        g = a.groups * seg / a.segs;
        r0 = g * a.rpg;
        r1 = a.groups * (seg + 1) / a.segs * a.rpg;
    }
    if (r1 > a.R) r1 = a.R;
    const float fc = (float)C, inv_c = 1.f / fc;
    const bool has_y = a.norm != PRISM_NORM_NONE;
    auto in = [&](int i) { return ((i / E) * T + t) * E < C; };          // whether channel i of the thread's eight is the row's
    // the means that belong to pair i: 0 past the row's end, where everything stays 0
    auto pair = [&](float m, int i) { return f2(in(2 * i) ? m : 0.f, in(2 * i + 1) ? m : 0.f); };

    // a stage: z, dz (TX), then dy, h (TH)
    const int threads = MAXT == 32 ? 256 : T, tid = MAXT == 32 ? threadIdx.y * T + t : t;
    const uint32_t ring = RING ? (uint32_t)__cvta_generic_to_shared(g_ring) : 0u;
    const int o_dz = LX::kBytes * threads, o_dy = 2 * LX::kBytes * threads, o_h = o_dy + LH::kBytes * threads;
    const int stage_bytes = (2 * LX::kBytes + (HAS_H ? 2 : 1) * LH::kBytes) * threads;
    Pack<TX, E> rz[RING ? 1 : U], rdz[RING ? 1 : U];
    Pack<TH, E> rh[RING ? 1 : U], rdy[RING ? 1 : U];
    if constexpr (RING) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            char* s = g_ring + i * stage_bytes;
            LX::clear(s, threads, tid, t, T, C, !has_y);
            LH::clear(s + o_dy, threads, tid, t, T, C, !has_y);
            LX::clear(s + o_dz, threads, tid, t, T, C, !a.dz);
            if constexpr (HAS_H) LH::clear(s + o_h, threads, tid, t, T, C, false);
        }
    } else {
        clear_units<TX, E>(rz);
        clear_units<TX, E>(rdz);
        clear_units<TH, E>(rdy);
        clear_units<TH, E>(rh);
    }
    auto fetch = [&](int64_t r, int stage) {
        if constexpr (RING) {
            if (r < r1) {
                const uint32_t s = ring + stage * stage_bytes;
                if (has_y) {
                    LX::fetch(s, threads, tid, (const TX*)a.z + r * a.ld_z, t, T, C);
                    LH::fetch(s + o_dy, threads, tid, (const TH*)a.dy + r * a.ld_dy, t, T, C);
                }
                if (a.dz) LX::fetch(s + o_dz, threads, tid, (const TX*)a.dz + r * a.ld_dz, t, T, C);
                if constexpr (HAS_H) LH::fetch(s + o_h, threads, tid, (const TH*)a.h + r * a.ld_h, t, T, C);
            }
            cp_commit();
        } else if (r < r1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                if (c < C) {
                    if (has_y) {
                        load(rz[u], (const TX*)a.z + r * a.ld_z + c);
                        load(rdy[u], (const TH*)a.dy + r * a.ld_dy + c);
                    }
                    if (a.dz) load(rdz[u], (const TX*)a.dz + r * a.ld_dz + c);
                    if (HAS_H) load(rh[u], (const TH*)a.h + r * a.ld_h + c);
                }
            }
        }
    };
#pragma unroll
    for (int i = 0; i < (RING ? D : 1); ++i) fetch(r0 + i * step, i);

    // The vectors stay in registers, or where these are too few (the widest teams) in shared memory behind the
    // ring, read again for each use.
    constexpr bool VSM = vec_shared(MAXT, sizeof(TX) + sizeof(TH) == 8);
    const uint32_t vec = (uint32_t)__cvta_generic_to_shared(g_ring) + (RING ? D * stage_bytes : 0) + tid * 16;
    auto keep = [&](const F2 (&v)[4], int which) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(vec + (2 * which + i) * threads * 16), "l"(v[2 * i].v),
                         "l"(v[2 * i + 1].v) : "memory");
    };
    auto get = [&](F2 (&v)[4], const F2 (&regs)[4], int which) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (VSM) {
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2 * i].v), "=l"(v[2 * i + 1].v)
                             : "r"(vec + (2 * which + i) * threads * 16) : "memory");
            } else {
                v[2 * i] = regs[2 * i];
                v[2 * i + 1] = regs[2 * i + 1];
            }
        }
    };
    int stage = 0;
    bool first = true;
    for (int64_t r = r0;;) {              // over the segment's groups
        const int64_t end = !whole || (g + 1) * a.rpg > r1 ? r1 : (g + 1) * a.rpg;
        F2 mul_[4], gate_[4];
        {
            float m[8], q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = q[i] = 1.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                float s[E];
                if (c < C) {
                    if (a.w) load_vec<E>(m + u * E, a.w + c);
                    if (a.scale) {
                        load_vec<E>(s, a.scale + g * a.ld_scale + c);
#pragma unroll
                        for (int e = 0; e < E; ++e) m[u * E + e] *= 1.f + s[e];
                    }
                    if (HAS_H) {
                        if (a.gate) load_vec<E>(q + u * E, a.gate + g * a.ld_gate + c);
                        if (a.w_post) {
                            load_vec<E>(s, a.w_post + c);
#pragma unroll
                            for (int e = 0; e < E; ++e) q[u * E + e] *= s[e];
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mul_[i] = f2(in(2 * i) ? m[2 * i] : 0.f, in(2 * i + 1) ? m[2 * i + 1] : 0.f);
                gate_[i] = f2(in(2 * i) ? q[2 * i] : 0.f, in(2 * i + 1) ? q[2 * i + 1] : 0.f);
            }
            if constexpr (VSM) {
                keep(mul_, 0);
                if constexpr (HAS_H) keep(gate_, 1);
            }
        }

        F2 sA[4], sD[4], sB[HAS_H ? 4 : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sA[i] = sD[i] = f2(0.f);
            if constexpr (HAS_H) sB[i] = f2(0.f);
        }

        // Teams of several warps take two rows at a time in part, so that a row has one barrier less: what the one's last
        // sum and the other's first one add up goes together.  The second row's values are read twice from the ring.
        // 61440 x 2048, layer norm: 251 -> 243 us, 13269 x 4096 128 -> 117; 8191 x 5120, two rms norms: 109 -> 98.
        [[maybe_unused]] auto store_dx = [&](int64_t row, const F2 (&d)[4]) {
            F2 o[4];
            const F2 res = f2(HAS_H ? a.res : 1.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = HAS_H ? d[i] * res : d[i];
            put_units<TX, E>((TX*)a.dx + row * a.ld_dx, o, t, T, C);
        };
        if constexpr (RING && D >= 2 && MAXT > 32 && MAXT < 1024) {      // with 64 registers it spills
            const char* base = g_ring;
            if constexpr (BR == kNormed) {
                if (!whole && a.norm == PRISM_NORM_RMS && a.post == PRISM_NORM_RMS) {
                    F2 d[4], h[4];
                    float rh_ = 0.f, last = 0.f;               // of the row before: 1/rms of h, sum of dn ∘ nh
                    for (bool have = false;; have = true) {
                        const bool more = r < end;
                        if (!more && !have) break;
                        const char* s = base + stage * stage_bytes;
                        float v[4] = {last, 0.f, 0.f, 0.f};
                        if (more) {
                            cp_wait<D - 1>();
                            F2 z[4], dy[4], x[4], mul[4], q[3];
                            LX::read(z, s, threads, tid);
                            LH::read(dy, s + o_dy, threads, tid);
                            LH::read(x, s + o_h, threads, tid);
                            get(mul, mul_, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const F2 c = dy[i] * mul[i];
                                q[0] = i ? fma(z[i], z[i], q[0]) : z[i] * z[i];
                                q[1] = i ? fma(c, z[i], q[1]) : c * z[i];
                                q[2] = i ? fma(x[i], x[i], q[2]) : x[i] * x[i];
                            }
#pragma unroll
                            for (int i = 0; i < 3; ++i) v[1 + i] = sum(q[i]);
                        }
                        team.sum(v);
                        if (have) {
                            const F2 mdn = f2(-v[0] * inv_c), rr = f2(rh_);
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[i] = rr * fma(h[i], mdn, d[i]);
                            put_units<TH, E>((TH*)a.dh + (r - step) * a.ld_dh, d, t, T, C);
                        }
                        if (!more) break;
                        const float rs = rsqrtf(v[1] * inv_c + a.eps), mcn = v[2] * rs * inv_c;
                        rh_ = rsqrtf(v[3] * inv_c + a.eps);
                        {
                            F2 z[4], dy[4], mul[4];
                            LX::read(z, s, threads, tid);
                            LH::read(dy, s + o_dy, threads, tid);
                            LX::read(d, s + o_dz, threads, tid);
                            get(mul, mul_, 0);
                            const F2 rs2 = f2(rs), mcn2 = f2(-mcn);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const F2 n = z[i] * rs2;
                                sA[i] = fma(dy[i], n, sA[i]);
                                sD[i] = sD[i] + dy[i];
                                d[i] = fma(rs2, fma(n, mcn2, dy[i] * mul[i]), d[i]);
                            }
                        }
                        store_dx(r, d);
                        F2 gate[4], q = f2(0.f);
                        LH::read(h, s + o_h, threads, tid);
                        get(gate, gate_, 1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = h[i] * f2(rh_);
                            sB[i] = fma(d[i], h[i], sB[i]);
                            d[i] = d[i] * gate[i];
                            q = fma(d[i], h[i], q);
                        }
                        last = sum(q);
                        fetch(r + D * step, stage);
                        stage = stage + 1 == D ? 0 : stage + 1;
                        r += step;
                    }
                }
            } else {
                if (!whole && a.norm == PRISM_NORM_LAYER && r < end) {
                    // sums of z and of c = dy ∘ mul over the row in the ring at s
                    auto first_sums = [&](const char* s, float* v) {
                        F2 z[4], dy[4], mul[4];
                        LX::read(z, s, threads, tid);
                        LH::read(dy, s + o_dy, threads, tid);
                        get(mul, mul_, 0);
                        F2 q = dy[0] * mul[0];
#pragma unroll
                        for (int i = 1; i < 4; ++i) q = fma(dy[i], mul[i], q);
                        v[0] = sum((z[0] + z[1]) + (z[2] + z[3]));
                        v[1] = sum(q);
                    };
                    float m[2];
                    cp_wait<D - 1>();
                    first_sums(base + stage * stage_bytes, m);
                    team.sum(m);
                    for (; r < end; r += step) {
                        const char* s = base + stage * stage_bytes;
                        const int after = stage + 1 == D ? 0 : stage + 1;
                        const float mz = -mean_of(m[0], fc, inv_c), mc = m[1] * inv_c;
                        F2 z[4], dy[4], mul[4], q[2];
                        LX::read(z, s, threads, tid);
                        LH::read(dy, s + o_dy, threads, tid);
                        get(mul, mul_, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            z[i] = z[i] + pair(mz, i);
                            q[0] = i ? fma(z[i], z[i], q[0]) : z[i] * z[i];
                            q[1] = i ? fma(dy[i] * mul[i], z[i], q[1]) : dy[i] * mul[i] * z[i];
                        }
                        float v[4] = {sum(q[0]), sum(q[1]), 0.f, 0.f};
                        if (r + step < end) {
                            cp_wait<D - 2>();
                            first_sums(base + after * stage_bytes, v + 2);
                        }
                        team.sum(v);
                        const float rs = rsqrtf(v[0] * inv_c + a.eps), mcn = v[1] * rs * inv_c;
                        const F2 rs2 = f2(rs), mcn2 = f2(-mcn);
                        F2 d[4];
                        LX::read(d, s + o_dz, threads, tid);
                        if constexpr (VSM) get(mul, mul_, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const F2 n = z[i] * rs2;
                            sA[i] = fma(dy[i], n, sA[i]);
                            sD[i] = sD[i] + dy[i];
                            d[i] = fma(rs2, fma(n, mcn2, fma(dy[i], mul[i], pair(-mc, i))), d[i]);
                        }
                        store_dx(r, d);
                        if constexpr (HAS_H) {
                            F2 h[4], gate[4];
                            LH::read(h, s + o_h, threads, tid);
                            get(gate, gate_, 1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                sB[i] = fma(d[i], h[i], sB[i]);
                                d[i] = d[i] * gate[i];
                            }
                            put_units<TH, E>((TH*)a.dh + r * a.ld_dh, d, t, T, C);
                        }
                        fetch(r + D * step, stage);
                        stage = after;
                        m[0] = v[2];
                        m[1] = v[3];
                    }
                }
            }
        }
        for (; r < end; r += step) {
            F2 z[4], dy[4], d[4], h[HAS_H ? 4 : 1];
            if constexpr (RING) {
                cp_wait<D - 1>();
                const char* s = g_ring + stage * stage_bytes;
                LX::read(z, s, threads, tid);
                LH::read(dy, s + o_dy, threads, tid);
                LX::read(d, s + o_dz, threads, tid);
                if constexpr (HAS_H) LH::read(h, s + o_h, threads, tid);
            } else {
                unpack_units<TX, E>(rz, z);
                unpack_units<TH, E>(rdy, dy);
                unpack_units<TX, E>(rdz, d);
                if constexpr (HAS_H) unpack_units<TH, E>(rh, h);
                fetch(r + step, 0);
            }

            // means first (layer): of z, of c = dy ∘ mul and of h
            constexpr int NS = BR == kNormed ? 3 : 2;
            float mc = 0.f;
            if (a.norm == PRISM_NORM_LAYER || (BR == kNormed && a.post == PRISM_NORM_LAYER)) {
                F2 mul[4];
                get(mul, mul_, 0);
                F2 q[3] = {z[0], dy[0] * mul[0], HAS_H ? h[0] : z[0]};
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    q[0] = q[0] + z[i];
                    q[1] = fma(dy[i], mul[i], q[1]);
                    if constexpr (BR == kNormed) q[2] = q[2] + h[i];
                }
                float s[NS];
#pragma unroll
                for (int i = 0; i < NS; ++i) s[i] = sum(q[i]);
                team.sum(s);
                if (a.norm == PRISM_NORM_LAYER) {
                    const float mz = -mean_of(s[0], fc, inv_c);
                    mc = s[1] * inv_c;
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = z[i] + pair(mz, i);
                }
                if constexpr (BR == kNormed) {
                    if (a.post == PRISM_NORM_LAYER) {
                        const float mh = -mean_of(s[NS - 1], fc, inv_c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = h[i] + pair(mh, i);
                    }
                }
            }
            // second moments, and c against z
            float rh_ = 1.f;
            if (has_y || BR == kNormed) {
                F2 q[3], mul[4];
                get(mul, mul_, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 c = dy[i] * mul[i];
                    q[0] = i ? fma(z[i], z[i], q[0]) : z[i] * z[i];
                    q[1] = i ? fma(c, z[i], q[1]) : c * z[i];
                    if constexpr (BR == kNormed) q[2] = i ? fma(h[i], h[i], q[2]) : h[i] * h[i];
                }
                float s[NS];
#pragma unroll
                for (int i = 0; i < NS; ++i) s[i] = sum(q[i]);
                team.sum(s);
                if constexpr (BR == kNormed) rh_ = rsqrtf(s[NS - 1] * inv_c + a.eps);
                if (has_y) {
                    const float rs = rsqrtf(s[0] * inv_c + a.eps), mcn = s[1] * rs * inv_c;
                    const F2 rs2 = f2(rs), mcn2 = f2(-mcn);
                    if constexpr (VSM) get(mul, mul_, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 n = z[i] * rs2;
                        sA[i] = fma(dy[i], n, sA[i]);
                        sD[i] = sD[i] + dy[i];
                        d[i] = fma(rs2, fma(n, mcn2, fma(dy[i], mul[i], pair(-mc, i))), d[i]);
                    }
                }
            }
            store_dx(r, d);
            if constexpr (HAS_H) {
                F2 q[2], gate[4];
                get(gate, gate_, 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (BR == kNormed) h[i] = h[i] * f2(rh_);
                    sB[i] = fma(d[i], h[i], sB[i]);
                    d[i] = d[i] * gate[i];
                    if constexpr (BR == kNormed) {
                        q[0] = i ? q[0] + d[i] : d[i];
                        q[1] = i ? fma(d[i], h[i], q[1]) : d[i] * h[i];
                    }
                }
                if constexpr (BR == kNormed) {
                    float s[2] = {sum(q[0]), sum(q[1])};
                    team.sum(s);
                    const F2 md = f2(a.post == PRISM_NORM_LAYER ? -s[0] * inv_c : 0.f), mdn = f2(-s[1] * inv_c), rr = f2(rh_);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = rr * fma(h[i], mdn, d[i] + md);
                }
                put_units<TH, E>((TH*)a.dh + r * a.ld_dh, d, t, T, C);
            }
            if constexpr (RING) {             // the row's own values have been used: their place is free
                fetch(r + D * step, stage);
                stage = stage + 1 == D ? 0 : stage + 1;
            }
        }
        float fA[8], fD[8], fB[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = both(sA[i]);
            fA[2 * i] = f.x; fA[2 * i + 1] = f.y;
            f = both(sD[i]);
            fD[2 * i] = f.x; fD[2 * i + 1] = f.y;
            f = both(sB[HAS_H ? i : 0]);
            fB[2 * i] = f.x; fB[2 * i + 1] = f.y;
        }
        if (MAXT == 32 && !whole) {
            // the CTA's teams add up through shared memory, whose rows have all been used
            if (!a.part) break;
            if constexpr (RING) cp_wait<0>();
            __syncthreads();
            float* all = reinterpret_cast<float*>(g_ring);
            const int width = 8 * T;
            float* mine = all + threadIdx.y * 3 * width;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = ((i / E) * T + t) * E + i % E;
                mine[c] = fA[i];
                mine[width + c] = fD[i];
                if constexpr (HAS_H) mine[2 * width + c] = fB[i];
            }
            __syncthreads();
            for (int i = threadIdx.y * T + t; i < (HAS_H ? 3 : 2) * width; i += 256) {
                float v = 0.f;
                for (int k = 0; k < (int)blockDim.y; ++k) v += all[k * 3 * width + i];
                const int which = i / width, c = i - which * width;
                if (c < C) a.part[(seg * 3 + which) * C + c] = v;
            }
            break;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * E;
            if (c >= C) continue;
            float w[E], b[E], f[E];
            if (whole && (a.dscale || a.dshift || a.part)) {
#pragma unroll
                for (int e = 0; e < E; ++e) { w[e] = 1.f; b[e] = f[e] = 0.f; }
                if (a.dscale) {
                    if (a.w) load_vec<E>(w, a.w + c);
                    if (a.b) load_vec<E>(b, a.b + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) w[e] = fmaf(w[e], fA[u * E + e], b[e] * fD[u * E + e]);
                    store_vec<E>(a.dscale + g * C + c, w);
                }
                if (a.dshift) store_vec<E>(a.dshift + g * C + c, fD + u * E);
                if (a.scale) load_vec<E>(f, a.scale + g * a.ld_scale + c);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    fA[u * E + e] = fmaf(f[e], fA[u * E + e], fA[u * E + e]);
                    fD[u * E + e] = fmaf(f[e], fD[u * E + e], fD[u * E + e]);
                }
            }
            if constexpr (HAS_H) {
                if (whole && (a.dgate || a.part)) {
#pragma unroll
                    for (int e = 0; e < E; ++e) w[e] = f[e] = 1.f;
                    if (a.w_post) load_vec<E>(w, a.w_post + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) w[e] *= fB[u * E + e];
                    if (a.dgate) store_vec<E>(a.dgate + g * C + c, w);
                    if (a.gate) load_vec<E>(f, a.gate + g * a.ld_gate + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) fB[u * E + e] *= f[e];
                }
            }
            if (a.part) {
                // the thread's own places: a run of groups adds up there
                float* p = a.part + seg * 3 * C + c;
                if (!first) {
                    load_own<E>(w, p);
                    load_own<E>(b, p + C);
#pragma unroll
                    for (int e = 0; e < E; ++e) { fA[u * E + e] += w[e]; fD[u * E + e] += b[e]; }
                    if constexpr (HAS_H) {
                        load_own<E>(w, p + 2 * C);
#pragma unroll
                        for (int e = 0; e < E; ++e) fB[u * E + e] += w[e];
                    }
                }
                store_vec<E>(p, fA + u * E);
                store_vec<E>(p + C, fD + u * E);
                if constexpr (HAS_H) store_vec<E>(p + 2 * C, fB + u * E);
            }
        }
        if (end >= r1) break;
        ++g;
        first = false;
    }
    if constexpr (RING) cp_wait<0>();
    let_next_start();
}

// Channels of the widest access, where stream and branch differ: 16 bytes of the branch forwards (f32 and bf16,
// 61440 x 2048: 236 us, 16 bytes of the stream 243), and of the stream backwards (372; of the branch 477: a lane's
// eight floats are then two copies that leave gaps in a warp's access).
template <typename T> constexpr int wide_unit() { return 16 / (int)sizeof(T); }
// threads of a team: 8 channels a thread; 8, 16 or a whole number of warps
inline int team_threads(int C) {
    const int n = (C + 7) / 8;
    return n <= 8 ? 8 : n <= 16 ? 16 : (n + 31) / 32 * 32;
}
// teams of a CTA: one, or 256 threads of teams within a warp
inline int cta_teams(int C) {
    const int t = team_threads(C);
    return t <= 32 ? 256 / t : 1;
}
// The kernel's MAXT for a team, and the CTAs of that many threads that an SM takes: as many as the registers allow
// without spills, or with few.  Forward: 2048 channels three CTAs 501 us, two 571, four with 32 bytes of spills 597
// (131072 rows); 4096 two 75, one 85 (13269 rows); 5416 without a branch two 72, one 91.  Backward: 2048 two 361 and
// three with 32 bytes 421 (61440 rows, before the pairs of fp32); 2560 two 72, one 92 (13269 rows).
constexpr int team_bucket(int threads) {
    for (int b : {32, 256, 320, 384, 512, 640, 768})
        if (threads <= b) return b;
    return 1024;
}
constexpr int fwd_ctas(int maxt, int unit, bool branch) {
    if (maxt <= 256) return maxt == 32 || unit < 4 ? 2 : 3;
    if (!branch && unit >= 4) return maxt <= 384 ? 3 : maxt <= 768 ? 2 : 1;
    return maxt <= 384 || (unit >= 4 && maxt <= 512) ? 2 : 1;
}
constexpr int bwd_ctas(int maxt, bool f32) { return maxt <= 320 || (maxt <= 384 && !f32) ? 2 : 1; }    // f32: stream and branch
// teams that run at a time on an SM
inline int sm_teams(int C, int ctas) {
    const int t = team_threads(C), most = team_bucket(t) == 32 ? 256 : team_bucket(t);
    return ctas * most / t;
}

// Leave for a kernel's dynamic shared memory, where with the static part it passes the 48 KB that need none.  FULL is
// what its widest team takes, not the call's: the limit is the kernel's, and a thread with narrower rows may set it
// between another's setting and its launch.
template <int FULL, typename F> bool allow_shared(F kernel) {
    static_assert(FULL <= 224 << 10, "with the static part, what a CTA can have");
    return FULL <= 40 << 10 || taken(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FULL));
}

// rows ahead in the backward (2: 5% slower, 4: the same), fewer where the widest rows leave no room
constexpr int kRowsAhead = 3;
template <typename TX, typename TH, int E, int MAXT, int H>
prism_status_t launch_bwd_one(const BwdArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
    constexpr bool f32 = sizeof(TX) + sizeof(TH) == 8;
    constexpr int CTAS = bwd_ctas(MAXT, f32), row = 8 * (int)(2 * sizeof(TX) + (H ? 2 : 1) * sizeof(TH));
    constexpr int threads = MAXT == 32 ? 256 : MAXT, vec = vec_shared(MAXT, f32) ? (H ? 64 : 32) : 0;
    constexpr int most = ((216 << 10) / CTAS - vec * threads) / (row * threads);
    constexpr int D = most < 1 ? 1 : most > kRowsAhead ? kRowsAhead : most;
    auto kernel = &k_block_norm_bwd<TX, TH, E, MAXT, H, CTAS, D>;
    constexpr int thread = (Lane<TX, E>::kAsync && Lane<TH, E>::kAsync ? D * row : 0) + vec;
    constexpr int least = MAXT == 32 ? kTeamSums : 0, full = thread * threads > least ? thread * threads : least;
    if (!allow_shared<full>(kernel)) return PRISM_ERR_CUDA;
    const int bytes = thread * (int)(block.x * block.y);
    kernel<<<grid, block, bytes > least ? bytes : least, s>>>(a);
    return PRISM_OK;
}
template <typename TX, typename TH, int E, int MAXT, int H>
prism_status_t launch_fwd_one(const FwdArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
    constexpr bool async = Lane<TX, E>::kAsync && Lane<TH, E>::kAsync && MAXT > 256;
    constexpr int row = 8 * (int)(sizeof(TX) + (H != kNoBranch ? sizeof(TH) : 0)), ctas = fwd_ctas(MAXT, E, H != kNoBranch);
    constexpr int most = (216 << 10) / ctas / (row * MAXT), D = !async ? 0 : most > kRowsAhead ? kRowsAhead : most;
    auto kernel = &k_block_norm_fwd<TX, TH, E, MAXT, H != kNoBranch, ctas, D>;
    if (!allow_shared<D * row * MAXT>(kernel)) return PRISM_ERR_CUDA;
    kernel<<<grid, block, D * row * (int)block.x, s>>>(a);
    return PRISM_OK;
}

// one launcher a pair of types (stream, branch); unit = channels an access
template <typename TX, typename TH> prism_status_t launch_fwd(const FwdArgs& a, int unit, cudaStream_t s);
template <typename TX, typename TH> prism_status_t launch_bwd(const BwdArgs& a, int unit, cudaStream_t s);

#define PRISM_BN_BY_SIZE(ONE, TX, TH, E, H)                                            \
    switch (team_bucket(block.x)) {                                                   \
        case 32: return ONE<TX, TH, E, 32, H>(a, grid, block, s);                     \
        case 256: return ONE<TX, TH, E, 256, H>(a, grid, block, s);                   \
        case 320: return ONE<TX, TH, E, 320, H>(a, grid, block, s);                   \
        case 384: return ONE<TX, TH, E, 384, H>(a, grid, block, s);                   \
        case 512: return ONE<TX, TH, E, 512, H>(a, grid, block, s);                   \
        case 640: return ONE<TX, TH, E, 640, H>(a, grid, block, s);                   \
        case 768: return ONE<TX, TH, E, 768, H>(a, grid, block, s);                   \
        default: return ONE<TX, TH, E, 1024, H>(a, grid, block, s);                   \
    }

#define PRISM_BN_BY_UNIT(ONE, TW, TX, TH, H)                                          \
    do {                                                                              \
        constexpr int kWide = wide_unit<TW>();                                        \
        if (unit == kWide) PRISM_BN_BY_SIZE(ONE, TX, TH, kWide, H)                    \
        if (unit == 2) PRISM_BN_BY_SIZE(ONE, TX, TH, 2, H)                            \
        PRISM_BN_BY_SIZE(ONE, TX, TH, 1, H)                                           \
    } while (0)

#define PRISM_BN_INSTANTIATE(TX, TH)                                                                   \
    template <> prism_status_t launch_fwd<TX, TH>(const FwdArgs& a, int unit, cudaStream_t s) {        \
        const dim3 block(team_threads(a.C), cta_teams(a.C));                                           \
        const int64_t want = (a.R + block.y - 1) / block.y;                                            \
        const int64_t most = kSMs * (int64_t)sm_teams(a.C, fwd_ctas(team_bucket(block.x), unit, a.h != nullptr)) / block.y;  \
        const dim3 grid((unsigned)(want < most ? want : most));                                        \
        if (a.h) PRISM_BN_BY_UNIT(launch_fwd_one, TH, TX, TH, kPlain);                                     \
        else PRISM_BN_BY_UNIT(launch_fwd_one, TH, TX, TH, kNoBranch);                                      \
    }                                                                                                  \
    template <> prism_status_t launch_bwd<TX, TH>(const BwdArgs& a, int unit, cudaStream_t s) {        \
        const dim3 block(team_threads(a.C), cta_teams(a.C));                                           \
        const dim3 grid((unsigned)(a.per_group > 0 ? a.segs : (a.segs + block.y - 1) / block.y));      \
        if (a.h && a.post != PRISM_NORM_NONE) PRISM_BN_BY_UNIT(launch_bwd_one, TX, TX, TH, kNormed);       \
        else if (a.h) PRISM_BN_BY_UNIT(launch_bwd_one, TX, TX, TH, kPlain);                                \
        else PRISM_BN_BY_UNIT(launch_bwd_one, TX, TX, TH, kNoBranch);                                      \
    }

}  // namespace bn
}  // namespace prism
