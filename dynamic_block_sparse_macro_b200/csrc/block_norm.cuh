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
// A row's threads hold eight channels each.  A thread takes only channels of the row into a sum: what its
// registers hold for places past the row's end is never used.
// Everything between a load and a store is fp32: statistics, means and column sums too.  A result
// that is stored as bf16 is rounded once, at its store; y comes from the unrounded z.
#pragma once

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
    // direct: each group is one segment and its gradients are written by the row kernel
    float *dgate, *dscale, *dshift;
    float* part;                       // [segments][3][C] column sums A, D, B; null: not wanted
    int64_t R, rpg, segs;              // segs = groups x segments a group
    int64_t ld_z, ld_h, ld_dz, ld_dy, ld_dx, ld_dh, ld_gate, ld_scale;
    int C, norm, post, per_group;
    float eps, res;
};

// The threads of a team hold U units of E consecutive channels each: unit u of thread t covers
// channels (u * threads + t) * E + [0, E), so that a warp's access to a unit is contiguous.
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

template <typename TX, typename TH, int E, int MAXT, bool HAS_H, int CTAS>
__global__ void __launch_bounds__(MAXT == 32 ? 256 : MAXT, CTAS) k_block_norm_fwd(const FwdArgs a) {
    constexpr int U = 8 / E;
    __shared__ float4 sums[Team<MAXT>::kBufs];
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

    Pack<TX, E> rx[U];
    Pack<TH, E> rh[U];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * E;
            if (c < C) {
                load(rx[u], x + r * a.ld_x + c);
                if (HAS_H) load(rh[u], h + r * a.ld_h + c);
            }
        }
    };
    fetch(r0);

    float mul[U * E], add[U * E], gate[HAS_H ? U * E : 1];
    auto vectors = [&](int64_t g) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * E;
            float s[E];
#pragma unroll
            for (int e = 0; e < E; ++e) { mul[u * E + e] = 1.f; add[u * E + e] = 0.f; }
            if constexpr (HAS_H) {
#pragma unroll
                for (int e = 0; e < E; ++e) gate[u * E + e] = 1.f;
            }
            if (c >= C) continue;
            if (a.norm != PRISM_NORM_NONE) {
                if (a.w) load_vec<E>(mul + u * E, a.w + c);
                if (a.b) load_vec<E>(add + u * E, a.b + c);
                if (a.scale) {
                    load_vec<E>(s, a.scale + g * a.ld_scale + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) { mul[u * E + e] *= 1.f + s[e]; add[u * E + e] *= 1.f + s[e]; }
                }
                if (a.shift) {
                    load_vec<E>(s, a.shift + g * a.ld_shift + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) add[u * E + e] += s[e];
                }
            }
            if constexpr (HAS_H) {
                if (a.gate) load_vec<E>(gate + u * E, a.gate + g * a.ld_gate + c);
                if (a.w_post) {
                    load_vec<E>(s, a.w_post + c);
#pragma unroll
                    for (int e = 0; e < E; ++e) gate[u * E + e] *= s[e];
                }
            }
        }
    };
    int64_t g = r0 / a.rpg, next = (g + 1) * a.rpg;
    vectors(g);

    for (int64_t r = r0; r < r1; r += step) {
        float v[U * E];
#pragma unroll
        for (int i = 0; i < U * E; ++i) v[i] = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if ((u * T + t) * E < C) unpack<E>(rx[u], v + u * E);
        float hv[HAS_H ? U * E : 1];
        if constexpr (HAS_H) {
#pragma unroll
            for (int i = 0; i < U * E; ++i) hv[i] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) unpack<E>(rh[u], hv + u * E);
        }
        if (r + step < r1) fetch(r + step);
        if (r >= next) {                  // steps are shorter than groups
            vectors(++g);
            next += a.rpg;
        }

        // mean (layer) and 1/std of the row held in f; f becomes f - mean
        auto stats = [&](float* f, int kind) {
            if (kind == PRISM_NORM_LAYER) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < U * E; ++i) s += f[i];
                const float m = mean_of(team.sum1(s), fc, inv_c);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if ((u * T + t) * E < C) {
#pragma unroll
                        for (int e = 0; e < E; ++e) f[u * E + e] -= m;
                    }
            }
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < U * E; ++i) q = fmaf(f[i], f[i], q);
            return rsqrtf(team.sum1(q) * inv_c + a.eps);
        };

        if constexpr (HAS_H) {
            if (a.post != PRISM_NORM_NONE) {
                const float rh_ = stats(hv, a.post);
#pragma unroll
                for (int i = 0; i < U * E; ++i) hv[i] *= rh_;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                if (c < C) {
#pragma unroll
                    for (int i = u * E; i < u * E + E; ++i) v[i] = fmaf(a.res, v[i], gate[i] * hv[i]);
                    Pack<TX, E> o;
                    pack<E>(o, v + u * E);
                    store((TX*)a.z + r * a.ld_z + c, o);
                }
            }
        }
        if (a.norm != PRISM_NORM_NONE) {
            const float rs = stats(v, a.norm);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                if (c < C) {
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = fmaf(v[u * E + e] * rs, mul[u * E + e], add[u * E + e]);
                    Pack<TH, E> p;
                    pack<E>(p, o);
                    store((TH*)a.y + r * a.ld_y + c, p);
                }
            }
        }
    }
}

template <typename TX, typename TH, int E, int MAXT, bool HAS_H, int CTAS>
__global__ void __launch_bounds__(MAXT == 32 ? 256 : MAXT, CTAS) k_block_norm_bwd(const BwdArgs a) {
    constexpr int U = 8 / E;
    __shared__ float4 sums[Team<MAXT>::kBufs];
    Team<MAXT> team;
    team.init(sums);
    const int t = threadIdx.x, T = blockDim.x, C = a.C;
    const int64_t seg = MAXT == 32 ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (seg >= a.segs) return;
    const int64_t g = seg / a.per_group;
    // segment s of a group takes its rows s, s + per_group, ...: all teams move over the rows together
    const int64_t r0 = g * a.rpg + (seg - g * a.per_group), step = a.per_group;
    int64_t r1 = (g + 1) * a.rpg;
    if (r1 > a.R) r1 = a.R;
    const float fc = (float)C, inv_c = 1.f / fc;
    const bool has_y = a.norm != PRISM_NORM_NONE;

    Pack<TX, E> rz[U], rdz[U];
    Pack<TH, E> rh[U], rdy[U];
    auto fetch = [&](int64_t r) {
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
    };
    if (r0 < r1) fetch(r0);

    float mul[U * E], gate[HAS_H ? U * E : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * T + t) * E;
        float s[E];
#pragma unroll
        for (int e = 0; e < E; ++e) mul[u * E + e] = 1.f;
        if constexpr (HAS_H) {
#pragma unroll
            for (int e = 0; e < E; ++e) gate[u * E + e] = 1.f;
        }
        if (c >= C) continue;
        if (a.w) load_vec<E>(mul + u * E, a.w + c);
        if (a.scale) {
            load_vec<E>(s, a.scale + g * a.ld_scale + c);
#pragma unroll
            for (int e = 0; e < E; ++e) mul[u * E + e] *= 1.f + s[e];
        }
        if constexpr (HAS_H) {
            if (a.gate) load_vec<E>(gate + u * E, a.gate + g * a.ld_gate + c);
            if (a.w_post) {
                load_vec<E>(s, a.w_post + c);
#pragma unroll
                for (int e = 0; e < E; ++e) gate[u * E + e] *= s[e];
            }
        }
    }

    float sA[U * E], sD[U * E], sB[HAS_H ? U * E : 1];
#pragma unroll
    for (int i = 0; i < U * E; ++i) sA[i] = sD[i] = 0.f;
    if constexpr (HAS_H) {
#pragma unroll
        for (int i = 0; i < U * E; ++i) sB[i] = 0.f;
    }

    for (int64_t r = r0; r < r1; r += step) {
        float z[U * E], dy[U * E], d[U * E], h[HAS_H ? U * E : 1];
#pragma unroll
        for (int i = 0; i < U * E; ++i) z[i] = dy[i] = d[i] = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if ((u * T + t) * E < C) {
                if (has_y) {
                    unpack<E>(rz[u], z + u * E);
                    unpack<E>(rdy[u], dy + u * E);
                }
                if (a.dz) unpack<E>(rdz[u], d + u * E);
            }
        if constexpr (HAS_H) {
#pragma unroll
            for (int i = 0; i < U * E; ++i) h[i] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) unpack<E>(rh[u], h + u * E);
        }
        if (r + step < r1) fetch(r + step);

        // means first (layer): of z, of c = dy ∘ mul and of h
        float mc = 0.f;
        if (a.norm == PRISM_NORM_LAYER || (HAS_H && a.post == PRISM_NORM_LAYER)) {
            float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) {
#pragma unroll
                    for (int i = u * E; i < u * E + E; ++i) {
                        s[0] += z[i];
                        s[1] = fmaf(dy[i], mul[i], s[1]);
                        if constexpr (HAS_H) s[2] += h[i];
                    }
                }
            team.sum(s);
            const float mz = a.norm == PRISM_NORM_LAYER ? mean_of(s[0], fc, inv_c) : 0.f;
            const float mh = a.post == PRISM_NORM_LAYER ? mean_of(s[2], fc, inv_c) : 0.f;
            mc = a.norm == PRISM_NORM_LAYER ? s[1] * inv_c : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        z[u * E + e] -= mz;
                        if constexpr (HAS_H) h[u * E + e] -= mh;
                    }
                }
        }
        // second moments, and c against z
        float rh_ = 1.f;
        if (has_y || (HAS_H && a.post != PRISM_NORM_NONE)) {
            float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) {
#pragma unroll
                    for (int i = u * E; i < u * E + E; ++i) {
                        s[0] = fmaf(z[i], z[i], s[0]);
                        s[1] = fmaf(dy[i] * mul[i], z[i], s[1]);
                        if constexpr (HAS_H) s[2] = fmaf(h[i], h[i], s[2]);
                    }
                }
            team.sum(s);
            if (has_y) {
                const float rs = rsqrtf(s[0] * inv_c + a.eps), mcn = s[1] * rs * inv_c;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if ((u * T + t) * E < C) {
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const int i = u * E + e;
                            const float n = z[i] * rs;
                            sA[i] = fmaf(dy[i], n, sA[i]);
                            sD[i] += dy[i];
                            d[i] = fmaf(rs, fmaf(dy[i], mul[i], -mc) - n * mcn, d[i]);
                        }
                    }
            }
            if (HAS_H && a.post != PRISM_NORM_NONE) rh_ = rsqrtf(s[2] * inv_c + a.eps);
        }
        const float res = HAS_H ? a.res : 1.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (u * T + t) * E;
            if (c < C) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = res * d[u * E + e];
                Pack<TX, E> p;
                pack<E>(p, o);
                store((TX*)a.dx + r * a.ld_dx + c, p);
            }
        }
        if constexpr (HAS_H) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((u * T + t) * E < C) {
#pragma unroll
                    for (int i = u * E; i < u * E + E; ++i) {
                        h[i] *= rh_;
                        sB[i] = fmaf(d[i], h[i], sB[i]);
                        d[i] *= gate[i];
                        s[0] += d[i];
                        s[1] = fmaf(d[i], h[i], s[1]);
                    }
                }
            float md = 0.f, mdn = 0.f;
            if (a.post != PRISM_NORM_NONE) {
                team.sum(s);
                md = a.post == PRISM_NORM_LAYER ? s[0] * inv_c : 0.f;
                mdn = s[1] * inv_c;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (u * T + t) * E;
                if (c < C) {
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = rh_ * (d[u * E + e] - md - h[u * E + e] * mdn);
                    Pack<TH, E> p;
                    pack<E>(p, o);
                    store((TH*)a.dh + r * a.ld_dh + c, p);
                }
            }
        }
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (u * T + t) * E;
        if (c >= C) continue;
        if (a.part) {
            float* p = a.part + seg * 3 * C + c;
            store_vec<E>(p, sA + u * E);
            store_vec<E>(p + C, sD + u * E);
            if constexpr (HAS_H) store_vec<E>(p + 2 * C, sB + u * E);
        }
        if (a.dscale) {
            float w[E], b[E];
#pragma unroll
            for (int e = 0; e < E; ++e) { w[e] = 1.f; b[e] = 0.f; }
            if (a.w) load_vec<E>(w, a.w + c);
            if (a.b) load_vec<E>(b, a.b + c);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = fmaf(w[e], sA[u * E + e], b[e] * sD[u * E + e]);
            store_vec<E>(a.dscale + g * C + c, w);
        }
        if (a.dshift) store_vec<E>(a.dshift + g * C + c, sD + u * E);
        if constexpr (HAS_H) {
            if (a.dgate) {
                float w[E];
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = 1.f;
                if (a.w_post) load_vec<E>(w, a.w_post + c);
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] *= sB[u * E + e];
                store_vec<E>(a.dgate + g * C + c, w);
            }
        }
    }
}

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
// the kernel's MAXT for a team, and the CTAs of at most that many threads that its registers leave room for on an SM
constexpr int team_bucket(int threads) {
    return threads <= 32 ? 32 : threads <= 256 ? 256 : threads <= 384 ? 384 : threads <= 512 ? 512 : threads <= 768 ? 768 : 1024;
}
constexpr int fwd_ctas(int maxt) { return maxt <= 256 ? 3 : maxt <= 384 ? 2 : 1; }
constexpr int bwd_ctas(int maxt) { return maxt <= 256 ? 2 : 1; }
// teams that run at a time on an SM
inline int sm_teams(int C, int ctas) {
    const int t = team_threads(C), most = team_bucket(t) == 32 ? 256 : team_bucket(t);
    return ctas * most / t;
}

// one launcher a pair of types (stream, branch); unit = channels an access
template <typename TX, typename TH> void launch_fwd(const FwdArgs& a, int unit, cudaStream_t s);
template <typename TX, typename TH> void launch_bwd(const BwdArgs& a, int unit, cudaStream_t s);

#define PRISM_BN_BY_SIZE(KERNEL, CTAS, TX, TH, E, H)                                                     \
    do {                                                                                                \
        switch (team_bucket(block.x)) {                                                                 \
            case 32: KERNEL<TX, TH, E, 32, H, CTAS(32)><<<grid, block, 0, s>>>(a); break;               \
            case 256: KERNEL<TX, TH, E, 256, H, CTAS(256)><<<grid, block, 0, s>>>(a); break;            \
            case 384: KERNEL<TX, TH, E, 384, H, CTAS(384)><<<grid, block, 0, s>>>(a); break;            \
            case 512: KERNEL<TX, TH, E, 512, H, CTAS(512)><<<grid, block, 0, s>>>(a); break;            \
            case 768: KERNEL<TX, TH, E, 768, H, CTAS(768)><<<grid, block, 0, s>>>(a); break;            \
            default: KERNEL<TX, TH, E, 1024, H, CTAS(1024)><<<grid, block, 0, s>>>(a); break;           \
        }                                                                                               \
    } while (0)

#define PRISM_BN_BY_UNIT(KERNEL, CTAS, TX, TH, H)                                      \
    do {                                                                              \
        if (unit == 8) PRISM_BN_BY_SIZE(KERNEL, CTAS, TX, TH, 8, H);                  \
        else if (unit == 2) PRISM_BN_BY_SIZE(KERNEL, CTAS, TX, TH, 2, H);             \
        else PRISM_BN_BY_SIZE(KERNEL, CTAS, TX, TH, 1, H);                            \
    } while (0)

#define PRISM_BN_INSTANTIATE(TX, TH)                                                                   \
    template <> void launch_fwd<TX, TH>(const FwdArgs& a, int unit, cudaStream_t s) {                  \
        const dim3 block(team_threads(a.C), cta_teams(a.C));                                           \
        const int64_t want = (a.R + block.y - 1) / block.y;                                            \
        const int64_t most = kSMs * (int64_t)sm_teams(a.C, fwd_ctas(team_bucket(block.x))) / block.y;  \
        const dim3 grid((unsigned)(want < most ? want : most));                                        \
        if (a.h) PRISM_BN_BY_UNIT(k_block_norm_fwd, fwd_ctas, TX, TH, true);                           \
        else PRISM_BN_BY_UNIT(k_block_norm_fwd, fwd_ctas, TX, TH, false);                              \
    }                                                                                                  \
    template <> void launch_bwd<TX, TH>(const BwdArgs& a, int unit, cudaStream_t s) {                  \
        const dim3 block(team_threads(a.C), cta_teams(a.C));                                           \
        const dim3 grid((unsigned)((a.segs + block.y - 1) / block.y));                                 \
        if (a.h) PRISM_BN_BY_UNIT(k_block_norm_bwd, bwd_ctas, TX, TH, true);                           \
        else PRISM_BN_BY_UNIT(k_block_norm_bwd, bwd_ctas, TX, TH, false);                              \
    }

}  // namespace bn
}  // namespace prism
