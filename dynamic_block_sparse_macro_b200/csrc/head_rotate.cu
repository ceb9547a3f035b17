// The norm of each head's channels and the rotation by the token's place in
// the grid, for Q and K before the attention.
//
//   n = N_rms(x) ∘ w over the head's d channels (or n = x)
//   (n_a, n_b) -> (n_a cos - n_b sin, n_a sin + n_b cos) for each pair (a, b)
//
// and backwards, with dn the pairs of dr turned back (by -angle), c = dn ∘ w, n = x r:
//   dx = r (c - n mean(c ∘ n)),  dw = sum over tokens and heads of dn ∘ n.
//
// Bound by HBM: each element is read and written once.  d/8 lanes hold a head's row, four channel pairs
// each, so that a pair turns within its lane in either pairing, and walk the heads of one token, so that the token's place, its cosines and its sines (a
// table of one row an axis position, which stays in L1) are fetched once for all its heads.  All
// arithmetic is fp32; the result is rounded once.
#include <initializer_list>
#include <type_traits>

#include "rows.cuh"

namespace prism {
namespace rot {

using namespace rows;

struct Side {
    const void *x, *dr;
    const float* w;
    void* out;
    int64_t ld_x, ld_dr, ld_out;
    int heads, parts;
};

struct Args {
    Side side[2];
    const float2* table;
    float* part;                     // backward: [2][gridDim.x][d] sums of dw; null: not wanted
    int64_t tokens;
    int T, H, W, nT, nH, nW, turn, norm;     // turn: the pairs that turn, nT + nH + nW
    float eps;
};

// Sums over the LPH lanes of a head.  Of two values each half of the lanes takes one over, so that the second
// costs one exchange more and not as many again.
template <int LPH> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LPH> __device__ __forceinline__ void lanes_sum(float& v, float& w, int l) {
    const bool hi = l & (LPH / 2);
    float k = (hi ? w : v) + __shfl_xor_sync(0xffffffffu, hi ? v : w, LPH / 2);
#pragma unroll
    for (int o = LPH / 4; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    const float other = __shfl_xor_sync(0xffffffffu, k, LPH / 2);
    v = hi ? other : k;
    w = hi ? k : other;
}

// A lane's four channel pairs: the first members in a, the second in b.
struct Pairs {
    F2 a[2], b[2];
};
// as they lie in memory: eight channels in a row (interleaved), or four of each half of the head
template <typename T, bool HALF> struct Raw {
    Pack<T, HALF ? 4 : 8> p[HALF ? 2 : 1];
};
template <int D, bool HALF> __device__ __forceinline__ int lane_at(int l) { return HALF ? 4 * l : 8 * l; }
template <typename T, int D, bool HALF> __device__ __forceinline__ void load_raw(Raw<T, HALF>& r, const T* head) {
    load(r.p[0], head);
    if constexpr (HALF) load(r.p[1], head + D / 2);
}
template <typename T, bool HALF> __device__ __forceinline__ Pairs pairs_of(const Raw<T, HALF>& r) {
    Pairs v;
    if constexpr (HALF) {
        float a[4], b[4];
        unpack<4>(r.p[0], a);
        unpack<4>(r.p[1], b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v.a[i] = f2(a[2 * i], a[2 * i + 1]);
            v.b[i] = f2(b[2 * i], b[2 * i + 1]);
        }
    } else {
        float f[8];
        unpack<8>(r.p[0], f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v.a[i] = f2(f[4 * i], f[4 * i + 2]);
            v.b[i] = f2(f[4 * i + 1], f[4 * i + 3]);
        }
    }
    return v;
}
template <typename T, int D, bool HALF> __device__ __forceinline__ void store_pairs(T* head, const Pairs& v) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 f = both(v.a[i]);
        a[2 * i] = f.x; a[2 * i + 1] = f.y;
        f = both(v.b[i]);
        b[2 * i] = f.x; b[2 * i + 1] = f.y;
    }
    if constexpr (HALF) {
        Pack<T, 4> p;
        pack<4>(p, a);
        store(head, p);
        pack<4>(p, b);
        store(head + D / 2, p);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = a[i]; f[2 * i + 1] = b[i]; }
        Pack<T, 8> p;
        pack<8>(p, f);
        store(head, p);
    }
}
// per-channel floats of a lane (weights, their sums)
template <int D, bool HALF> __device__ __forceinline__ int channel(int l, int i, bool second) {
    return HALF ? 4 * l + i + (second ? D / 2 : 0) : 8 * l + 2 * i + second;
}

// cosine and sine of the lane's pairs for one token
__device__ __forceinline__ void angles(const Args& a, uint32_t token, int l, F2 (&cs)[2], F2 (&sn)[2]) {
    const uint32_t hw = (uint32_t)a.H * a.W, at = token % ((uint32_t)a.T * hw);
    const uint32_t pt = at / hw, r = at - pt * hw, ph = r / a.W, pw = r - ph * a.W;
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = l * 4 + j, q = p - a.nT, s = q - a.nH;
        const int at_t = pt * a.nT + p, at_h = a.T * a.nT + ph * a.nH + q, at_w = a.T * a.nT + a.H * a.nH + pw * a.nW + s;
        v[j] = make_float2(1.f, 0.f);
        if (s < a.nW) v[j] = __ldg(a.table + (q < 0 ? at_t : s < 0 ? at_h : at_w));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        cs[i] = f2(v[2 * i].x, v[2 * i + 1].x);
        sn[i] = f2(v[2 * i].y, v[2 * i + 1].y);
    }
}

// Pairs from `turn` on do not turn (STILL: there are some).  A sine of 0 does for finite values, but an infinity or NaN
// times it is NaN, so what is to be multiplied by it is taken as 0 there, of the lane's pairs 2i and 2i + 1.  Forwards
// at every head; backwards only where a head's sum shows a value that is not finite.  61440 x 24 x 128 bf16 interleaved,
// 53 of 64 pairs turning: 261 us forwards (with the sine alone 249), 418 backwards (394; by selection 436).
template <bool STILL> __device__ __forceinline__ F2 turning(int turn, int l, int i, F2 v) {
    if constexpr (!STILL) return v;
    const float2 f = both(v);
    return f2(4 * l + 2 * i < turn ? f.x : 0.f, 4 * l + 2 * i + 1 < turn ? f.y : 0.f);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// A lane's channels of one head on their way through its own part of shared memory, in planes of one access a thread.
template <typename T, bool HALF> struct Copy {
    static constexpr int B = HALF ? 4 * (int)sizeof(T) : 16, P = 8 * (int)sizeof(T) / B;
    template <int D> static __device__ __forceinline__ void fetch(uint32_t s, const T* head) {
#pragma unroll
        for (int p = 0; p < P; ++p) cp_async<B>(s + p * 256 * B, head + p * (HALF ? D / 2 : 16 / (int)sizeof(T)));
    }
    static __device__ __forceinline__ void read(Raw<T, HALF>& r, const char* s) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(s + p * 256 * B);
            uint32_t* w = HALF ? r.p[p * HALF].w : r.p[0].w + 4 * p;
            if constexpr (B == 16) {
                const uint4 v = *reinterpret_cast<const uint4*>(q);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(q);
                w[0] = v.x; w[1] = v.y;
            }
        }
    }
};

// CTAs on an SM, heads of a lane at a time and steps that are copied ahead (0: a step's rows are loaded when it begins):
// what the registers allow without spills, at 24 heads of 128 channels.
// Forward (294912 tokens, passes back to back): bf16 4 x 3 1167 us, 3 x 6 1172, 3 x 4 1192, 4 x 4 1211, 5 x 3 with 24
// bytes of spills 1247, 4 x 2 1286, 3 x 3 1308; f32 (30720)
// 3 x 2 246, 3 x 3 249-263, 3 x 4 249-271.
// Backward (61440 tokens, bf16): interleaved 3 x 1, 4 ahead 364 us, 3 x 2, 2 ahead 402, without copies 401; half
// 3 x 2, 2 ahead 358, 3 x 1, 4 ahead 380.  f32 (30720): 2 x 2 without copies 355; a lane's eight floats are two
// copies that leave gaps in a warp's access: interleaved 585.
constexpr int ctas_sm(int elem, bool bwd) { return bwd ? (elem == 2 ? 3 : 2) : elem == 2 ? 4 : 3; }
constexpr int heads_at_once(int elem, bool half, bool bwd) { return bwd ? (elem == 2 && !half ? 1 : 2) : elem == 2 ? 3 : 2; }
constexpr int steps_ahead(int elem, bool half, bool bwd) { return bwd && elem == 2 ? (half ? 2 : 4) : 0; }
extern __shared__ __align__(16) char g_rows[];

template <typename T, int D, bool HALF, bool BWD, bool STILL>
__global__ void __launch_bounds__(256, ctas_sm(sizeof(T), BWD)) k_head_rotate(const Args a) {
    constexpr int LPH = D / 8, TPW = 32 / LPH;       // lanes a head, heads a warp
    constexpr int HU = heads_at_once(sizeof(T), HALF, BWD), S = steps_ahead(sizeof(T), HALF, BWD);
    using CP = Copy<T, HALF>;
    constexpr int kRow = CP::P * CP::B * 256, kStage = 2 * HU * kRow;     // of a CTA: one head a lane, x and dr of a step
    const Side& sd = a.side[blockIdx.y];
    const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
    // the same for all lanes, and so known to the compiler: its step's counters and rows need no registers of theirs
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int64_t warps = (int64_t)gridDim.x * 8, items = a.tokens * sd.parts;
    const int stride = TPW * sd.parts, c0 = lane_at<D, HALF>(l);
    const F2 zero = f2(0.f);
    Pairs w, dw;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w.a[i] = w.b[i] = f2(1.f);
        dw.a[i] = dw.b[i] = zero;
        if (sd.w) {
            w.a[i] = f2(__ldg(sd.w + channel<D, HALF>(l, 2 * i, false)), __ldg(sd.w + channel<D, HALF>(l, 2 * i + 1, false)));
            w.b[i] = f2(__ldg(sd.w + channel<D, HALF>(l, 2 * i, true)), __ldg(sd.w + channel<D, HALF>(l, 2 * i + 1, true)));
        }
    }
    // A step: HU heads of each of the warp's lane groups, of one token.
    struct Step {
        int64_t it;
        uint32_t token;
        int first, h0;
    };
    auto begin = [&](Step& s, int64_t it) {
        s.it = it;
        s.token = sd.parts == 1 ? (uint32_t)it : (uint32_t)(it / sd.parts);
        s.first = s.h0 = (int)(it - (int64_t)s.token * sd.parts) * TPW;
    };
    auto advance = [&](Step& s) {
        s.h0 += HU * stride;
        if (s.h0 >= sd.heads) begin(s, s.it + warps);
    };
    // Lanes past the last head repeat it (or, where the results take its place, them); they neither store nor add to dw.
    auto head_of = [&](const Step& s, int u) {
        const int h = s.h0 + sub + u * stride;
        return h < sd.heads ? h : sd.heads - 1;
    };
    Step now, ahead;
    auto none = [&](int u) { return u && now.h0 + u * stride >= sd.heads; };     // no lane of the warp has a u-th head
    begin(now, (int64_t)blockIdx.x * 8 + warp);
    ahead = now;
    const uint32_t ring = S ? (uint32_t)__cvta_generic_to_shared(g_rows) + threadIdx.x * CP::B : 0u;
    int stage = 0;
    auto fetch = [&](int st) {
        if (ahead.it < items) {
            const T* x = (const T*)sd.x + (int64_t)ahead.token * sd.ld_x + c0;
            const T* dr = (const T*)sd.dr + (int64_t)ahead.token * sd.ld_dr + c0;
#pragma unroll
            for (int u = 0; u < HU; ++u) {
                const int h = head_of(ahead, u) * D;
                if (a.norm) CP::template fetch<D>(ring + st * kStage + 2 * u * kRow, x + h);
                CP::template fetch<D>(ring + st * kStage + (2 * u + 1) * kRow, dr + h);
            }
            advance(ahead);
        }
        cp_commit();
    };
    if constexpr (S > 0) {
#pragma unroll
        for (int i = 0; i < S; ++i) fetch(i);
    }
    F2 cs[2], sn[2], sm[2];                      // sm = -sn
    F2 ta[2], tb[2], ua[2], ub[2];               // forward: the turn with the weights in it, a' = a ta + b tb, b' = a ua + b ub
    // every lane of the warp takes part in the exchanges of every step
    while (now.it < items) {
        Raw<T, HALF> px[HU], pr[BWD ? HU : 1];
        if constexpr (S > 0) {
            cp_wait<S - 1>();
        } else {
            const T* x = (const T*)sd.x + (int64_t)now.token * sd.ld_x + c0;
            const T* dr = (const T*)sd.dr + (int64_t)now.token * sd.ld_dr + c0;
#pragma unroll
            for (int u = 0; u < HU; ++u) {
                const int h = head_of(now, u) * D;
                if (!BWD || a.norm) load_raw<T, D, HALF>(px[u], x + h);
                if constexpr (BWD) load_raw<T, D, HALF>(pr[u], dr + h);
            }
        }
        if (now.h0 == now.first) {
            angles(a, now.token, l, cs, sn);
            sm[0] = sn[0] * f2(-1.f);
            sm[1] = sn[1] * f2(-1.f);
            if constexpr (!BWD) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ta[i] = w.a[i] * cs[i];
                    tb[i] = turning<STILL>(a.turn, l, i, w.b[i]) * sm[i];
                    ua[i] = turning<STILL>(a.turn, l, i, w.a[i]) * sn[i];
                    ub[i] = w.b[i] * cs[i];
                }
            }
        }
        T* out = (T*)sd.out + (int64_t)now.token * sd.ld_out + c0;
#pragma unroll
        for (int u = 0; u < HU; ++u) {
            // Not so around the loads, which go out together: 16 heads bf16 (61440 tokens) 181 us, with it there 185, without 188.
            if (S == 0 && none(u)) break;
            const bool in = now.h0 + sub + u * stride < sd.heads;
            Pairs v, o;
            if constexpr (!BWD) {
                v = pairs_of<T, HALF>(px[u]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    o.a[i] = fma(v.a[i], ta[i], turning<STILL>(a.turn, l, i, v.b[i]) * tb[i]);
                    o.b[i] = fma(turning<STILL>(a.turn, l, i, v.a[i]), ua[i], v.b[i] * ub[i]);
                }
                if (a.norm) {
                    const float q = lanes_sum<LPH>(sum(fma(v.a[0], v.a[0], v.a[1] * v.a[1]) +
                                                       fma(v.b[0], v.b[0], v.b[1] * v.b[1])));
                    const F2 r = f2(rsqrtf(q * (1.f / D) + a.eps));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o.a[i] = o.a[i] * r;
                        o.b[i] = o.b[i] * r;
                    }
                }
            } else {
                const char* row = g_rows + stage * kStage + 2 * u * kRow + threadIdx.x * CP::B;
                if constexpr (S > 0) CP::read(pr[u], row + kRow);
                const Pairs d = pairs_of<T, HALF>(pr[u]);
                auto turn = [&](auto still) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o.a[i] = fma(d.a[i], cs[i], turning<still.value>(a.turn, l, i, d.b[i]) * sn[i]);
                        o.b[i] = fma(d.b[i], cs[i], turning<still.value>(a.turn, l, i, d.a[i]) * sm[i]);
                    }
                };
                turn(std::false_type());
                if constexpr (STILL)
                    if (!finite(sum((o.a[0] + o.a[1]) + (o.b[0] + o.b[1])))) turn(std::true_type());
                if (a.norm) {
                    if constexpr (S > 0) CP::read(px[u], row);
                    v = pairs_of<T, HALF>(px[u]);
                    // x once against itself, once against dn ∘ w; dx = r (dn ∘ w - x r (r mean(dn ∘ w ∘ x))): r may be as
                    // large as eps^-1/2, and meets what makes it small again before its next power
                    Pairs t;
                    F2 q2 = v.a[0] * v.a[0], m2;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        t.a[i] = o.a[i] * v.a[i];
                        t.b[i] = o.b[i] * v.b[i];
                        if (i) q2 = fma(v.a[i], v.a[i], q2);
                        q2 = fma(v.b[i], v.b[i], q2);
                        m2 = i ? fma(t.a[i], w.a[i], m2) : t.a[i] * w.a[i];
                        m2 = fma(t.b[i], w.b[i], m2);
                    }
                    float q = sum(q2), m = sum(m2);
                    lanes_sum<LPH>(q, m, l);
                    const float r = rsqrtf(q * (1.f / D) + a.eps);
                    const F2 r2 = f2(r), k = f2(-(r * m * (1.f / D)) * r);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (in) {
                            dw.a[i] = fma(t.a[i], r2, dw.a[i]);
                            dw.b[i] = fma(t.b[i], r2, dw.b[i]);
                        }
                        o.a[i] = fma(v.a[i], k, o.a[i] * w.a[i]) * r2;
                        o.b[i] = fma(v.b[i], k, o.b[i] * w.b[i]) * r2;
                    }
                }
            }
            if (in) store_pairs<T, D, HALF>(out + (now.h0 + sub + u * stride) * D, o);
        }
        advance(now);
        if constexpr (S > 0) {                // the step's own rows have been used: their place is free
            fetch(stage);
            stage = stage + 1 == S ? 0 : stage + 1;
        }
    }
    if constexpr (S > 0) cp_wait<0>();
    if constexpr (BWD) {
        let_next_start();
        if (!a.part) return;
        __shared__ float sh[256 / LPH][D];
        const int team = threadIdx.x / LPH;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 f = both(dw.a[i]);
            sh[team][channel<D, HALF>(l, 2 * i, false)] = f.x;
            sh[team][channel<D, HALF>(l, 2 * i + 1, false)] = f.y;
            f = both(dw.b[i]);
            sh[team][channel<D, HALF>(l, 2 * i, true)] = f.x;
            sh[team][channel<D, HALF>(l, 2 * i + 1, true)] = f.y;
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int i = 0; i < 256 / LPH; ++i) s += sh[i][threadIdx.x];
            a.part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
        }
    }
}

// dw of one side a CTA column: 32 channels, 16 rows of threads over the CTAs' sums, in a fixed order
__global__ void __launch_bounds__(512) k_head_rotate_join(const float* part, int n, int D, float* dwq, float* dwk) {
    __shared__ float sh[16][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float* dw = blockIdx.y ? dwk : dwq;
    wait_for_previous();
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += 16) s += part[((int64_t)blockIdx.y * n + i) * D + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && dw) {
        for (int y = 1; y < 16; ++y) s += sh[y][threadIdx.x];
        dw[c] = s;
    }
}

constexpr int kMaxCtas = kSMs * 4;     // as many as run at a time

static prism_status_t check(const prism_rotate_t* p) {
    if (!p) return PRISM_ERR_INVALID_ARG;
    if (p->tokens < 0 || p->T < 1 || p->H < 1 || p->W < 1) return PRISM_ERR_SHAPE;
    // one factor at a time: the product of three may pass 64 bits
    if (p->tokens > INT32_MAX || (int64_t)p->T * p->H > INT32_MAX || (int64_t)p->T * p->H * p->W > INT32_MAX ||
        (int64_t)p->T * p->pairs_t + (int64_t)p->H * p->pairs_h + (int64_t)p->W * p->pairs_w > INT32_MAX)
        return PRISM_ERR_UNSUPPORTED;
    if (p->dtype != PRISM_F32 && p->dtype != PRISM_BF16) return PRISM_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 128) return PRISM_ERR_UNSUPPORTED;
    if (p->heads_q < 0 || p->heads_q > 1024 || p->heads_k < 0 || p->heads_k > 1024) return PRISM_ERR_UNSUPPORTED;
    if (p->pairs_t < 0 || p->pairs_h < 0 || p->pairs_w < 0 || p->pairs_t > 64 || p->pairs_h > 64 || p->pairs_w > 64 ||
        p->pairs_t + p->pairs_h + p->pairs_w > p->head_dim / 2)
        return PRISM_ERR_SHAPE;
    if (p->pairing != PRISM_PAIRS_INTERLEAVED && p->pairing != PRISM_PAIRS_HALF) return PRISM_ERR_INVALID_ARG;
    if (p->norm != 0 && p->norm != 1) return PRISM_ERR_INVALID_ARG;
    if (!(p->eps > 0.f) || !isfinite(p->eps)) return PRISM_ERR_INVALID_ARG;
    return PRISM_OK;
}

// token stride in elements (0: dense): no overlap, and every row on a 16-byte boundary
static bool ld_of(int64_t ld, const prism_rotate_t* p, int heads, int64_t* out) {
    *out = ld == 0 ? (int64_t)heads * p->head_dim : ld;
    return *out >= (int64_t)heads * p->head_dim && *out % (p->dtype == PRISM_BF16 ? 8 : 4) == 0;
}

// warps that share a token: more than one only where the tokens alone would leave SMs without work
static int parts_of(int64_t tokens, int heads, int d) {
    const int per_warp = 256 / d, most = (heads + per_warp - 1) / per_warp;
    int64_t want = (int64_t)kSMs * 16 / (tokens > 0 ? tokens : 1);
    if (want > most) want = most;
    return want < 1 ? 1 : (int)want;
}

static unsigned ctas_of(const Args& a, int sides, int per_sm) {
    int64_t items = 0;
    for (int i = 0; i < sides; ++i) {
        const int64_t n = a.tokens * a.side[i].parts;
        if (n > items) items = n;
    }
    const int64_t want = (items + 7) / 8, most = (int64_t)kSMs * per_sm / sides;
    return (unsigned)(want < most ? want : most);
}

template <typename T, int D, bool HALF, bool BWD> static void launch_one(const Args& a, dim3 grid, cudaStream_t s) {
    auto kernel = a.turn < D / 2 ? &k_head_rotate<T, D, HALF, BWD, true> : &k_head_rotate<T, D, HALF, BWD, false>;
    constexpr int bytes = steps_ahead(sizeof(T), HALF, BWD) * 2 * heads_at_once(sizeof(T), HALF, BWD) * 8 * (int)sizeof(T) * 256;
    static_assert(bytes <= 36 << 10, "with the static part, within the 48 KB that need no leave");
    kernel<<<grid, 256, bytes, s>>>(a);
}
template <bool BWD> static void launch(const prism_rotate_t* p, const Args& a, dim3 grid, cudaStream_t s) {
#define PRISM_ROT_D(T)                                                                                                 \
    do {                                                                                                               \
        if (p->head_dim == 128)                                                                                        \
            return p->pairing == PRISM_PAIRS_HALF ? launch_one<T, 128, true, BWD>(a, grid, s)                          \
                                                  : launch_one<T, 128, false, BWD>(a, grid, s);                        \
        return p->pairing == PRISM_PAIRS_HALF ? launch_one<T, 64, true, BWD>(a, grid, s)                               \
                                              : launch_one<T, 64, false, BWD>(a, grid, s);                             \
    } while (0)
    if (p->dtype == PRISM_BF16) PRISM_ROT_D(__nv_bfloat16);
    PRISM_ROT_D(float);
#undef PRISM_ROT_D
}

}  // namespace rot
}  // namespace prism

using namespace prism;
using namespace prism::rot;

extern "C" prism_status_t prism_head_rotate_ws_bytes(const prism_rotate_t* p, size_t* bytes) {
    const prism_status_t st = check(p);
    if (st != PRISM_OK) return st;
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    *bytes = (size_t)kMaxCtas * p->head_dim * sizeof(float);
    return PRISM_OK;
}

static prism_status_t rotate(const prism_rotate_t* p, const void* Q, const void* K, const float* wq, const float* wk,
                             const float* table, const void* dQr, const void* dKr, void* oQ, void* oK, float* dwq,
                             float* dwk, void* ws, size_t ws_bytes, bool bwd, cudaStream_t stream) {
    const prism_status_t st = check(p);
    if (st != PRISM_OK) return st;
    const bool hq = p->heads_q > 0, hk = p->heads_k > 0;
    if (!hq && !hk) return PRISM_ERR_SHAPE;
    if (!p->norm && (wq || wk || dwq || dwk)) return PRISM_ERR_INVALID_ARG;
    if ((!hq && (Q || oQ || wq || dQr || dwq)) || (!hk && (K || oK || wk || dKr || dwk))) return PRISM_ERR_INVALID_ARG;
    if (!ok_opt(wq) || !ok_opt(wk) || !ok_opt(dwq) || !ok_opt(dwk) || !ok_opt(ws)) return PRISM_ERR_INVALID_ARG;
    const bool any_pair = p->pairs_t + p->pairs_h + p->pairs_w > 0;
    if (any_pair ? !ok_ptr(table) : !ok_opt(table)) return PRISM_ERR_INVALID_ARG;
    Args a{};
    int sides = 0;
    for (int i = 0; i < 2; ++i) {
        if (i ? !hk : !hq) continue;
        Side& s = a.side[sides++];
        s.heads = i ? p->heads_k : p->heads_q;
        s.x = i ? K : Q; s.dr = i ? dKr : dQr; s.w = i ? wk : wq; s.out = i ? oK : oQ;
        if (!ld_of(i ? p->ld_k : p->ld_q, p, s.heads, &s.ld_x) || !ld_of(i ? p->ld_ko : p->ld_qo, p, s.heads, &s.ld_out) ||
            !ld_of(i ? p->ld_dk : p->ld_dq, p, s.heads, &s.ld_dr))
            return PRISM_ERR_SHAPE;
        s.parts = parts_of(p->tokens, s.heads, p->head_dim);
        if (p->tokens && ((bwd && !p->norm ? !ok_opt(s.x) : !ok_ptr(s.x)) || !ok_ptr(s.out) || (bwd && !ok_ptr(s.dr))))
            return PRISM_ERR_INVALID_ARG;
    }
    if (p->tokens == 0) {
        for (float* w : {dwq, dwk})
            if (w && !taken(cudaMemsetAsync(w, 0, p->head_dim * sizeof(float), stream))) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    a.table = (const float2*)table;
    a.tokens = p->tokens;
    a.T = p->T; a.H = p->H; a.W = p->W;
    a.nT = p->pairs_t; a.nH = p->pairs_h; a.nW = p->pairs_w; a.turn = a.nT + a.nH + a.nW;
    a.norm = p->norm; a.eps = p->eps;
    const unsigned ctas = ctas_of(a, sides, ctas_sm(p->dtype == PRISM_BF16 ? 2 : 4, bwd));
    const dim3 grid(ctas, sides);
    if (!bwd) {
        launch<false>(p, a, grid, stream);
        return launch_status(1);
    }
    const bool dw = dwq || dwk;
    if (dw) {
        if (!ws || ws_bytes < (size_t)kMaxCtas * p->head_dim * sizeof(float)) return PRISM_ERR_WORKSPACE;
        a.part = (float*)ws;
    }
    launch<true>(p, a, grid, stream);
    if (dw) {
        if (!launched() ||
            !launch_after(k_head_rotate_join, dim3(p->head_dim / 32, sides), dim3(32, 16), 1, stream, (const float*)a.part,
                          (int)ctas, (int)p->head_dim, hq ? dwq : dwk, hq ? dwk : (float*)nullptr))
            return PRISM_ERR_CUDA;
    }
    return launch_status(dw ? 2 : 1);
}

extern "C" prism_status_t prism_head_rotate_fwd(const prism_rotate_t* p, const void* Q, const void* K, const float* wq,
                                                const float* wk, const float* table, void* Qr, void* Kr,
                                                cudaStream_t stream) {
    return rotate(p, Q, K, wq, wk, table, nullptr, nullptr, Qr, Kr, nullptr, nullptr, nullptr, 0, false, stream);
}

extern "C" prism_status_t prism_head_rotate_bwd(const prism_rotate_t* p, const void* Q, const void* K, const float* wq,
                                                const float* wk, const float* table, const void* dQr, const void* dKr,
                                                void* dQ, void* dK, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                                cudaStream_t stream) {
    return rotate(p, Q, K, wq, wk, table, dQr, dKr, dQ, dK, dwq, dwk, ws, ws_bytes, true, stream);
}
