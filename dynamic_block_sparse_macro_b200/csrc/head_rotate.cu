// The norm of each head's channels and the rotation by the token's place in
// the grid, for Q and K before the attention.
//
//   n = N_rms(x) ∘ w over the head's d channels (or n = x)
//   (n_a, n_b) -> (n_a cos - n_b sin, n_a sin + n_b cos) for each pair (a, b)
//
// and backwards, with dn the pairs of dr turned back (by -angle), c = dn ∘ w, n = x r:
//   dx = r (c - n mean(c ∘ n)),  dw = sum over tokens and heads of dn ∘ n.
//
// Bound by HBM: each element is read and written once.  d/8 lanes hold a head's row, eight channels
// each, and walk the heads of one token, so that the token's place, its cosines and its sines (a
// table of one row an axis position, which stays in L1) are fetched once for all its heads.  All
// arithmetic is fp32; the result is rounded once.
#include <initializer_list>

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
    int T, H, W, nT, nH, nW, norm;
    float eps;
};

template <int LPH> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// cosine and sine of the lane's pairs for one token
template <int D, bool HALF>
__device__ __forceinline__ void angles(const Args& a, int64_t token, int l, float* cs, float* sn) {
    const uint32_t hw = (uint32_t)a.H * a.W;
    const uint32_t at = (uint32_t)(token % ((int64_t)a.T * hw));
    const uint32_t pt = at / hw, r = at - pt * hw, ph = r / a.W, pw = r - ph * a.W;
    constexpr int NP = HALF ? 8 : 4;
    const int p0 = HALF ? (l % (D / 16)) * 8 : l * 4;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int p = p0 + j, q = p - a.nT, s = q - a.nH;
        float2 v = make_float2(1.f, 0.f);
        if (p < a.nT) v = __ldg(a.table + pt * a.nT + p);
        else if (q < a.nH) v = __ldg(a.table + a.T * a.nT + ph * a.nH + q);
        else if (s < a.nW) v = __ldg(a.table + a.T * a.nT + a.H * a.nH + pw * a.nW + s);
        cs[j] = v.x;
        sn[j] = v.y;
    }
}

// turns the lane's eight channels by the angle (dir = 1) or back (dir = -1)
template <int D, bool HALF>
__device__ __forceinline__ void turn(float (&v)[8], const float* cs, const float* sn, int l, float dir) {
    if constexpr (HALF) {
        // the pair's other half lies d/16 lanes away: the first half gets a cos - b sin, the second b cos + a sin
        const float s = l < D / 16 ? -dir : dir;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float o = __shfl_xor_sync(0xffffffffu, v[j], D / 16);
            v[j] = fmaf(v[j], cs[j], s * sn[j] * o);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = v[2 * j], q = v[2 * j + 1], s = dir * sn[j];
            v[2 * j] = fmaf(p, cs[j], -s * q);
            v[2 * j + 1] = fmaf(p, s, q * cs[j]);
        }
    }
}

template <typename T, int D, bool HALF, bool BWD>
__global__ void __launch_bounds__(256) k_head_rotate(const Args a) {
    constexpr int LPH = D / 8, TPW = 32 / LPH;       // lanes a head, heads a warp
    constexpr int HU = BWD ? 2 : 4;                  // heads of a lane in flight
    const Side& sd = a.side[blockIdx.y];
    const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
    const int64_t warps = (int64_t)gridDim.x * 8, items = a.tokens * sd.parts;
    const int stride = TPW * sd.parts;
    float w[8], dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) { w[j] = 1.f; dw[j] = 0.f; }
    if (sd.w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __ldg(sd.w + l * 8 + j);
    }
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += warps) {
        const int64_t token = it / sd.parts;
        const int first = (int)(it - token * sd.parts) * TPW + sub;
        const T* x = (const T*)sd.x + token * sd.ld_x + l * 8;
        const T* dr = BWD ? (const T*)sd.dr + token * sd.ld_dr + l * 8 : nullptr;
        T* out = (T*)sd.out + token * sd.ld_out + l * 8;
        float cs[8], sn[8];
        angles<D, HALF>(a, token, l, cs, sn);
        // every lane of the warp takes part in the shuffles of every step: first - sub is the warp's
        for (int h0 = first - sub; h0 < sd.heads; h0 += HU * stride) {
            Pack<T, 8> px[HU], pr[BWD ? HU : 1];
#pragma unroll
            for (int u = 0; u < HU; ++u) {
                const int h = h0 + sub + u * stride;
                if (h < sd.heads) {
                    if (!BWD || a.norm) load(px[u], x + h * D);
                    if constexpr (BWD) load(pr[u], dr + h * D);
                }
            }
#pragma unroll
            for (int u = 0; u < HU; ++u) {
                const int h = h0 + sub + u * stride;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.f;
                if (h < sd.heads && (!BWD || a.norm)) unpack<8>(px[u], v);
                float r = 1.f;
                if (a.norm) {
                    float q = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
                    r = rsqrtf(lanes_sum<LPH>(q) * (1.f / D) + a.eps);
                }
                if constexpr (!BWD) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= r * w[j];
                    turn<D, HALF>(v, cs, sn, l, 1.f);
                } else {
                    float d[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = 0.f;
                    if (h < sd.heads) unpack<8>(pr[u], d);
                    turn<D, HALF>(d, cs, sn, l, -1.f);
                    if (a.norm) {
                        float m = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            v[j] *= r;
                            dw[j] = fmaf(d[j], v[j], dw[j]);
                            d[j] *= w[j];
                            m = fmaf(d[j], v[j], m);
                        }
                        m = lanes_sum<LPH>(m) * (1.f / D);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = r * fmaf(-v[j], m, d[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = d[j];
                    }
                }
                if (h < sd.heads) {
                    Pack<T, 8> o;
                    pack<8>(o, v);
                    store(out + h * D, o);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        __shared__ float sh[256 / LPH][D];
        const int team = threadIdx.x / LPH;
#pragma unroll
        for (int j = 0; j < 8; ++j) sh[team][l * 8 + j] = dw[j];
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

constexpr int kMaxCtas = kSMs * 6;

static prism_status_t check(const prism_rotate_t* p) {
    if (!p) return PRISM_ERR_INVALID_ARG;
    if (p->tokens < 0 || p->T < 1 || p->H < 1 || p->W < 1) return PRISM_ERR_SHAPE;
    if (p->tokens > (int64_t(1) << 40) || (int64_t)p->T * p->H * p->W > INT32_MAX ||
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

static unsigned ctas_of(const Args& a, int sides) {
    int64_t items = 0;
    for (int i = 0; i < sides; ++i) {
        const int64_t n = a.tokens * a.side[i].parts;
        if (n > items) items = n;
    }
    const int64_t want = (items + 7) / 8, most = kMaxCtas / sides;
    return (unsigned)(want < most ? want : most);
}

template <bool BWD> static void launch(const prism_rotate_t* p, const Args& a, dim3 grid, cudaStream_t s) {
#define PRISM_ROT(T, D, HALF) k_head_rotate<T, D, HALF, BWD><<<grid, 256, 0, s>>>(a)
#define PRISM_ROT_D(T)                                                                              \
    do {                                                                                            \
        if (p->head_dim == 128) { if (p->pairing == PRISM_PAIRS_HALF) PRISM_ROT(T, 128, true); else PRISM_ROT(T, 128, false); } \
        else { if (p->pairing == PRISM_PAIRS_HALF) PRISM_ROT(T, 64, true); else PRISM_ROT(T, 64, false); } \
    } while (0)
    if (p->dtype == PRISM_BF16) PRISM_ROT_D(__nv_bfloat16);
    else PRISM_ROT_D(float);
#undef PRISM_ROT_D
#undef PRISM_ROT
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
            if (w && cudaMemsetAsync(w, 0, p->head_dim * sizeof(float), stream) != cudaSuccess) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    a.table = (const float2*)table;
    a.tokens = p->tokens;
    a.T = p->T; a.H = p->H; a.W = p->W;
    a.nT = p->pairs_t; a.nH = p->pairs_h; a.nW = p->pairs_w;
    a.norm = p->norm; a.eps = p->eps;
    const unsigned ctas = ctas_of(a, sides);
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
    if (dw)
        k_head_rotate_join<<<dim3(p->head_dim / 32, sides), dim3(32, 16), 0, stream>>>(
            a.part, (int)ctas, p->head_dim, hq ? dwq : dwk, hq ? dwk : nullptr);
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
