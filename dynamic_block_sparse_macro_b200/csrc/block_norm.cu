// Block norms: argument checks, the split of the rows into segments and the
// sums of the segments' column sums (formulas in block_norm.cuh).
#include <initializer_list>

#include "block_norm.cuh"

namespace prism {
namespace bn {

constexpr int kMaxJoin = 64;

template <> prism_status_t launch_fwd<float, float>(const FwdArgs&, int, cudaStream_t);
template <> prism_status_t launch_fwd<float, __nv_bfloat16>(const FwdArgs&, int, cudaStream_t);
template <> prism_status_t launch_fwd<__nv_bfloat16, __nv_bfloat16>(const FwdArgs&, int, cudaStream_t);
template <> prism_status_t launch_bwd<float, float>(const BwdArgs&, int, cudaStream_t);
template <> prism_status_t launch_bwd<float, __nv_bfloat16>(const BwdArgs&, int, cudaStream_t);
template <> prism_status_t launch_bwd<__nv_bfloat16, __nv_bfloat16>(const BwdArgs&, int, cudaStream_t);

struct JoinArgs {
    const float* part;                  // [segments][3][C]
    const float *w, *b, *w_post, *scale, *gate;
    float *dgate, *dscale, *dshift;     // [groups][C]
    float *dw, *db, *dw_post;           // [C]
    float* part2;                       // [gridDim.y][3][C] where gridDim.y > 1
    int64_t groups, segs, ld_scale, ld_gate;
    int C, per_group;
};

// 32 channels a CTA, 16 rows of threads that take every 16th segment; their sums meet in a fixed
// order, so the result does not depend on scheduling.
__device__ __forceinline__ void join_rows(float (&v)[3], float (*sh)[3][32]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) sh[threadIdx.y][i][threadIdx.x] = v[i];
    __syncthreads();
    if (threadIdx.y == 0) {
#pragma unroll
        for (int y = 1; y < 16; ++y)
#pragma unroll
            for (int i = 0; i < 3; ++i) v[i] += sh[y][i][threadIdx.x];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(512) k_block_norm_groups(const JoinArgs a) {
    __shared__ float sh[16][3][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    for (int64_t g = blockIdx.y; g < a.groups; g += gridDim.y) {
        float v[3] = {0.f, 0.f, 0.f};
        if (c < a.C) {
#pragma unroll 4
            for (int s = threadIdx.y; s < a.per_group; s += 16) {
                const float* p = a.part + (g * a.per_group + s) * 3 * a.C + c;
                if (a.dscale) v[0] += p[0];
                if (a.dscale || a.dshift) v[1] += p[a.C];
                if (a.dgate) v[2] += p[2 * a.C];
            }
        }
        join_rows(v, sh);
        if (threadIdx.y == 0 && c < a.C) {
            if (a.dscale) a.dscale[g * a.C + c] = fmaf(a.w ? a.w[c] : 1.f, v[0], a.b ? a.b[c] * v[1] : 0.f);
            if (a.dshift) a.dshift[g * a.C + c] = v[1];
            if (a.dgate) a.dgate[g * a.C + c] = a.w_post ? a.w_post[c] * v[2] : v[2];
        }
    }
}

__global__ void __launch_bounds__(512) k_block_norm_affine(const JoinArgs a) {
    __shared__ float sh[16][3][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const int64_t p0 = a.segs * blockIdx.y / gridDim.y, p1 = a.segs * (blockIdx.y + 1) / gridDim.y;
    float v[3] = {0.f, 0.f, 0.f};
    if (c < a.C) {
#pragma unroll 4
        for (int64_t s = p0 + threadIdx.y; s < p1; s += 16) {
            const float* p = a.part + s * 3 * a.C + c;
            const int64_t g = s / a.per_group;
            const float one = a.scale ? 1.f + a.scale[g * a.ld_scale + c] : 1.f;
            if (a.dw) v[0] = fmaf(one, p[0], v[0]);
            if (a.db) v[1] = fmaf(one, p[a.C], v[1]);
            if (a.dw_post) v[2] = fmaf(a.gate ? a.gate[g * a.ld_gate + c] : 1.f, p[2 * a.C], v[2]);
        }
    }
    join_rows(v, sh);
    if (threadIdx.y != 0 || c >= a.C) return;
    if (gridDim.y > 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) a.part2[((int64_t)blockIdx.y * 3 + i) * a.C + c] = v[i];
        return;
    }
    if (a.dw) a.dw[c] = v[0];
    if (a.db) a.db[c] = v[1];
    if (a.dw_post) a.dw_post[c] = v[2];
}

__global__ void __launch_bounds__(512) k_block_norm_affine_join(const JoinArgs a, int n) {
    __shared__ float sh[16][3][32];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v[3] = {0.f, 0.f, 0.f};
    if (c < a.C) {
        for (int s = threadIdx.y; s < n; s += 16)
#pragma unroll
            for (int i = 0; i < 3; ++i) v[i] += a.part2[((int64_t)s * 3 + i) * a.C + c];
    }
    join_rows(v, sh);
    if (threadIdx.y != 0 || c >= a.C) return;
    if (a.dw) a.dw[c] = v[0];
    if (a.db) a.db[c] = v[1];
    if (a.dw_post) a.dw_post[c] = v[2];
}

struct Split {
    int64_t groups, per_group, segs;
};

// Segments of rows, none across a group's end.  Where there are few groups, each is cut so that the
// segments fill the teams that run at a time once; where groups are many, into about eight rounds of
// such teams, so that the last round's idle part is small.  No segment below four rows is cut:
// its column sums cost as much as three rows.
static Split split_rows(const prism_block_norm_t* n) {
    Split s{0, 1, 0};
    if (n->rows == 0) return s;
    const int64_t rpg = n->rows_per_group < n->rows ? n->rows_per_group : n->rows;
    s.groups = (n->rows + rpg - 1) / rpg;
    const int64_t teams = (int64_t)kSMs * sm_teams(n->channels, bwd_ctas(team_bucket(team_threads(n->channels))));
    int64_t per = s.groups * 4 <= teams ? teams / s.groups : 8 * teams / s.groups;
    const int64_t most = (rpg + 3) / 4;
    if (per > most) per = most;
    if (per < 1) per = 1;
    s.per_group = per;
    s.segs = s.groups * s.per_group;
    return s;
}

static prism_status_t check(const prism_block_norm_t* n) {
    if (!n) return PRISM_ERR_INVALID_ARG;
    if (n->rows < 0 || n->rows_per_group < 1 || n->channels < 1) return PRISM_ERR_SHAPE;
    if (n->channels > kMaxChannels || n->rows > (int64_t(1) << 40)) return PRISM_ERR_UNSUPPORTED;
    const bool xf = n->stream_dtype == PRISM_F32, xb = n->stream_dtype == PRISM_BF16;
    const bool hf = n->branch_dtype == PRISM_F32, hb = n->branch_dtype == PRISM_BF16;
    if (!(xf && (hf || hb)) && !(xb && hb)) return PRISM_ERR_UNSUPPORTED;
    for (int k : {n->norm, n->post_norm})
        if (k != PRISM_NORM_NONE && k != PRISM_NORM_RMS && k != PRISM_NORM_LAYER) return PRISM_ERR_INVALID_ARG;
    if (!(n->eps > 0.f) || !isfinite(n->eps) || !isfinite(n->res_scale)) return PRISM_ERR_INVALID_ARG;
    return PRISM_OK;
}

// the row stride in elements (0: dense); false when rows would overlap
static bool ld_of(int64_t ld, int C, int64_t* out) {
    *out = ld == 0 ? C : ld;
    return *out >= C;
}

// channels an access may take: all strides in use and the width are multiples of it, and all addresses of its bytes
static int unit_of(int C, std::initializer_list<int64_t> lds, std::initializer_list<const void*> ptrs) {
    Bits n, p;
    n.bytes(C);
    for (int64_t l : lds) n.bytes(l);
    for (const void* q : ptrs) p << q;
    return n.multiple_of(8) && p.multiple_of(16) ? 8 : n.multiple_of(2) && p.multiple_of(8) ? 2 : 1;
}
static int esize(int dtype) { return dtype == PRISM_BF16 ? 2 : 4; }

}  // namespace bn
}  // namespace prism

using namespace prism;
using namespace prism::bn;

extern "C" prism_status_t prism_block_norm_ws_bytes(const prism_block_norm_t* n, size_t* bytes) {
    const prism_status_t st = check(n);
    if (st != PRISM_OK) return st;
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    *bytes = (size_t)(split_rows(n).segs + kMaxJoin) * 3 * n->channels * sizeof(float);
    return PRISM_OK;
}

extern "C" prism_status_t prism_block_norm_fwd(const prism_block_norm_t* n, const void* x, const void* h,
                                               const float* gate, const float* w_post, const float* w, const float* b,
                                               const float* scale, const float* shift, void* z, void* y,
                                               cudaStream_t stream) {
    prism_status_t st = check(n);
    if (st != PRISM_OK) return st;
    FwdArgs a{};
    const int C = n->channels;
    if (!ld_of(n->ld_x, C, &a.ld_x) || !ld_of(n->ld_h, C, &a.ld_h) || !ld_of(n->ld_z, C, &a.ld_z) ||
        !ld_of(n->ld_y, C, &a.ld_y) || !ld_of(n->ld_gate, C, &a.ld_gate) || !ld_of(n->ld_scale, C, &a.ld_scale) ||
        !ld_of(n->ld_shift, C, &a.ld_shift))
        return PRISM_ERR_SHAPE;
    const bool has_y = n->norm != PRISM_NORM_NONE;
    if (!h && (z || gate || w_post || n->post_norm != PRISM_NORM_NONE || !has_y)) return PRISM_ERR_INVALID_ARG;
    if (!has_y && (y || w || b || scale || shift)) return PRISM_ERR_INVALID_ARG;
    if (w_post && n->post_norm == PRISM_NORM_NONE) return PRISM_ERR_INVALID_ARG;
    if (n->rows == 0) return PRISM_OK;
    const int es = esize(n->stream_dtype), eb = esize(n->branch_dtype);
    if (!on(x, es) || !opt_on(h, eb) || (h && !on(z, es)) || (has_y && !on(y, eb)) || !opt_on(gate, 4) ||
        !opt_on(w_post, 4) || !opt_on(w, 4) || !opt_on(b, 4) || !opt_on(scale, 4) || !opt_on(shift, 4))
        return PRISM_ERR_INVALID_ARG;
    a.x = x; a.h = h; a.gate = gate; a.w_post = w_post; a.w = w; a.b = b; a.scale = scale; a.shift = shift;
    a.z = z; a.y = y;
    a.R = n->rows;
    a.rpg = n->rows_per_group < n->rows ? n->rows_per_group : n->rows;
    a.C = C; a.norm = n->norm; a.post = n->post_norm; a.eps = n->eps; a.res = n->res_scale;
    const int unit = unit_of(C, {a.ld_x, h ? a.ld_h : 0, h ? a.ld_z : 0, has_y ? a.ld_y : 0, gate ? a.ld_gate : 0,
                                 scale ? a.ld_scale : 0, shift ? a.ld_shift : 0},
                             {x, h, gate, w_post, w, b, scale, shift, z, y});
    if (n->stream_dtype == PRISM_BF16) st = launch_fwd<__nv_bfloat16, __nv_bfloat16>(a, unit, stream);
    else if (n->branch_dtype == PRISM_BF16) st = launch_fwd<float, __nv_bfloat16>(a, unit, stream);
    else st = launch_fwd<float, float>(a, unit, stream);
    return st == PRISM_OK ? launch_status(1) : st;
}

extern "C" prism_status_t prism_block_norm_bwd(const prism_block_norm_t* n, const void* z, const void* h,
                                               const float* gate, const float* w_post, const float* w, const float* b,
                                               const float* scale, const void* dz, const void* dy, void* dx, void* dh,
                                               float* dgate, float* dw_post, float* dw, float* db, float* dscale,
                                               float* dshift, void* ws, size_t ws_bytes, cudaStream_t stream) {
    prism_status_t st = check(n);
    if (st != PRISM_OK) return st;
    BwdArgs a{};
    const int C = n->channels;
    if (!ld_of(n->ld_z, C, &a.ld_z) || !ld_of(n->ld_h, C, &a.ld_h) || !ld_of(n->ld_dz, C, &a.ld_dz) ||
        !ld_of(n->ld_dy, C, &a.ld_dy) || !ld_of(n->ld_dx, C, &a.ld_dx) || !ld_of(n->ld_dh, C, &a.ld_dh) ||
        !ld_of(n->ld_gate, C, &a.ld_gate) || !ld_of(n->ld_scale, C, &a.ld_scale))
        return PRISM_ERR_SHAPE;
    const bool has_y = n->norm != PRISM_NORM_NONE;
    if (!h && (dh || gate || w_post || dgate || dw_post || n->post_norm != PRISM_NORM_NONE || !has_y))
        return PRISM_ERR_INVALID_ARG;
    if (!has_y && (!dz || dy || w || b || scale || dw || db || dscale || dshift)) return PRISM_ERR_INVALID_ARG;
    if (n->post_norm == PRISM_NORM_NONE && (w_post || dw_post)) return PRISM_ERR_INVALID_ARG;
    if ((dgate && !gate) || (dw_post && !w_post) || (dw && !w) || (db && !b) || (dscale && !scale))
        return PRISM_ERR_INVALID_ARG;
    for (const void* p : {(const void*)gate, (const void*)w_post, (const void*)w, (const void*)b, (const void*)scale,
                          (const void*)dgate, (const void*)dw_post, (const void*)dw, (const void*)db,
                          (const void*)dscale, (const void*)dshift})
        if (!opt_on(p, 4)) return PRISM_ERR_INVALID_ARG;
    if (!ok_opt(ws)) return PRISM_ERR_INVALID_ARG;
    if (n->rows == 0) {
        // sums over no rows; there are no groups
        for (float* p : {dw_post, dw, db})
            if (p && cudaMemsetAsync(p, 0, C * sizeof(float), stream) != cudaSuccess) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    const int es = esize(n->stream_dtype), eb = esize(n->branch_dtype);
    if (!opt_on(dz, es) || (has_y && (!on(z, es) || !on(dy, eb))) || !on(dx, es) || (h && (!on(h, eb) || !on(dh, eb))))
        return PRISM_ERR_INVALID_ARG;
    const Split s = split_rows(n);
    const bool groups = dgate || dscale || dshift, affine = dw || db || dw_post, direct = s.per_group == 1;
    const bool part = affine || (groups && !direct);
    if (part && (!ws || ws_bytes < (size_t)(s.segs + kMaxJoin) * 3 * C * sizeof(float))) return PRISM_ERR_WORKSPACE;
    if (s.segs > INT32_MAX) return PRISM_ERR_UNSUPPORTED;
    a.z = z; a.h = h; a.dz = dz; a.dy = dy;
    a.gate = gate; a.w_post = w_post; a.w = w; a.b = b; a.scale = scale;
    a.dx = dx; a.dh = dh;
    a.part = part ? (float*)ws : nullptr;
    if (direct) { a.dgate = dgate; a.dscale = dscale; a.dshift = dshift; }
    a.R = n->rows;
    a.rpg = n->rows_per_group < n->rows ? n->rows_per_group : n->rows;
    a.segs = s.segs; a.per_group = (int)s.per_group;
    a.C = C; a.norm = n->norm; a.post = n->post_norm; a.eps = n->eps; a.res = n->res_scale;
    const int unit = unit_of(C, {has_y ? a.ld_z : 0, h ? a.ld_h : 0, dz ? a.ld_dz : 0, has_y ? a.ld_dy : 0, a.ld_dx,
                                 h ? a.ld_dh : 0, gate ? a.ld_gate : 0, scale ? a.ld_scale : 0},
                             {has_y ? z : nullptr, h, gate, w_post, w, b, scale, dz, dy, dx, dh, dgate, dscale, dshift,
                              part ? ws : nullptr});
    if (n->stream_dtype == PRISM_BF16) st = launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, unit, stream);
    else if (n->branch_dtype == PRISM_BF16) st = launch_bwd<float, __nv_bfloat16>(a, unit, stream);
    else st = launch_bwd<float, float>(a, unit, stream);
    if (st != PRISM_OK) return st;
    int launches = 1;
    JoinArgs j{(const float*)ws, w, b, w_post, scale, gate, dgate, dscale, dshift, dw, db, dw_post,
               (float*)ws + s.segs * 3 * C, s.groups, s.segs, a.ld_scale, a.ld_gate, C, (int)s.per_group};
    const unsigned gx = (unsigned)((C + 31) / 32);
    if (groups && !direct) {
        k_block_norm_groups<<<dim3(gx, (unsigned)(s.groups < 65535 ? s.groups : 65535)), dim3(32, 16), 0, stream>>>(j);
        ++launches;
    }
    if (affine) {
        int64_t n2 = s.segs / 64;
        n2 = n2 < 1 ? 1 : n2 > kMaxJoin ? kMaxJoin : n2;
        k_block_norm_affine<<<dim3(gx, (unsigned)n2), dim3(32, 16), 0, stream>>>(j);
        if (n2 > 1) k_block_norm_affine_join<<<gx, dim3(32, 16), 0, stream>>>(j, (int)n2);
        launches += n2 > 1 ? 2 : 1;
    }
    return launch_status(launches);
}
