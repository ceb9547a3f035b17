// Block norms: argument checks, the split of the rows into segments and the
// sums of the segments' column sums (formulas in block_norm.cuh).
#include <initializer_list>

#include "block_norm.cuh"

namespace prism {
namespace bn {

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
    int64_t groups, segs, ld_scale, ld_gate;
    int C, per_group, wide;             // per_group as in BwdArgs
};

// The segments' column sums to the vectors' gradients.  32 channels a CTA, whose 16 warps take every 16th segment.
// The CTAs of a cluster share the work out among them: the segments where there is one group and a long one (`wide`)
// or each segment has whole groups, else the groups; the first of them adds up what the others have.  All in a fixed
// order, so that the result does not depend on scheduling.
constexpr int kJoinRows = 16, kMaxCluster = 8;
__global__ void __launch_bounds__(32 * kJoinRows) k_block_norm_join(const JoinArgs a) {
    __shared__ float sh[kJoinRows][3][32];
    __shared__ float sums[3][32];
    const int x = threadIdx.x, y = threadIdx.y, c = blockIdx.x * 32 + x;
    const bool in = c < a.C, affine = a.dw || a.db || a.dw_post;
    const int64_t n = gridDim.y, me = blockIdx.y;
    wait_for_previous();
    // v: the sums over the segments s0, s0 + 1, ... s1 - 1, in the threads y = 0
    auto read = [&](int64_t s0, int64_t s1, float (&v)[3]) {
        v[0] = v[1] = v[2] = 0.f;
        if (in) {
            const bool a0 = a.dscale || a.dw, a1 = a.dscale || a.dshift || a.db, a2 = a.dgate || a.dw_post;
#pragma unroll 4
            for (int64_t s = s0 + y; s < s1; s += kJoinRows) {
                const float* p = a.part + s * 3 * a.C + c;
                if (a0) v[0] += p[0];
                if (a1) v[1] += p[a.C];
                if (a2) v[2] += p[2 * a.C];
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) sh[y][i][x] = v[i];
        __syncthreads();
        if (y < 3) {
            float s = 0.f;
#pragma unroll 8
            for (int k = 0; k < kJoinRows; ++k) s += sh[k][y][x];
            sums[y][x] = s;
        }
        __syncthreads();
        if (y == 0) {
#pragma unroll
            for (int i = 0; i < 3; ++i) v[i] = sums[i][x];
        }
    };
    // v of the cluster's CTAs, added up in the first one
    auto gather = [&](float (&v)[3]) {
        if (n == 1) return;
        __syncthreads();
        if (y == 0) {
#pragma unroll
            for (int i = 0; i < 3; ++i) sums[i][x] = v[i];
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (me == 0) {
            for (int q = y; q < 3 * (int)n; q += kJoinRows) {      // a warp each, so that they are under way together
                const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&sums[q % 3][x]);
                uint32_t there;
                float f;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(q / 3));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(there) : "memory");
                sh[q / 3][q % 3][x] = f;
            }
            __syncthreads();
            if (y == 0)
                for (int k = 1; k < (int)n; ++k)
#pragma unroll
                    for (int i = 0; i < 3; ++i) v[i] += sh[k][i][x];
        }
        // no CTA overwrites its sums, or ends, while the first one reads them
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    float t[3] = {0.f, 0.f, 0.f};
    auto group = [&](int64_t g, const float (&v)[3]) {
        if (a.dscale) a.dscale[g * a.C + c] = fmaf(a.w ? a.w[c] : 1.f, v[0], a.b ? a.b[c] * v[1] : 0.f);
        if (a.dshift) a.dshift[g * a.C + c] = v[1];
        if (a.dgate) a.dgate[g * a.C + c] = a.w_post ? a.w_post[c] * v[2] : v[2];
        const float one = a.scale ? 1.f + a.scale[g * a.ld_scale + c] : 1.f;
        t[0] = fmaf(one, v[0], t[0]);
        t[1] = fmaf(one, v[1], t[1]);
        t[2] = fmaf(a.gate ? a.gate[g * a.ld_gate + c] : 1.f, v[2], t[2]);
    };
    float v[3];
    if (a.per_group == 0) {
        read(a.segs * me / n, a.segs * (me + 1) / n, t);
        gather(t);
    } else if (a.wide) {
        read(a.per_group * me / n, a.per_group * (me + 1) / n, v);
        gather(v);
        if (me == 0 && y == 0 && in) group(0, v);
    } else {
        for (int64_t g = me; g < a.groups; g += n) {
            read(g * a.per_group, (g + 1) * a.per_group, v);
            if (y == 0 && in) group(g, v);
        }
        if (affine) gather(t);          // the same for all CTAs of the cluster
    }
    if (me != 0 || y != 0 || !in) return;
    if (a.dw) a.dw[c] = t[0];
    if (a.db) a.db[c] = t[1];
    if (a.dw_post) a.dw_post[c] = t[2];
}

static prism_status_t launch_join(JoinArgs j, cudaStream_t stream) {
    // one group of 1184 segments: 6 us by a cluster, 11 by one CTA a column; of 148: 12 and 6; two of 592: 8 and 7
    j.wide = j.groups == 1 && j.per_group >= 512;
    const int64_t parts = j.per_group == 0 || j.wide ? kMaxCluster : j.groups;
    int n = 1;
    while (n < kMaxCluster && 2 * n <= parts) n *= 2;
    const dim3 grid((unsigned)((j.C + 31) / 32), (unsigned)n);
    return launch_after(k_block_norm_join, grid, dim3(32, kJoinRows), n, stream, j) ? PRISM_OK : PRISM_ERR_CUDA;
}

struct Split {
    int64_t groups, rpg, segs;
    int per_group;               // segments a group; 0: a segment has whole groups
};

// Segments of rows, one a CTA.  Where there are few groups, each is cut so that the segments fill the CTAs that run at
// a time once; where groups are many, into about eight rounds of such CTAs, so that the last round's idle part is
// small.  A segment has four rows a team at least (two where CTAs are left over): its column sums cost as much as three.
// Groups that are not cut are shared out among the teams in runs.
static Split split_rows(const prism_block_norm_t* n, bool one_group) {
    Split s{0, 1, 0, 0};
    if (n->rows == 0) return s;
    s.rpg = !one_group && n->rows_per_group < n->rows ? n->rows_per_group : n->rows;
    s.groups = (n->rows + s.rpg - 1) / s.rpg;
    const int ctas_sm = bwd_ctas(team_bucket(team_threads(n->channels)), n->branch_dtype == PRISM_F32);
    const int64_t teams = (int64_t)kSMs * sm_teams(n->channels, ctas_sm);
    const int64_t per_cta = cta_teams(n->channels), ctas = teams / per_cta;
    // of the CTAs a group's share by its rows: the last group may be shorter than the others
    int64_t per = (s.groups * 4 <= ctas ? ctas : 8 * ctas) * s.rpg / n->rows;
    int64_t most = (s.rpg + 4 * per_cta - 1) / (4 * per_cta);
    if (s.groups * most < ctas) most = (s.rpg + 2 * per_cta - 1) / (2 * per_cta);   // little work: the shorter chain counts
    if (per > most) per = most;
    // a group that is not cut keeps the teams of a CTA busy only if it is long
    if (per > 1 || (per_cta > 1 && s.rpg >= 8 && s.groups * 4 <= teams)) {
        s.per_group = per < 1 ? 1 : (int)per;
        s.segs = s.groups * s.per_group;
    } else {
        s.segs = s.groups < teams ? s.groups : teams;
    }
    return s;
}
static int64_t part_floats(const Split& s, int C) { return s.segs * 3 * C; }

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

// channels an access may take: all strides in use and the width are multiples of it, and all addresses of its bytes
static int unit_of(int wide, int C, std::initializer_list<int64_t> lds, std::initializer_list<const void*> ptrs) {
    Bits n, p;
    n.bytes(C);
    for (int64_t l : lds) n.bytes(l);
    for (const void* q : ptrs) p << q;
    return n.multiple_of(wide) && p.multiple_of(16) ? wide : n.multiple_of(2) && p.multiple_of(8) ? 2 : 1;
}

}  // namespace bn
}  // namespace prism

using namespace prism;
using namespace prism::bn;

extern "C" prism_status_t prism_block_norm_ws_bytes(const prism_block_norm_t* n, size_t* bytes) {
    const prism_status_t st = check(n);
    if (st != PRISM_OK) return st;
    if (!bytes) return PRISM_ERR_INVALID_ARG;
    const int64_t a = part_floats(split_rows(n, false), n->channels), b = part_floats(split_rows(n, true), n->channels);
    *bytes = (size_t)(a > b ? a : b) * sizeof(float);
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
    const int unit = unit_of(eb == 2 ? 8 : 4, C,
                             {a.ld_x, h ? a.ld_h : 0, h ? a.ld_z : 0, has_y ? a.ld_y : 0, gate ? a.ld_gate : 0,
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
            if (p && !taken(cudaMemsetAsync(p, 0, C * sizeof(float), stream))) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    const int es = esize(n->stream_dtype), eb = esize(n->branch_dtype);
    if (!opt_on(dz, es) || (has_y && (!on(z, es) || !on(dy, eb))) || !on(dx, es) || (h && (!on(h, eb) || !on(dh, eb))))
        return PRISM_ERR_INVALID_ARG;
    // rows that share all their vectors are one group
    const bool groups = dgate || dscale || dshift, affine = dw || db || dw_post;
    const Split s = split_rows(n, !groups && !gate && !scale);
    const bool part = affine || (groups && s.per_group > 0);
    if (part && (!ws || ws_bytes < (size_t)part_floats(s, C) * sizeof(float))) return PRISM_ERR_WORKSPACE;
    a.z = z; a.h = h; a.dz = dz; a.dy = dy;
    a.gate = gate; a.w_post = w_post; a.w = w; a.b = b; a.scale = scale;
    a.dx = dx; a.dh = dh;
    a.part = part ? (float*)ws : nullptr;
    if (s.per_group == 0) { a.dgate = dgate; a.dscale = dscale; a.dshift = dshift; }
    a.R = n->rows;
    a.rpg = s.rpg; a.groups = s.groups; a.segs = s.segs; a.per_group = s.per_group;
    a.C = C; a.norm = n->norm; a.post = n->post_norm; a.eps = n->eps; a.res = n->res_scale;
    const int unit = unit_of(es == 2 ? 8 : 4, C,
                             {has_y ? a.ld_z : 0, h ? a.ld_h : 0, dz ? a.ld_dz : 0, has_y ? a.ld_dy : 0, a.ld_dx,
                              h ? a.ld_dh : 0, gate ? a.ld_gate : 0, scale ? a.ld_scale : 0},
                             {has_y ? z : nullptr, h, gate, w_post, w, b, scale, dz, dy, dx, dh, dgate, dscale, dshift,
                              part ? ws : nullptr});
    if (n->stream_dtype == PRISM_BF16) st = launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, unit, stream);
    else if (n->branch_dtype == PRISM_BF16) st = launch_bwd<float, __nv_bfloat16>(a, unit, stream);
    else st = launch_bwd<float, float>(a, unit, stream);
    if (st != PRISM_OK) return st;
    if (!part) return launch_status(1);
    if (!launched()) return PRISM_ERR_CUDA;           // the join would add up what was never written
    st = launch_join(JoinArgs{(const float*)ws, w, b, w_post, scale, gate, s.per_group ? dgate : nullptr,
                              s.per_group ? dscale : nullptr, s.per_group ? dshift : nullptr, dw, db, dw_post, s.groups,
                              s.segs, a.ld_scale, a.ld_gate, C, s.per_group, 0},
                     stream);
    return st == PRISM_OK ? launch_status(2) : st;
}
