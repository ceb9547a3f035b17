// Tokens sorted by expert and back.
//
// A slot is one choice j of one token t, its flat index i = t k + j and its expert ids[i]; an id outside
// [0, E) drops the slot.  The sorted layout holds each expert's slots in ascending i, from row
// offsets[e] on, offsets[e + 1] = offsets[e] + counts[e] rounded up to a multiple of `align`:
//
//   pos[i] = row of slot i (-1: dropped),  src[row] = i (-1: no slot)
//   dispatch:  xs[pos[i]] = x[t]                        its gradient:  dx[t] = sum_j dxs[pos[i]]
//   combine:   out[t] = add[t] + sum_j w[i] y[pos[i]]   its gradient:  dy[pos[i]] = w[i] dout[t],
//                                                                     dw[i] = y[pos[i]] . dout[t]
//
// The moves are bound by HBM.  All of them go by token: a token's row is read or written once however many
// experts it has, and no two threads add to one value, so nothing is atomic and sums have a fixed order
// (j ascending, in fp32, one rounding at the store).  61440 x 2048 bf16, two choices: dispatch 114 us (117 at the
// measured copy rate), combine 113 (117), its backward 205 (194); 32768 x 1024, eight choices: dispatch 99 (93),
// combine 97 (93).
// The plan is bound by latency: a count of each CTA's slots and a placement, 11 us for 122880 slots of 16 experts, 21
// for 262144 of 128; by one CTA 6147 slots took 13 us, by two launches 10.
#include <initializer_list>

#include "rows.cuh"

namespace prism {
namespace ex {

using namespace rows;

constexpr int kMaxTopK = 16, kMaxExperts = 1024, kMaxAlign = 4096;
constexpr int kHist = 8192;                    // shared-memory counters: warps x experts
constexpr int kOneCta = 2048;                  // slots that one CTA sorts alone
constexpr int kTile = 1024;                    // slots a CTA at least, where several sort
constexpr int kBatch = 8;                      // ids of a lane that are on their way at a time

struct PlanArgs {
    const void* ids;
    int32_t *counts, *offsets, *pos, *src, *ws;     // ws [CTAs][E]: each CTA's counts
    int64_t n, cap;
    int E, align, id_bytes;
    int64_t tile;                                   // slots a CTA, a multiple of 32
};

__device__ __forceinline__ int expert_of(const PlanArgs& a, int64_t i, int64_t end) {
    if (i >= end) return -1;
    const int64_t v = a.id_bytes == 8 ? __ldg((const int64_t*)a.ids + i) : (int64_t)__ldg((const int32_t*)a.ids + i);
    return v >= 0 && v < a.E ? (int)v : -1;
}

// The slots of a CTA, cut into one contiguous run a warp; a warp counts 32 slots at a time, lanes with
// the same expert found by one match.
struct Runs {
    int64_t begin, end;      // of this warp
    int warps;               // that have a run
};
__device__ __forceinline__ Runs runs_of(const PlanArgs& a) {
    Runs r;
    const int most = kHist / a.E < 32 ? kHist / a.E : 32;
    const int64_t b0 = (int64_t)blockIdx.x * a.tile, b1 = b0 + a.tile < a.n ? b0 + a.tile : a.n;
    const int64_t steps = (b1 - b0 + 31) / 32, per = (steps + most - 1) / most;
    r.warps = per > 0 ? (int)((steps + per - 1) / per) : 0;
    const int w = threadIdx.x >> 5;
    r.begin = b0 + per * 32 * w;
    r.end = w < r.warps ? (r.begin + per * 32 < b1 ? r.begin + per * 32 : b1) : r.begin;
    return r;
}

// the experts of a lane's next kBatch slots from i on, 32 apart (-1: none)
__device__ __forceinline__ void batch_of(const PlanArgs& a, int64_t i, int64_t end, int (&e)[kBatch]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) e[j] = expert_of(a, i + 32 * j + lane, end);
}

// e holds the run's first batch, and still does afterwards where the run has no more
__device__ __forceinline__ void count_runs(const PlanArgs& a, const Runs& r, int* hist, int (&e)[kBatch]) {
    batch_of(a, r.begin, r.end, e);
    for (int i = threadIdx.x; i < r.warps * a.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    int* mine = hist + (threadIdx.x >> 5) * a.E;
    for (int64_t i = r.begin; i < r.end; i += 32 * kBatch) {
        if (i > r.begin) batch_of(a, i, r.end, e);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i + 32 * j >= r.end) break;
            const unsigned same = __match_any_sync(0xffffffffu, e[j]);
            if (e[j] >= 0 && (same & ((1u << lane) - 1)) == 0) mine[e[j]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
}

// exclusive sum over a CTA of 1024 threads; *total gets the whole sum
__device__ __forceinline__ int cta_scan(int v, int* sh, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) sh[w] = s;
    __syncthreads();
    if (w == 0) {
        int t = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += u;
        }
        sh[lane] = t;
    }
    __syncthreads();
    *total = sh[31];
    return s - v + (w ? sh[w - 1] : 0);
}

// Where several CTAs sort: each CTA's counts.
__global__ void __launch_bounds__(1024) k_expert_count(const PlanArgs a) {
    __shared__ int hist[kHist];
    let_next_start();
    const Runs r = runs_of(a);
    int ids[kBatch];
    count_runs(a, r, hist, ids);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int s = 0;
#pragma unroll 8
        for (int w = 0; w < r.warps; ++w) s += hist[w * a.E + e];
        a.ws[(int64_t)blockIdx.x * a.E + e] = s;
    }
}

// Ranks and rows.  A slot's row = its expert's offset + the expert's slots in earlier CTAs, earlier warps of
// this CTA and earlier lanes.  Every CTA sums the counts of all CTAs itself (a few hundred KB from L2), which
// takes less time than a launch of its own for it.
__global__ void __launch_bounds__(1024, 2) k_expert_place(const PlanArgs a) {
    __shared__ int hist[kHist], before[kMaxExperts], total[kMaxExperts], sh[32];
    const int E = a.E, tid = threadIdx.x;
    const Runs r = runs_of(a);
    for (int e = tid; e < E; e += 1024) before[e] = total[e] = 0;
    int ids[kBatch];
    count_runs(a, r, hist, ids);
    if (gridDim.x > 1) {
        wait_for_previous();             // the counts of all CTAs, and what was in the outputs before
        const int groups = 1024 / E, e = tid % E, gr = tid / E;
        if (gr < groups) {
            int p = 0, t = 0;
#pragma unroll 8
            for (int b = gr; b < (int)gridDim.x; b += groups) {
                const int c = a.ws[(int64_t)b * E + e];
                t += c;
                if (b < (int)blockIdx.x) p += c;
            }
            atomicAdd(&before[e], p);         // integers: the order does not matter
            atomicAdd(&total[e], t);
        }
        __syncthreads();
    }
    int run = 0;
    if (tid < E) {
        if (gridDim.x > 1) run = before[tid];
        for (int w = 0; w < r.warps; ++w) {
            const int c = hist[w * E + tid];
            hist[w * E + tid] = run;
            run += c;
        }
        if (gridDim.x == 1) total[tid] = run;
    }
    const int mine = tid < E ? total[tid] : 0;
    int whole;
    const int off = cta_scan((mine + a.align - 1) / a.align * a.align, sh, &whole);
    if (tid < E) {
        before[tid] = off;
        if (blockIdx.x == 0) {
            a.counts[tid] = mine;
            a.offsets[tid] = off;
            if (tid == 0) a.offsets[E] = whole;
        }
    }
    __syncthreads();

    const int lane = tid & 31;
    int* rank = hist + (tid >> 5) * E;
    const bool again = r.end - r.begin > 32 * kBatch;
    for (int64_t i0 = r.begin; i0 < r.end; i0 += 32 * kBatch) {
        if (again) batch_of(a, i0, r.end, ids);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t i = i0 + 32 * j;
            if (i >= r.end) break;
            const int e = ids[j];
            const unsigned same = __match_any_sync(0xffffffffu, e), lower = same & ((1u << lane) - 1);
            int row = -1;
            if (e >= 0) row = before[e] + rank[e] + __popc(lower);
            __syncwarp();
            if (e >= 0 && lower == 0) rank[e] += __popc(same);
            __syncwarp();
            if (i + lane < r.end) {
                a.pos[i + lane] = row;
                if (row >= 0) a.src[row] = (int32_t)(i + lane);
            }
        }
    }
    // rows without a slot: behind each expert's last one (a warp an expert), and behind the last expert
    if (a.align > 1)
        for (int e = (int)blockIdx.x * 32 + (tid >> 5); e < E; e += (int)gridDim.x * 32) {
            const int next = e + 1 < E ? before[e + 1] : whole;
            for (int row = before[e] + total[e] + lane; row < next; row += 32) a.src[row] = -1;
        }
    for (int64_t row = whole + (int64_t)blockIdx.x * 1024 + tid; row < a.cap; row += (int64_t)gridDim.x * 1024)
        a.src[row] = -1;
}

// ------------------------------------------------------------------ moves
struct MoveArgs {
    const void *in, *y, *add;            // by token; sorted; by token
    void *out, *dy;                      // by token; sorted
    const int32_t *pos, *counts, *offsets;
    const float* w;
    float* dw;
    int64_t R, cap, ld_in, ld_out, ld_add;   // strides in elements
    int C, k, E, units, segs;                // units: accesses a row; segs: warps a row
    unsigned token_ctas;                     // CTAs that move rows; those behind them clear some
    int gap_ctas;
};

// CTAs behind the tokens' write zeros: one an expert the rows of its last, partial unit of `align`, so that a
// product over whole units gets nothing from them, and kTailCtas, where asked for, the rows behind the last expert.
constexpr int kTailCtas = kSMs;
template <typename T, int N> __device__ __forceinline__ void clear_rows(const MoveArgs& a, T* sorted) {
    const int i = (int)(blockIdx.x - a.token_ctas);
    int64_t r0, r1;
    if (i < a.gap_ctas) {
        r0 = (int64_t)a.offsets[i] + a.counts[i];
        r1 = a.offsets[i + 1];
    } else {
        const int64_t used = a.offsets[a.E], left = a.cap - used;
        r0 = used + left * (i - a.gap_ctas) / kTailCtas;
        r1 = used + left * (i - a.gap_ctas + 1) / kTailCtas;
    }
    if (r0 < 0 || r1 > a.cap) return;
    Pack<T, N> z;
#pragma unroll
    for (int j = 0; j < (int)(sizeof(z.w) / 4); ++j) z.w[j] = 0u;
    // rows are dense: one run of accesses
    T* p = sorted + r0 * a.C;
    const int64_t n = (r1 - r0) * a.units;
    for (int64_t u = threadIdx.x; u < n; u += blockDim.x) store(p + u * N, z);
}

// this token's rows: lane j holds pos of choice j, -1 where there is none
__device__ __forceinline__ int64_t token_pos(const MoveArgs& a, int64_t t, int lane) {
    int64_t p = lane < a.k ? (int64_t)__ldg(a.pos + t * a.k + lane) : -1;
    return p < a.cap ? p : -1;               // a row that the plan cannot have written is never touched
}

template <typename T, int N> __global__ void __launch_bounds__(256) k_expert_dispatch(const MoveArgs a) {
    constexpr int U = 4;
    if (blockIdx.x >= a.token_ctas) return clear_rows<T, N>(a, (T*)a.dy);
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), t = item / a.segs;
    if (t >= a.R) return;
    const int u0 = (int)(item - t * a.segs) * (32 * U) + lane;
    const T* in = (const T*)a.in + t * a.ld_in;
    Pack<T, N> v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (u0 + 32 * i < a.units) load(v[i], in + (u0 + 32 * i) * N);
    const int64_t p = token_pos(a, t, lane);
    for (int j = 0; j < a.k; ++j) {
        const int64_t row = __shfl_sync(0xffffffffu, p, j);
        if (row < 0) continue;
        T* out = (T*)a.dy + row * a.C;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (u0 + 32 * i < a.units) store(out + (u0 + 32 * i) * N, v[i]);
    }
}

// J choices at a time with U accesses of a lane each, eight on their way; ALL: there are no more than J choices, and
// each access is summed and stored by itself.
template <typename T, int N, int J, bool ALL> __global__ void __launch_bounds__(256) k_expert_combine(const MoveArgs a) {
    constexpr int U = 8 / J;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int64_t item = (int64_t)blockIdx.x * 8 + warp, t = item / a.segs;
    if (t >= a.R) return;
    const int u0 = (int)(item - t * a.segs) * (32 * U) + lane;
    const int64_t p = token_pos(a, t, lane);
    const float w = a.w && lane < a.k ? __ldg(a.w + t * a.k + lane) : 1.f;
    const T* add = a.add ? (const T*)a.add + t * a.ld_add : nullptr;
    T* out = (T*)a.out + t * a.ld_out;
    Pack<T, N> v[J][U];
    int64_t row[J];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            row[j] = __shfl_sync(0xffffffffu, p, (j0 + j) & 31);
            if (j0 + j >= a.k) row[j] = -1;
            if (row[j] >= 0) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (u0 + 32 * i < a.units) load(v[j][i], (const T*)a.y + row[j] * a.C + (u0 + 32 * i) * N);
            }
        }
    };
    auto start = [&](int i, float* s) {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = 0.f;
        if (add && u0 + 32 * i < a.units) {
            Pack<T, N> q;
            load(q, add + (u0 + 32 * i) * N);
            unpack<N>(q, s);
        }
    };
    auto finish = [&](int i, const float* s) {
        if (u0 + 32 * i < a.units) {
            Pack<T, N> q;
            pack<N>(q, s);
            store(out + (u0 + 32 * i) * N, q);
        }
    };
    if constexpr (ALL) {
        fetch(0);
        float wj[J];
#pragma unroll
        for (int j = 0; j < J; ++j) wj[j] = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float s[N];
            start(i, s);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (row[j] >= 0) {                        // a dropped choice's weight, NaN or not, is not used
                    float f[N];
                    unpack<N>(v[j][i], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) s[e] = fmaf(wj[j], f[e], s[e]);
                }
            finish(i, s);
        }
    } else {
        float s[U][N];
#pragma unroll
        for (int i = 0; i < U; ++i) start(i, s[i]);
        for (int j0 = 0; j0 < a.k; j0 += J) {
            fetch(j0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                if (row[j] < 0) continue;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    float f[N];
                    unpack<N>(v[j][i], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) s[i][e] = fmaf(wj, f[e], s[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) finish(i, s[i]);
    }
}

// segs warps of a CTA share a token; K >= k choices, whose dot products stay in registers
template <typename T, int N, int K> __global__ void __launch_bounds__(256) k_expert_combine_bwd(const MoveArgs a) {
    __shared__ float sh[8][K];
    if (blockIdx.x >= a.token_ctas) return clear_rows<T, N>(a, (T*)a.dy);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (8 / a.segs) + warp / a.segs;
    const int part = warp % a.segs;
    const bool in = t < a.R;
    const int64_t p = in ? token_pos(a, t, lane) : -1;
    const float w = a.w && in && lane < a.k ? __ldg(a.w + t * a.k + lane) : 1.f;
    int64_t row[K];
    float wj[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        row[j] = __shfl_sync(0xffffffffu, p, j);
        wj[j] = __shfl_sync(0xffffffffu, w, j);
        dot[j] = 0.f;
    }
    if (in) {
        for (int u = part * 32 + lane; u < a.units; u += a.segs * 32) {
            Pack<T, N> d, v[K];
            load(d, (const T*)a.in + t * a.ld_in + (int64_t)u * N);
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (row[j] >= 0) load(v[j], (const T*)a.y + row[j] * a.C + (int64_t)u * N);
            }
            float g[N];
            unpack<N>(d, g);
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (row[j] >= 0) {
                    float f[N];
                    if (a.dw) {
                        unpack<N>(v[j], f);
#pragma unroll
                        for (int e = 0; e < N; ++e) dot[j] = fmaf(f[e], g[e], dot[j]);
                    }
#pragma unroll
                    for (int e = 0; e < N; ++e) f[e] = wj[j] * g[e];
                    Pack<T, N> o;
                    pack<N>(o, f);
                    store((T*)a.dy + row[j] * a.C + (int64_t)u * N, o);
                }
        }
    }
    if (!a.dw) return;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        dot[j] = warp_sum(dot[j]);
        if (lane == 0) sh[warp][j] = dot[j];
    }
    __syncthreads();
    if (in && part == 0 && lane < a.k) {
        float s = 0.f;
        for (int i = 0; i < a.segs; ++i) s += sh[warp + i][lane];
        a.dw[t * a.k + lane] = s;
    }
}

// ------------------------------------------------------------------ host
static prism_status_t check(const prism_experts_t* e) {
    if (!e) return PRISM_ERR_INVALID_ARG;
    if (e->rows < 0 || e->top_k < 1 || e->experts < 1 || e->align < 1) return PRISM_ERR_SHAPE;
    if (e->top_k > kMaxTopK || e->experts > kMaxExperts || e->align > kMaxAlign) return PRISM_ERR_UNSUPPORTED;
    if (e->rows > (int64_t(1) << 30) / e->top_k) return PRISM_ERR_UNSUPPORTED;
    if (e->id_bytes != 4 && e->id_bytes != 8) return PRISM_ERR_INVALID_ARG;
    return PRISM_OK;
}

static int64_t capacity(const prism_experts_t* e) {
    const int64_t n = e->rows * e->top_k;
    return n + (n < e->experts ? n : e->experts) * (e->align - 1);
}

// slots a CTA: all of them where one CTA sorts alone, else a share of at most 148
static int64_t tile_of(const prism_experts_t* e) {
    const int64_t n = e->rows * e->top_k;
    if (n <= kOneCta) return n > 0 ? (n + 31) / 32 * 32 : 32;
    int64_t t = (n + kSMs - 1) / kSMs;
    if (t < kTile) t = kTile;
    return (t + 31) / 32 * 32;
}
static int64_t ctas_of(const prism_experts_t* e) {
    const int64_t n = e->rows * e->top_k, t = tile_of(e);
    return n > 0 ? (n + t - 1) / t : 1;
}

// bytes an access: 16 where every row starts on 16 bytes, else 4 or one element
static int unit_bytes(int esz, int64_t C, std::initializer_list<int64_t> lds, std::initializer_list<const void*> ptrs) {
    Bits m;
    m.bytes(C * esz);
    for (int64_t l : lds) m.bytes(l * esz);
    for (const void* p : ptrs) m << p;
    return m.multiple_of(16) ? 16 : m.multiple_of(4) ? 4 : 2;
}

static prism_status_t move_args(const prism_experts_t* e, int dtype, int64_t channels, const int32_t* pos, MoveArgs* a) {
    const prism_status_t st = check(e);
    if (st != PRISM_OK) return st;
    if (dtype != PRISM_F32 && dtype != PRISM_BF16) return PRISM_ERR_UNSUPPORTED;
    if (channels < 1) return PRISM_ERR_SHAPE;
    if (channels > (1 << 20)) return PRISM_ERR_UNSUPPORTED;
    *a = MoveArgs{};
    a->R = e->rows; a->cap = capacity(e); a->C = (int)channels; a->k = e->top_k; a->E = e->experts;
    a->pos = pos;
    return PRISM_OK;
}

#define PRISM_EX_BY_UNIT(KERNEL, B, GRID, S, A)                                        \
    do {                                                                               \
        if (dtype == PRISM_BF16) {                                                     \
            if ((B) == 16) KERNEL<__nv_bfloat16, 8><<<GRID, 256, 0, S>>>(A);           \
            else if ((B) == 4) KERNEL<__nv_bfloat16, 2><<<GRID, 256, 0, S>>>(A);       \
            else KERNEL<__nv_bfloat16, 1><<<GRID, 256, 0, S>>>(A);                     \
        } else {                                                                       \
            if ((B) == 16) KERNEL<float, 4><<<GRID, 256, 0, S>>>(A);                   \
            else KERNEL<float, 1><<<GRID, 256, 0, S>>>(A);                             \
        }                                                                              \
    } while (0)

template <int J, bool ALL> static void launch_combine(int dtype, int b, unsigned grid, cudaStream_t s, const MoveArgs& a) {
    if (dtype == PRISM_BF16) {
        if (b == 16) k_expert_combine<__nv_bfloat16, 8, J, ALL><<<grid, 256, 0, s>>>(a);
        else if (b == 4) k_expert_combine<__nv_bfloat16, 2, J, ALL><<<grid, 256, 0, s>>>(a);
        else k_expert_combine<__nv_bfloat16, 1, J, ALL><<<grid, 256, 0, s>>>(a);
    } else {
        if (b == 16) k_expert_combine<float, 4, J, ALL><<<grid, 256, 0, s>>>(a);
        else k_expert_combine<float, 1, J, ALL><<<grid, 256, 0, s>>>(a);
    }
}

template <int K> static void launch_bwd(int dtype, int b, unsigned grid, cudaStream_t s, const MoveArgs& a) {
    if (dtype == PRISM_BF16) {
        if (b == 16) k_expert_combine_bwd<__nv_bfloat16, 8, K><<<grid, 256, 0, s>>>(a);
        else if (b == 4) k_expert_combine_bwd<__nv_bfloat16, 2, K><<<grid, 256, 0, s>>>(a);
        else k_expert_combine_bwd<__nv_bfloat16, 1, K><<<grid, 256, 0, s>>>(a);
    } else {
        if (b == 16) k_expert_combine_bwd<float, 4, K><<<grid, 256, 0, s>>>(a);
        else k_expert_combine_bwd<float, 1, K><<<grid, 256, 0, s>>>(a);
    }
}

// the grid: CTAs that move rows, then those that clear some; false where a grid cannot hold them
static bool grid_of(int64_t ctas, bool sorted_out, int align, int clear_tail, MoveArgs* a, unsigned* grid) {
    a->gap_ctas = sorted_out && align > 1 ? a->E : 0;
    const int64_t n = ctas + a->gap_ctas + (sorted_out && clear_tail ? kTailCtas : 0);
    if (n > INT32_MAX) return false;
    a->token_ctas = (unsigned)ctas;
    *grid = (unsigned)n;
    return true;
}

}  // namespace ex
}  // namespace prism

using namespace prism;
using namespace prism::ex;

extern "C" prism_status_t prism_expert_sizes(const prism_experts_t* e, int64_t* rows_sorted, size_t* ws_bytes) {
    const prism_status_t st = check(e);
    if (st != PRISM_OK) return st;
    if (!rows_sorted || !ws_bytes) return PRISM_ERR_INVALID_ARG;
    *rows_sorted = capacity(e);
    const int64_t ctas = ctas_of(e);
    *ws_bytes = ctas > 1 ? (size_t)ctas * e->experts * sizeof(int32_t) : 0;
    return PRISM_OK;
}

extern "C" prism_status_t prism_expert_plan(const prism_experts_t* e, const void* ids, int32_t* counts, int32_t* offsets,
                                            int32_t* pos, int32_t* src, void* ws, size_t ws_bytes, cudaStream_t stream) {
    const prism_status_t st = check(e);
    if (st != PRISM_OK) return st;
    if (!on(counts, 4) || !on(offsets, 4) || !opt_on(ws, 4)) return PRISM_ERR_INVALID_ARG;
    if (e->rows > 0 && (!on(ids, e->id_bytes) || !on(pos, 4) || !on(src, 4))) return PRISM_ERR_INVALID_ARG;
    const int64_t ctas = ctas_of(e);
    if (ctas > 1 && (!ws || ws_bytes < (size_t)ctas * e->experts * sizeof(int32_t))) return PRISM_ERR_WORKSPACE;
    const PlanArgs a{ids, counts, offsets, pos, src, (int32_t*)ws, e->rows * e->top_k, capacity(e),
                     e->experts, e->align, e->id_bytes, tile_of(e)};
    if (ctas == 1) {
        k_expert_place<<<1, 1024, 0, stream>>>(a);
        return launch_status(1);
    }
    k_expert_count<<<(unsigned)ctas, 1024, 0, stream>>>(a);
    if (!launched() || !launch_after(k_expert_place, dim3((unsigned)ctas), dim3(1024), 1, stream, a)) return PRISM_ERR_CUDA;
    return launch_status(2);
}

extern "C" prism_status_t prism_expert_dispatch(const prism_experts_t* e, int32_t dtype, int64_t channels, const void* x,
                                                int64_t ld_x, const int32_t* pos, const int32_t* counts,
                                                const int32_t* offsets, int32_t clear_tail, void* xs,
                                                cudaStream_t stream) {
    MoveArgs a;
    const prism_status_t st = move_args(e, dtype, channels, pos, &a);
    if (st != PRISM_OK) return st;
    if (!ld_of(ld_x, channels, &a.ld_in)) return PRISM_ERR_SHAPE;
    if (clear_tail != 0 && clear_tail != 1) return PRISM_ERR_INVALID_ARG;
    if (e->rows == 0) return PRISM_OK;
    const int esz = esize(dtype);
    if (!on(x, esz) || !on(pos, 4) || !on(counts, 4) || !on(offsets, 4) || !on(xs, esz)) return PRISM_ERR_INVALID_ARG;
    a.in = x; a.dy = xs; a.counts = counts; a.offsets = offsets;
    const int b = unit_bytes(esz, channels, {a.ld_in}, {x, xs});
    a.units = (int)(channels * esz / b);
    a.segs = (a.units + 127) / 128;
    unsigned grid;
    if (!grid_of((a.R * a.segs + 7) / 8, true, e->align, clear_tail, &a, &grid)) return PRISM_ERR_UNSUPPORTED;
    PRISM_EX_BY_UNIT(k_expert_dispatch, b, grid, stream, a);
    return launch_status(1);
}

extern "C" prism_status_t prism_expert_combine(const prism_experts_t* e, int32_t dtype, int64_t channels, const void* y,
                                               const int32_t* pos, const float* weights, const void* add, int64_t ld_add,
                                               void* out, int64_t ld_out, cudaStream_t stream) {
    MoveArgs a;
    const prism_status_t st = move_args(e, dtype, channels, pos, &a);
    if (st != PRISM_OK) return st;
    if (!ld_of(ld_out, channels, &a.ld_out) || !ld_of(ld_add, channels, &a.ld_add)) return PRISM_ERR_SHAPE;
    if (e->rows == 0) return PRISM_OK;
    const int esz = esize(dtype);
    if (!on(y, esz) || !on(pos, 4) || !opt_on(weights, 4) || !opt_on(add, esz) || !on(out, esz))
        return PRISM_ERR_INVALID_ARG;
    a.y = y; a.w = weights; a.add = add; a.out = out;
    const int b = unit_bytes(esz, channels, {a.ld_out, add ? a.ld_add : 0}, {y, add, out});
    a.units = (int)(channels * esz / b);
    // choices at a time: up to four, or eight of short rows, whose lanes' further accesses would be idle
    int J = a.k <= 1 ? 1 : a.k <= 2 ? 2 : 4;
    if (a.units <= 32 && a.k > 4) J = 8;
    const int lanes = 32 * (8 / J);
    a.segs = (a.units + lanes - 1) / lanes;
    unsigned grid;
    if (!grid_of((a.R * a.segs + 7) / 8, false, 1, 0, &a, &grid)) return PRISM_ERR_UNSUPPORTED;
    if (J == 1) launch_combine<1, true>(dtype, b, grid, stream, a);
    else if (J == 2) launch_combine<2, true>(dtype, b, grid, stream, a);
    else if (J == 8 && a.k <= 8) launch_combine<8, true>(dtype, b, grid, stream, a);
    else if (J == 8) launch_combine<8, false>(dtype, b, grid, stream, a);
    else if (a.k <= 4) launch_combine<4, true>(dtype, b, grid, stream, a);
    else launch_combine<4, false>(dtype, b, grid, stream, a);
    return launch_status(1);
}

extern "C" prism_status_t prism_expert_combine_bwd(const prism_experts_t* e, int32_t dtype, int64_t channels,
                                                   const void* dout, int64_t ld_dout, const void* y, const int32_t* pos,
                                                   const float* weights, const int32_t* counts, const int32_t* offsets,
                                                   int32_t clear_tail, void* dy, float* dweights,
                                                   cudaStream_t stream) {
    MoveArgs a;
    const prism_status_t st = move_args(e, dtype, channels, pos, &a);
    if (st != PRISM_OK) return st;
    if (!ld_of(ld_dout, channels, &a.ld_in)) return PRISM_ERR_SHAPE;
    if (clear_tail != 0 && clear_tail != 1) return PRISM_ERR_INVALID_ARG;
    if (e->rows == 0) return PRISM_OK;
    const int esz = esize(dtype);
    if (!on(dout, esz) || (dweights && !on(y, esz)) || !on(pos, 4) || !opt_on(weights, 4) || !on(counts, 4) ||
        !on(offsets, 4) || !on(dy, esz) || !opt_on(dweights, 4))
        return PRISM_ERR_INVALID_ARG;
    a.in = dout; a.y = y; a.w = weights; a.dw = dweights; a.dy = dy; a.counts = counts; a.offsets = offsets;
    const int b = unit_bytes(esz, channels, {a.ld_in}, {dout, dweights ? y : nullptr, dy});
    a.units = (int)(channels * esz / b);
    // warps a token: one where the tokens fill the GPU, more where they do not and the row has work for them
    a.segs = 1;
    while (a.segs < 8 && a.R * a.segs < kSMs * 32 && a.units > 32 * a.segs) a.segs *= 2;
    unsigned grid;
    const int per = 8 / a.segs;
    if (!grid_of((a.R + per - 1) / per, true, e->align, clear_tail, &a, &grid)) return PRISM_ERR_UNSUPPORTED;
    if (a.k == 1) launch_bwd<1>(dtype, b, grid, stream, a);
    else if (a.k == 2) launch_bwd<2>(dtype, b, grid, stream, a);
    else if (a.k <= 4) launch_bwd<4>(dtype, b, grid, stream, a);
    else if (a.k <= 8) launch_bwd<8>(dtype, b, grid, stream, a);
    else launch_bwd<16>(dtype, b, grid, stream, a);
    return launch_status(1);
}
