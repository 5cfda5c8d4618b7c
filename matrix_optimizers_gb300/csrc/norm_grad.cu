// The gradient of block_norm (see norm.cu): with yn = y ry,
//   t = dy + ry (dh pre - yn mean(dh pre yn))          dresidual = residual_scale t
//   c = block_scale t g post,  xn = x rx               dx = rx (c - xn mean(c xn))
//   dpre = sum dh yn,   S = block_scale sum t xn,      dpost = sum over gates of g S,  dgate = post S
// Since t is linear in dy, dh pre and y, all means come from six sums over x, y, dy and dh,
// taken at once.  One pass over the rows as forward.  A block's rows belong to one gate at a time, so that
// S is summed in registers.
//
// 16384 rows of 4096 (bf16, float32 stream; 1.21 GB): 195 us with the sums' joining, 6.2 TB/s, 92 % of a
// copy's rate; 238 us with 512 threads of 16 columns, whose values do not fit in registers.
#include "norm_common.cuh"

namespace mo {
namespace {

struct GradArgs {
    mo_block_norm p;
    const void* y;
    const void* dy;
    const void* dh;
    void* dx;
    void* dres;
    int64_t ldy, lddy, lddh, lddx, lddr;
    // the rows of a gate are cut into `cuts` units, a block takes units a grid apart
    int64_t gates, units;
    int cuts, parts, accumulate;
    float *dpost, *dgate, *dpre;
    float *part_post, *part_pre, *part_s;      // [parts][dim], [parts][dim], [units][dim]
    NormShape shape;
};

template <typename X, typename S, int K, int kMode, int L, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) norm_grad_kernel(GradArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ __align__(16) TeamRed red;
    launch_dependents();
    constexpr int V = kPiece<X, S>;
    using C = Cols<K, V, kMode, L>;
    const mo_block_norm& p = a.p;
    const C cols(p.dim, a.shape.threads);
    TeamSum<C, L> team(cols, red);
    const float inv_dim = 1.f / static_cast<float>(p.dim);
    const bool want_s = a.dpost != nullptr || a.dgate != nullptr, pre = p.pre != nullptr, given = a.dy != nullptr;
    Gains<K, V, kMode, L> in(cols, smem), gains(cols, smem + a.shape.gains);     // block_scale gate post;  pre
    char* stages = smem + 2 * a.shape.gains + cols.team * a.shape.count * a.shape.bytes;
    Rows<X, K, V, kMode, L> xs(cols, p.ldx, stages, a.shape.at[0]), dhs(cols, a.lddh, stages, a.shape.at[3]);
    Rows<S, K, V, kMode, L> ys(cols, a.ldy, stages, a.shape.at[1]), dys(cols, a.lddy, stages, a.shape.at[2]);
    Ahead ahead(a.shape.bytes, a.shape.count);
    auto fetch = [&](bool wanted, int stage) {
        if (wanted) {
            xs.fetch(stage);
            if (given) dys.fetch(stage);
            if (pre) {
                ys.fetch(stage);
                dhs.fetch(stage);
            }
        }
        ahead.close();
    };
    float acc_pre[K];
#pragma unroll
    for (int j = 0; j < K; ++j) acc_pre[j] = 0.f;
    if (cols.team == 0) {
        float v[K];
        cols.param(p.pre, p.param_dtype, 0, v);
#pragma unroll
        for (int j = 0; j < K; ++j) gains.set(j, v[j]);
    }
    // v of the first team becomes the sum over the teams, in their order, by way of `in`
    auto join_teams = [&](float (&v)[K], Gains<K, V, kMode, L>& by) {
        constexpr int kTeams = 32 / L;              // of a warp
        const int last = a.shape.teams / kTeams - 1;
#pragma unroll
        for (int o = L; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < K; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        for (int k = last; k >= 0; --k) {
            __syncthreads();
            if (cols.team / kTeams != k) continue;
            if (k < last) {
                float w[K];
                by.get(w);
#pragma unroll
                for (int j = 0; j < K; ++j) v[j] += w[j];
            }
            if (k > 0) {
#pragma unroll
                for (int j = 0; j < K; ++j) by.set(j, v[j]);
            }
        }
    };
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int64_t gate = u / a.cuts, cut = u - gate * a.cuts;
        const int64_t begin = p.gate != nullptr ? gate * p.rows_per_gate : 0;
        const int64_t rows = p.gate != nullptr ? min(p.rows_per_gate, p.n - begin) : p.n;
        const int64_t cuts = static_cast<int64_t>(a.cuts) * a.shape.teams, mine = cut * a.shape.teams + cols.team;
        const int64_t r0 = begin + rows * mine / cuts;
        const int count = static_cast<int>(begin + rows * (mine + 1) / cuts - r0);
        xs.start(p.x, r0);
        ys.start(a.y, r0);
        dys.start(a.dy, r0);
        dhs.start(a.dh, r0);
        ahead.turn = 0;                             // (of the unit before, only empty groups are left)
        for (int k = 0; k < ahead.count; ++k) fetch(k < count, k * ahead.bytes);
        __syncthreads();                            // the other teams are done with the gains
        if (cols.team == 0) {
            float g[K], v[K];
            cols.param(p.gate, p.param_dtype, gate * p.ldgate, g);
            cols.param(p.post, p.param_dtype, 0, v);
#pragma unroll
            for (int j = 0; j < K; ++j) in.set(j, p.block_scale * g[j] * v[j]);
        }
        __syncthreads();
        float acc[K];                               // sum of t xn
#pragma unroll
        for (int j = 0; j < K; ++j) acc[j] = 0.f;
        X* dx_row = static_cast<X*>(a.dx) + r0 * a.lddx + cols.base;
        S* dr_row = static_cast<S*>(a.dres) + r0 * a.lddr + cols.base;
        int left = count;
        for (int turns = turns_of<L>(left); turns > 0; --turns, --left, dx_row += a.lddx, dr_row += a.lddr) {
            Held<X, K> x, dh;
            Held<S, K> y, dy;
            float w[K];
            ahead.wait();
            if (kMode == kNarrow) cols.sync();
            xs.read(ahead.turn, x);
            if (given) {
                dys.read(ahead.turn, dy);
            } else {
#pragma unroll
                for (uint32_t& v : dy.w) v = 0;
            }
            if (pre) {
                ys.read(ahead.turn, y);
                dhs.read(ahead.turn, dh);
            }
            if (kMode == kNarrow) cols.sync();
            fetch(ahead.count < left, ahead.turn);
            ahead.next();
            // x^2, y^2, p y, c dy, c p, c y   with p = dh pre, c = block_scale g post x
            float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, c[K];
            in.get(c);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                s[0] = fmaf(x[j], x[j], s[0]);
                s[3] = fmaf(c[j] * x[j], dy[j], s[3]);
            }
            if (pre) {
                gains.get(w);
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const float pj = dh[j] * w[j], cj = c[j] * x[j];
                    s[1] = fmaf(y[j], y[j], s[1]);
                    s[2] = fmaf(pj, y[j], s[2]);
                    s[4] = fmaf(cj, pj, s[4]);
                    s[5] = fmaf(cj, y[j], s[5]);
                }
            }
            team.sum(s);
            if (L < 32 && left <= 0) continue;
            const float rx = p.post != nullptr ? rsqrtf(s[0] * inv_dim + p.eps) : 1.f;
            float t[K], mx = s[3];                   // sum of c t, t being linear in dy, p and y
#pragma unroll
            for (int j = 0; j < K; ++j) t[j] = dy[j];
            if (pre) {
                const float ry = rsqrtf(s[1] * inv_dim + p.eps), back = ry * ry * (s[2] * ry * inv_dim);  // ry^2 mean(p yn)
                mx += ry * s[4] - back * s[5];
                gains.get(w);
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    acc_pre[j] = fmaf(dh[j], y[j] * ry, acc_pre[j]);
                    t[j] += ry * (dh[j] * w[j]) - back * y[j];
                }
            }
            if (a.dres != nullptr) {
#pragma unroll
                for (int j = 0; j < K; ++j) w[j] = p.residual_scale * t[j];
                cols.store(dr_row, w);
            }
            const bool post = p.post != nullptr;
            mx *= rx * rx * inv_dim;                 // rx mean(c xn)
            in.get(c);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const float xn = x[j] * rx;          // (x itself without a post norm)
                acc[j] = fmaf(t[j], xn, acc[j]);
                t[j] = post ? rx * (t[j] * c[j] - x[j] * mx) : t[j] * c[j];
            }
            cols.store(dx_row, t);
        }
        if (!want_s) continue;
        join_teams(acc, in);
        if (cols.team != 0) continue;
        float* to_post = a.part_post + static_cast<int64_t>(blockIdx.x) * p.dim + cols.base;
        float* to_s = (a.cuts == 1 ? a.dgate + gate * p.dim : a.part_s + u * p.dim) + cols.base;
        float v[K], old[K];
#pragma unroll
        for (int j = 0; j < K; ++j) acc[j] *= p.block_scale;
        if (a.dpost != nullptr) {
            const bool more = u != blockIdx.x;
            cols.param(p.gate, p.param_dtype, gate * p.ldgate, v);
#pragma unroll
            for (int j = 0; j < K; ++j) old[j] = more && cols.has(j) ? to_post[C::step(j)] : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (cols.has(j)) to_post[C::step(j)] = old[j] + v[j] * acc[j];
        }
        if (a.dgate != nullptr) {
            const bool whole = a.cuts == 1, more = whole && a.accumulate;
            cols.param(whole ? p.post : nullptr, p.param_dtype, 0, v);
#pragma unroll
            for (int j = 0; j < K; ++j) old[j] = more && cols.has(j) ? to_s[C::step(j)] : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (cols.has(j)) to_s[C::step(j)] = old[j] + v[j] * acc[j];
        }
    }
    if (a.dpre == nullptr) return;
    join_teams(acc_pre, in);
    if (cols.team != 0) return;
    float* to = a.part_pre + static_cast<int64_t>(blockIdx.x) * p.dim + cols.base;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (cols.has(j)) to[C::step(j)] = acc_pre[j];
}

// Joins the blocks' sums: 32 columns to a block, 8 warps over the parts.
// blockIdx.y: 0 dpre, 1 dpost, 2 + g: gate g's units.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(GradArgs a) {
    __shared__ float s[kJoinWarps][32];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, what = blockIdx.y;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int64_t gate = what - 2;
    float* out = what == 0 ? a.dpre : what == 1 ? a.dpost : a.dgate;
    const float* part = what == 0 ? a.part_pre : what == 1 ? a.part_post : a.part_s + gate * a.cuts * a.p.dim;
    const int count = what < 2 ? a.parts : a.cuts;
    if (out == nullptr) return;
    float v = 0.f;
    if (e < a.p.dim) {
#pragma unroll 8
        for (int k = warp; k < count; k += kJoinWarps) v += part[k * a.p.dim + e];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || e >= a.p.dim) return;
    for (int w = 1; w < kJoinWarps; ++w) v += s[w][lane];
    if (what >= 2) {
        out += gate * a.p.dim;
        if (a.p.post != nullptr)
            v *= a.p.param_dtype == MO_F32 ? static_cast<const float*>(a.p.post)[e]
                                           : __bfloat162float(static_cast<const bf16*>(a.p.post)[e]);
    }
    out[e] = (a.accumulate ? out[e] : 0.f) + v;
}

// Blocks with sums of their own.
int64_t grad_blocks(int64_t n) { return n < kSms ? n : kSms; }

// At most kThreads to a block.
template <typename X, typename S, int K, int kMode, int L, int kThreads>
cudaError_t launch_grad(GradArgs& a, cudaStream_t s) {
    static SmemAllowed allowed;
    a.shape = norm_shape(a.p.dim, K, L, kMode == kWide, kThreads, op_ceil_div(a.p.n, kSms),
                         {a.p.x_dtype, a.p.stream_dtype, a.p.stream_dtype, a.p.x_dtype},
                         {true, a.p.pre != nullptr, a.dy != nullptr, a.p.pre != nullptr});
    auto kernel = norm_grad_kernel<X, S, K, kMode, L, kThreads>;
    const cudaError_t e = allowed.allow(kernel, kNormSmem);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(a.parts), a.shape.threads * a.shape.teams, a.shape.smem(), s>>>(a);
    return cudaGetLastError();
}

// f(columns of a thread, lanes of a row (32: warps), threads of a block), of these forms, which hold
// their values in registers:
//   8 columns, 512 threads (128 registers)     short rows: least of their lanes is empty
//   16 columns, 384 threads (168)              up to 6144 columns
//   16 columns, 512 threads (128)              longer rows, in spite of spilling
// Rows of 67 million values, bf16 with a float32 stream, in us: 1024 columns 191, 211, 246; 2048 191, 211,
// 255; 3000 227, 199, 326; 4096 214, 192, 237; 5120 -, 196, 287.  All bf16 (pieces of eight, few spills):
// 512 columns 149, 151, 154; 1024 155, 137, 147; 2048 163, 141, 153; and 4096, where 512 threads have two
// rows and 384 only one, 190, 169, 155.  These rows lie on 16-byte boundaries; off them the all-bf16 rule holds,
// too: 4001 columns -, 310, 292; 3500 -, 345, 343.
template <typename X, typename S, typename F>
cudaError_t with_columns(int64_t dim, F&& f) {
    constexpr bool kSmall = sizeof(X) + sizeof(S) == 4;
    std::integral_constant<int, 8> k8, l8;
    std::integral_constant<int, 16> k16, l16;
    std::integral_constant<int, 32> l32;
    std::integral_constant<int, 384> t384;
    std::integral_constant<int, 512> t512;
    if (dim <= 64) return f(k8, l8, t512);
    if (dim <= 128) return f(k8, l16, t512);
    if (dim <= (kSmall ? 512 : 2048)) return f(k8, l32, t512);
    const bool two = dim <= 256 * 16 && dim > 192 * 16;
    if (dim <= 384 * 16 && !(kSmall && two)) return f(k16, l32, t384);
    return f(k16, l32, t512);
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int block_norm_grad_workspace_bytes(int64_t n, int64_t dim, int64_t gates, size_t* bytes_out) {
    if (n < 0 || dim < 0 || gates < 0 || bytes_out == nullptr) return MO_ERR_INVALID_ARG;
    if (n > INT32_MAX || dim > kMaxNormDim || gates > INT32_MAX) return MO_ERR_UNSUPPORTED;
    const size_t part = op_align_up(static_cast<size_t>(grad_blocks(n)) * static_cast<size_t>(dim) * 4, 256);
    *bytes_out = part > 0 ? (gates > 0 ? 3 : 2) * part : 256;
    return MO_OK;
}

int block_norm_grad(const mo_block_norm* p, const void* y, int64_t ldy, const void* dy, int64_t lddy, const void* dh,
                    int64_t lddh, void* dx, int64_t lddx, void* dresidual, int64_t lddr, float* dpost, float* dgate,
                    float* dpre, int accumulate, void* ws, size_t ws_bytes, mo_stream_t stream) {
    int st = check_norm(p, true);
    if (st != MO_OK) return st;
    if ((accumulate != 0 && accumulate != 1) || (p->n > 0 && (p->pre != nullptr) != (dh != nullptr)) ||
        (p->pre == nullptr && dpre != nullptr) || (p->post == nullptr && dpost != nullptr) ||
        (p->gate == nullptr && dgate != nullptr))
        return MO_ERR_INVALID_ARG;
    if (p->dim == 0) return MO_OK;
    if (p->n > 0) {
        if (dx == nullptr || lddx < p->dim || (dy != nullptr && lddy < p->dim) ||
            (p->pre != nullptr && (y == nullptr || ldy < p->dim || lddh < p->dim)) ||
            (dresidual != nullptr && lddr < p->dim) || (dresidual != nullptr && dresidual == dy && lddr != lddy) ||
            (dx == p->x && lddx != p->ldx) || (dx == dh && dh != nullptr && lddx != lddh))
            return MO_ERR_INVALID_ARG;
        const size_t xs = op_elem_size(p->x_dtype), ss = op_elem_size(p->stream_dtype);
        if (!op_aligned(dx, xs) || !op_aligned(dy, ss) || !op_aligned(y, ss) || !op_aligned(dresidual, ss) ||
            !op_aligned(dh, xs))
            return MO_ERR_ALIGNMENT;
    }
    if (!op_aligned(dpost, 4) || !op_aligned(dgate, 4) || !op_aligned(dpre, 4)) return MO_ERR_ALIGNMENT;
    GradArgs a = {};
    a.p = *p;
    if (a.p.rows_per_gate > p->n) a.p.rows_per_gate = p->n > 0 ? p->n : 1;               // (one gate for all rows)
    a.gates = p->gate != nullptr ? op_ceil_div(p->n, a.p.rows_per_gate) : 1;
    size_t need = 0;
    if ((st = block_norm_grad_workspace_bytes(p->n, p->dim, p->gate != nullptr ? a.gates : 0, &need)) != MO_OK) return st;
    if ((st = op_check_ws(ws, ws_bytes, need)) != MO_OK) return st;
    const int64_t most = grad_blocks(p->n);
    a.cuts = a.gates > 0 && most > a.gates ? static_cast<int>(most / a.gates) : 1;
    a.units = p->n > 0 ? a.gates * a.cuts : 0;
    a.parts = static_cast<int>(a.units < most ? a.units : most);
    a.accumulate = accumulate;
    a.y = y;
    a.ldy = ldy;
    a.dy = dy;
    a.lddy = lddy;
    a.dh = dh;
    a.lddh = lddh;
    a.dx = dx;
    a.lddx = lddx;
    a.dres = dresidual;
    a.lddr = lddr;
    a.dpost = dpost;
    a.dgate = dgate;
    a.dpre = dpre;
    const size_t part = op_align_up(static_cast<size_t>(most) * static_cast<size_t>(p->dim) * 4, 256);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.part_post = reinterpret_cast<float*>(base);
    a.part_pre = reinterpret_cast<float*>(base + part);
    a.part_s = reinterpret_cast<float*>(base + 2 * part);
    const bool wide = norm_row_aligned(p->x, p->ldx, p->x_dtype) && norm_row_aligned(dx, lddx, p->x_dtype) &&
                      (dy == nullptr || norm_row_aligned(dy, lddy, p->stream_dtype)) &&
                      (dresidual == nullptr || norm_row_aligned(dresidual, lddr, p->stream_dtype)) &&
                      (p->pre == nullptr || (norm_row_aligned(y, ldy, p->stream_dtype) && norm_row_aligned(dh, lddh, p->x_dtype)));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_NORM_GRAD, s, [&] {
        cudaError_t e = cudaSuccess;
        if (a.units > 0) {
            e = norm_with_types(*p, [&](auto xt, auto st) {
                using X = decltype(xt);
                using S = decltype(st);
                return with_columns<X, S>(p->dim, [&](auto k, auto lanes, auto threads) {
                    constexpr int K = decltype(k)::value, L = decltype(lanes)::value, kThreads = decltype(threads)::value;
                    return wide ? launch_grad<X, S, K, kWide, L, kThreads>(a, s) : launch_grad<X, S, K, kNarrow, L, kThreads>(a, s);
                });
            });
            if (e != cudaSuccess) return e;
        }
        const bool join_gate = dgate != nullptr && a.units > 0 && a.cuts > 1;
        if (dpre == nullptr && dpost == nullptr && !join_gate) return cudaSuccess;
        const dim3 grid(static_cast<unsigned>(op_ceil_div(p->dim, 32)), join_gate ? 2 + static_cast<unsigned>(a.gates) : 2);
        if (a.units > 0) return launch_after(norm_join_kernel, grid, 32 * kJoinWarps, s, a);
        norm_join_kernel<<<grid, 32 * kJoinWarps, 0, s>>>(a);
        return cudaGetLastError();
    }));
}

}  // extern "C"
