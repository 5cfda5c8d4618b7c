// Distillation from a teacher's top logits: per row
//   p = softmax(t / T) over the teacher's present entries,
//   q = softmax(s / T) over the whole vocabulary,
//   loss = w T^2 sum_k p_k (log p_k - log q[idx_k]),
//   d loss / d s_j = g w T (q_j - sum_{k : idx_k = j} p_k).
// A row needs one running maximum and sum over its logits (kept in float32 as
// m = max s and z = sum exp((s - m) / T)); the gradient then is exp again,
// scaled, with the few teacher places corrected afterwards.
//
// The work is the bytes: the loss reads the logits once, the gradient reads and
// writes them once.  Loss and gradient in one call read them twice, but the second
// time from L2: a cluster of CTAs shares a row, so that the rows at work on the
// device (about 230 of 256 KB at 64 KB per CTA) stay there.  Measured for 8192 rows
// of 128000 bf16 (4.2 GB at least): 705 us and 4.1 GB of DRAM traffic; with one CTA
// per row 917 us and 6.3 GB; without the L2 prefetch below 748 us; 32 KB per CTA
// 916 us and 128 KB 958 us.  Rows kept in shared memory (one read, no L2) were slower,
// 1020 us with a kernel per row and 1170 us with rows streamed through a persistent
// cluster: what fits on the chip leaves too few warps to cover a row's chain of
// barriers and small loads.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>

#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;
namespace cg = cooperative_groups;

namespace {

constexpr int kMaxTop = 1024;
constexpr int64_t kMaxVocab = INT32_MAX - 1024;       // a thread's next column, one stride past the last, still fits an int
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kRowAhead = 4;                          // 16-byte pieces in flight per thread
constexpr int kMaxCluster = 8;
// of a row, per CTA, when loss and gradient are wanted.  Rows past eight such slices get larger ones and
// are read again from DRAM in part (2048 float32 rows: 131072 logits 355 us, 6.0 TB/s of their two passes; 200064
// logits 714 us, 4.6 TB/s, and 732 as two calls).
constexpr int64_t kSliceBytes = 65536;

struct DistillArgs {
    mo_distill d;
    float* loss;             // or null
    float* stats_out;        // or null
    const float* stats_in;   // the gradient alone: the loss call's statistics
    void* grad;
    int64_t ldg;
    float c;                 // log2(e) / T
};

// One row's teacher: the places (-1: absent) and probabilities, in shared memory.
struct Teacher {
    int* at;                 // [top]
    float* p;                // [top]
    float* x;                // [top]: the student's logit there, read before any gradient is written
    float* red;              // [kRowWarps + 1]
};

__device__ __forceinline__ float block_max(float v, float* red) {
    v = warp_max(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) r = fmaxf(r, red[w]);
    return r;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) r += red[w];
    return r;
}

// Fills `t` and returns whether any present entry lies above -inf (a NaN
// counts, and spreads).  *log_z is log sum exp((t - max) / T); (t - max) / T is
// log p_k + log_z.  The maximum is taken off before the division, so that logits
// at the type's lowest value stay finite.
__device__ __forceinline__ bool load_teacher(const DistillArgs& a, int64_t row, const Teacher& t) {
    const int top = a.d.top;
    float mx = -INFINITY;
    int live = 0;
    for (int k = threadIdx.x; k < top; k += blockDim.x) {
        const int64_t id = load_id(a.d.idx, a.d.idx_dtype, row * top + k, a.d.vocab);
        const float x = a.d.teacher_dtype == MO_F32
                            ? static_cast<const float*>(a.d.teacher)[row * top + k]
                            : __bfloat162float(static_cast<const bf16*>(a.d.teacher)[row * top + k]);
        const bool on = id >= 0 && x != -INFINITY;
        t.at[k] = on ? static_cast<int>(id) : -1;
        t.p[k] = x;
        if (on) {
            mx = fmaxf(mx, x);
            live = 1;
        }
    }
    live = __syncthreads_or(live);
    if (!live) return false;
    mx = block_max(mx, t.red);
    float z = 0.f;
    for (int k = threadIdx.x; k < top; k += blockDim.x) {
        if (t.at[k] < 0) continue;
        z += exp2f((t.p[k] - mx) * a.c);
    }
    z = block_sum(z, t.red);
    for (int k = threadIdx.x; k < top; k += blockDim.x)
        t.p[k] = t.at[k] < 0 ? 0.f : exp2f((t.p[k] - mx) * a.c) / z;
    __syncthreads();
    return true;
}

// 2^x to about 2^-22 of its value; results below the smallest normal number become 0
// (a probability that small changes no float32 sum and no gradient that is not itself that small).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two float32 operations in one instruction (sm_100 and later).
struct F2 {
    unsigned long long v;
    F2() = default;
    __device__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// The exponent of exp((v - m) / T) in base 2, as one fused v c - b with c =
// log2(e) / T and b = m c rounded: the same b stands in every term of a sum and of a
// quotient, so that its rounding cancels (rho, what b lacks of m c, appears where sums of
// different shifts meet and where the loss needs m itself).  Each term then carries 2^rho, so
// this form is taken only while b's last place is at most 1 and |rho| at most 1/2.  Larger
// products take (v - m) c, whose rounding is relative to the difference: logits near the
// maximum lose nothing.
constexpr float kFusedShift = 16777216.f;              // 2^24
struct Shift {
    float m, c, b;
    bool fused;
    __device__ Shift(float m_, float c_) : m(m_), c(c_), b(m_ * c_), fused(fabsf(m_ * c_) < kFusedShift) {}
    __device__ float operator()(float v) const { return fused ? fmaf(v, c, -b) : (v - m) * c; }
    __device__ float rho() const { return fused ? fmaf(m, c, -b) : 0.f; }
};

// m and z = sum of 2^shift(s) of a run of logits.  m starts at the lowest finite
// value, so that a masked logit (-inf) adds 2^-inf = 0 and no difference of two
// infinities arises; z == 0 marks a row of -inf only, for which q is 0 throughout.
struct MaxSum {
    float m, z;
};
// The factor that takes a sum from maximum `from` to maximum `to` >= from: b minus b,
// which is (from - to) c - rho(from) + rho(to), the form that also holds where only one
// is fused (1% of the batch's time: 698 us without it).
__device__ __forceinline__ float rescale(float from, float to, float c) {
    const Shift x(from, c), y(to, c);
    return exp2_fast(x.fused && y.fused ? x.b - y.b : (from - to) * c - x.rho() + y.rho());
}
__device__ __forceinline__ void add_logit(MaxSum& a, float x, float c) {
    const float m = fmaxf(a.m, x);
    a.z = a.z * rescale(a.m, m, c) + exp2_fast(Shift(m, c)(x));
    a.m = m;
}
__device__ __forceinline__ MaxSum block_join(const MaxSum& a, float c, float* red) {
    MaxSum r;
    r.m = block_max(a.m, red);
    r.z = block_sum(a.z * rescale(a.m, r.m, c), red);
    return r;
}

// Sixteen bytes of logits.
template <typename S>
__device__ __forceinline__ float piece_max(const uint4& u);
template <>
__device__ __forceinline__ float piece_max<float>(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <>
__device__ __forceinline__ float piece_max<bf16>(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
template <typename S>
__device__ __forceinline__ uint4 minus_inf_piece() {
    const uint32_t w = sizeof(S) == 4 ? 0xff800000u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}
// e[k] = 2^shift(logit k)
template <typename S>
__device__ __forceinline__ void piece_exp(const uint4& u, const Shift& sh, F2 (&e)[Elem<S>::kVec / 2]) {
    constexpr int kV = Elem<S>::kVec;
    float v[kV];
    unpack16(u, v);
    if (sh.fused) {
        const F2 c2(sh.c, sh.c), b2(-sh.b, -sh.b);
#pragma unroll
        for (int k = 0; k < kV / 2; ++k) {
            float x, y;
            fma2(F2(v[2 * k], v[2 * k + 1]), c2, b2).get(x, y);
            e[k] = F2(exp2_fast(x), exp2_fast(y));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kV / 2; ++k) e[k] = F2(exp2_fast(sh(v[2 * k])), exp2_fast(sh(v[2 * k + 1])));
    }
}
// Adds n pieces to a: one maximum over all of them, then the terms.
template <typename S, int n>
__device__ __forceinline__ void add_pieces(MaxSum& a, const uint4 (&p)[n], float c) {
    float m = a.m;
#pragma unroll
    for (int i = 0; i < n; ++i) m = fmaxf(m, piece_max<S>(p[i]));
    const Shift sh(m, c);
    F2 z(a.z * rescale(a.m, m, c), 0.f);
#pragma unroll
    for (int i = 0; i < n; ++i) {
        F2 e[Elem<S>::kVec / 2];
        piece_exp<S>(p[i], sh, e);
#pragma unroll
        for (int k = 0; k < Elem<S>::kVec / 2; ++k) z = add2(z, e[k]);
    }
    float x, y;
    z.get(x, y);
    a.m = m;
    a.z = x + y;
}
// The gradient of one piece away from the teacher's places: qs 2^shift(logit).
template <typename S, typename G>
__device__ __forceinline__ void put_piece(const uint4& u, const Shift& sh, float qs, G* g, bool wide) {
    constexpr int kV = Elem<S>::kVec;
    F2 e[kV / 2];
    piece_exp<S>(u, sh, e);
    float v[kV];
    const F2 q2(qs, qs);
#pragma unroll
    for (int k = 0; k < kV / 2; ++k) mul2(e[k], q2).get(v[2 * k], v[2 * k + 1]);
    store_run<G, kV>(g, v, wide);
}

// Logits of [0, vocab) before the first 16-byte boundary.
template <typename S>
__device__ __forceinline__ int row_head(const S* row, int vocab) {
    const int h = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(S));
    return h < vocab ? h : vocab;
}

// The row's loss over T, by the whole block.
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Teacher& t, const MaxSum& st) {
    const Shift sh(st.m, a.c);
    const float log_z = logf(st.z) - sh.rho() * 0.693147180559945f;    // of sum exp((s - m) / T)
    float part = 0.f;
    for (int k = threadIdx.x; k < a.d.top; k += blockDim.x) {
        const float p = t.p[k];
        if (t.at[k] < 0 || p == 0.f) continue;
        // T (log p - log q), with T log q = (x - m) - T log z: finite also where (x - m) / T is not
        part += st.z == 0.f ? INFINITY : p * (a.d.temperature * (logf(p) + log_z) - (t.x[k] - st.m));
    }
    return block_sum(part, t.red);
}

// The gradient at the teacher's places for which mine(place) holds, after the
// block has written the rest.  A place that several entries name is written once,
// by the first of them.  Every entry is compared with every other, which is nothing for the
// few entries a teacher keeps and most of the time for many (2048 rows of 32000 bf16, loss and gradient:
// 64 entries 56 us, 256 84, 1024 636).
template <typename G, typename F>
__device__ __forceinline__ void fix_places(const DistillArgs& a, const Teacher& t, const MaxSum& st, float coef, float inv,
                                           G* g, F&& mine) {
    const Shift sh(st.m, a.c);
    for (int k = threadIdx.x; k < a.d.top; k += blockDim.x) {
        const int at = t.at[k];
        if (at < 0 || !mine(at)) continue;
        float p = 0.f;
        bool first = true;
        for (int q = 0; q < a.d.top; ++q) {
            if (t.at[q] != at) continue;
            if (q < k) first = false;
            p += t.p[q];
        }
        if (first) g[at] = Elem<G>::from_float(coef * (exp2_fast(sh(t.x[k])) * inv - p));
    }
}

// {max s, sum exp((s - max) / T)}, and the z of a MaxSum back from it
__device__ __forceinline__ void put_stats(const DistillArgs& a, int64_t row, const MaxSum& st) {
    if (a.stats_out == nullptr) return;
    a.stats_out[2 * row] = st.m;
    a.stats_out[2 * row + 1] = st.z * exp2f(-Shift(st.m, a.c).rho());
}
__device__ __forceinline__ MaxSum get_stats(const DistillArgs& a, int64_t row) {
    const float m = a.stats_in[2 * row];
    return {m, a.stats_in[2 * row + 1] * exp2f(Shift(m, a.c).rho())};
}

// A row's m and z from its slices' parts, in rank order.
__device__ __forceinline__ MaxSum join_parts(const MaxSum* part, int ctas, float c) {
    MaxSum p[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) p[k] = k < ctas ? part[k] : MaxSum{-FLT_MAX, 0.f};
    MaxSum r = {p[0].m, 0.f};
#pragma unroll
    for (int k = 1; k < kMaxCluster; ++k) r.m = fmaxf(r.m, p[k].m);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) r.z += p[k].z * rescale(p[k].m, r.m, c);
    return r;
}

// A cluster of 1 to 8 CTAs works on a row, a slice of its 16-byte pieces each;
// the slices' parts meet through distributed shared memory, joined in rank order.
template <typename S, typename G, bool kLoss, bool kGrad, bool kSplit>
__global__ void __launch_bounds__(kRowThreads) distill_row_kernel(const __grid_constant__ DistillArgs a, int slice) {
    extern __shared__ float words[];
    __shared__ float red[kRowWarps + 1];
    __shared__ MaxSum part[kMaxCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = kSplit ? static_cast<int>(cluster.num_blocks()) : 1;
    const int rank = kSplit ? static_cast<int>(cluster.block_rank()) : 0;
    if (kSplit) cluster.barrier_arrive();              // (waited for before anything reaches another CTA)
    const int top = a.d.top, V = static_cast<int>(a.d.vocab);
    const Teacher t = {reinterpret_cast<int*>(words), words + top, words + 2 * top, red};
    const int64_t row = blockIdx.x / ctas;
    constexpr int kV = Elem<S>::kVec;
    const S* s = static_cast<const S*>(a.d.logits) + row * a.d.ldl;
    G* g = static_cast<G*>(a.grad) + (kGrad ? row * a.ldg : 0);
    const float w = a.d.row_weight != nullptr ? a.d.row_weight[row] : 1.f;
    const int head = row_head(s, V), nvec = (V - head) / kV, tail = head + nvec * kV;
    const int v0 = min(rank * slice, nvec), count = min(slice, nvec - v0);       // this CTA's pieces
    const int edge0 = rank == 0 ? 0 : head, edge1 = rank == ctas - 1 ? V : tail; // and what lies outside the 16-byte grid
    const uint4* sv = reinterpret_cast<const uint4*>(s + head) + v0;
    if (kLoss && kGrad && w != 0.f) {                   // the slice into L2, ahead of the teacher's chain of small loads
        constexpr int kPart = 512;                      // pieces
        const int j = static_cast<int>(threadIdx.x) * kPart;
        if (j < count)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(sv + j), "r"(min(kPart, count - j) * 16) : "memory");
    }
    const bool live = w != 0.f && load_teacher(a, row, t);                       // the same in every CTA of the cluster
    if (!live) {
        if (kSplit) cluster.barrier_wait();
        if (kLoss && rank == 0 && threadIdx.x == 0) {
            a.loss[row] = 0.f;
            put_stats(a, row, MaxSum{0.f, 1.f});
        }
        if (kGrad) {
            const int from = rank == 0 ? 0 : head + v0 * kV, to = rank == ctas - 1 ? V : head + (v0 + count) * kV;
            for (int j = from + threadIdx.x; j < to; j += kRowThreads) g[j] = Elem<G>::from_float(0.f);
        }
        return;
    }
    for (int k = threadIdx.x; k < top; k += kRowThreads)
        if (t.at[k] >= 0) t.x[k] = Elem<S>::to_float(s[t.at[k]]);
    MaxSum st;
    if (kLoss) {
        MaxSum ms = {-FLT_MAX, 0.f};
        for (int j = edge0 + threadIdx.x; j < head; j += kRowThreads) add_logit(ms, Elem<S>::to_float(s[j]), a.c);
        for (int j = tail + threadIdx.x; j < edge1; j += kRowThreads) add_logit(ms, Elem<S>::to_float(s[j]), a.c);
        for (int j0 = threadIdx.x; j0 < count; j0 += kRowThreads * kRowAhead) {
            uint4 raw[kRowAhead];
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u)        // past the end: -inf, which adds nothing
                raw[u] = j0 + u * kRowThreads < count ? sv[j0 + u * kRowThreads] : minus_inf_piece<S>();
            add_pieces<S>(ms, raw, a.c);
        }
        st = block_join(ms, a.c, red);
        if (kSplit) {
            cluster.barrier_wait();                    // every CTA has started
            if (static_cast<int>(threadIdx.x) < ctas) *cluster.map_shared_rank(&part[rank], threadIdx.x) = st;
            cluster.sync();                            // the parts are here; every x of the row is read
            st = join_parts(part, ctas, a.c);
        }
        if (rank == 0) {
            const float l = row_loss(a, t, st);
            if (threadIdx.x == 0) {
                a.loss[row] = w * a.d.temperature * l;
                put_stats(a, row, st);
            }
        }
    } else {
        st = get_stats(a, row);
        if (kSplit) {
            cluster.barrier_wait();
            cluster.sync();                            // dlogits may be the logits: every x of the row is read
        }
    }
    if (kGrad) {
        const float inv = st.z == 0.f ? 0.f : 1.f / st.z;
        const float coef = a.d.grad_scale * w * a.d.temperature, qs = coef * inv;
        const Shift sh(st.m, a.c);
        __syncthreads();                               // dlogits may be the logits: every x is read before any is written
        for (int j = edge0 + threadIdx.x; j < head; j += kRowThreads)
            g[j] = Elem<G>::from_float(exp2_fast(sh(Elem<S>::to_float(s[j]))) * qs);
        for (int j = tail + threadIdx.x; j < edge1; j += kRowThreads)
            g[j] = Elem<G>::from_float(exp2_fast(sh(Elem<S>::to_float(s[j]))) * qs);
        G* gv = g + head + v0 * kV;
        const bool wide = (reinterpret_cast<uintptr_t>(gv) & 15) == 0;
        for (int j0 = threadIdx.x; j0 < count; j0 += kRowThreads * kRowAhead) {
            uint4 raw[kRowAhead];
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u) raw[u] = sv[min(j0 + u * kRowThreads, count - 1)];
#pragma unroll
            for (int u = 0; u < kRowAhead; ++u) {
                const int j = j0 + u * kRowThreads;
                if (j < count) put_piece<S>(raw[u], sh, qs, gv + j * kV, wide);
            }
        }
        __syncthreads();
        fix_places(a, t, st, coef, inv, g, [&](int at) {
            return (at < head ? 0 : at >= tail ? ctas - 1 : (at - head) / kV / slice) == rank;
        });
    }
}

template <typename S, typename G, bool kLoss, bool kGrad>
cudaError_t launch_rows(const DistillArgs& a, int64_t ctas, cudaStream_t s) {
    const int slice = static_cast<int>(op_ceil_div(op_ceil_div(a.d.vocab, Elem<S>::kVec), ctas));
    const unsigned grid = static_cast<unsigned>(a.d.n * ctas);
    const size_t smem = static_cast<size_t>(a.d.top) * 12;
    if (ctas == 1) {
        distill_row_kernel<S, G, kLoss, kGrad, false><<<grid, kRowThreads, smem, s>>>(a, slice);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, distill_row_kernel<S, G, kLoss, kGrad, true>, a, slice);
}

template <typename S, typename G>
cudaError_t launch_distill(const DistillArgs& a, bool loss, bool grad, cudaStream_t s) {
    const int64_t bytes = a.d.vocab * static_cast<int64_t>(sizeof(S));
    int64_t ctas = 1;
    // loss and gradient: a CTA's share is at most kSliceBytes (while eight CTAs do), so
    // that the rows at work stay in L2 between their two reads
    if (loss && grad) ctas = std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, op_ceil_div(bytes, kSliceBytes)));
    // few rows: more CTAs each, down to 8 KB, so that every SM has some (8 rows of
    // 32000 bf16: 8 CTAs each 9 us, one each 12 us)
    while (ctas * 2 <= kMaxCluster && a.d.n * ctas * 2 <= device_sm_count() && bytes > ctas * 8192) ctas *= 2;
    if (!loss) return launch_rows<S, G, false, true>(a, ctas, s);
    return grad ? launch_rows<S, G, true, true>(a, ctas, s) : launch_rows<S, G, true, false>(a, ctas, s);
}

// MO_OK with *none set when there is nothing to do.
int check_distill(const mo_distill* d, bool* none) {
    if (d == nullptr) return MO_ERR_INVALID_ARG;
    *none = false;
    if (d->n < 0 || d->vocab < 0 || d->top < 1 || !op_valid_dtype(d->logits_dtype) ||
        !op_valid_dtype(d->teacher_dtype) || !op_valid_id_dtype(d->idx_dtype) ||
        !(d->temperature >= FLT_MIN && d->temperature <= FLT_MAX))    // (log2(e) / T overflows for smaller ones)
        return MO_ERR_INVALID_ARG;
    if (d->n == 0) {
        *none = true;
        return MO_OK;
    }
    if ((d->vocab > 0 && d->logits == nullptr) || d->idx == nullptr || d->teacher == nullptr || d->ldl < d->vocab)
        return MO_ERR_INVALID_ARG;
    if (d->top > kMaxTop || d->vocab > kMaxVocab || d->n > INT32_MAX / kMaxCluster) return MO_ERR_UNSUPPORTED;
    if (!op_aligned(d->logits, op_elem_size(d->logits_dtype)) || !op_aligned(d->teacher, op_elem_size(d->teacher_dtype)) ||
        !op_aligned(d->idx, op_id_size(d->idx_dtype)) || !op_aligned(d->row_weight, 4))
        return MO_ERR_ALIGNMENT;
    return MO_OK;
}

int run_distill(const mo_distill* d, float* loss, float* stats_out, const float* stats_in, void* grad, int g_dtype,
                int64_t ldg, bool want_loss, bool want_grad, mo_stream_t stream) {
    bool none = false;
    int st = check_distill(d, &none);
    if (st != MO_OK) return st;
    if (want_grad && !op_valid_dtype(g_dtype)) return MO_ERR_INVALID_ARG;
    if (none) return MO_OK;
    if (want_loss && loss == nullptr) return MO_ERR_INVALID_ARG;
    if (want_grad && ((d->vocab > 0 && grad == nullptr) || ldg < d->vocab)) return MO_ERR_INVALID_ARG;
    // in place: each element is read before it is written only where the two coincide
    if (want_grad && grad == d->logits && d->vocab > 0 && (g_dtype != d->logits_dtype || ldg != d->ldl))
        return MO_ERR_INVALID_ARG;
    if (!op_aligned(loss, 4) || !op_aligned(stats_out, 4) || !op_aligned(stats_in, 4) ||
        (want_grad && !op_aligned(grad, op_elem_size(g_dtype))))
        return MO_ERR_ALIGNMENT;
    DistillArgs a;
    a.d = *d;
    a.loss = loss;
    a.stats_out = stats_out;
    a.stats_in = stats_in;
    a.grad = grad;
    a.ldg = ldg;
    a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(d->temperature));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_DISTILL, s, [&] {
        const bool gf = g_dtype == MO_F32;
        if (d->logits_dtype == MO_F32)
            return gf ? launch_distill<float, float>(a, want_loss, want_grad, s)
                      : launch_distill<float, bf16>(a, want_loss, want_grad, s);
        return gf ? launch_distill<bf16, float>(a, want_loss, want_grad, s)
                  : launch_distill<bf16, bf16>(a, want_loss, want_grad, s);
    }));
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int distill_topk_loss(const mo_distill* d, float* loss, float* stats, mo_stream_t stream) {
    if (d != nullptr && d->n > 0 && stats == nullptr) return MO_ERR_INVALID_ARG;
    return run_distill(d, loss, stats, nullptr, nullptr, MO_F32, 0, true, false, stream);
}

int distill_topk_grad(const mo_distill* d, const float* stats, void* dlogits, int g_dtype, int64_t ldg,
                      mo_stream_t stream) {
    if (d != nullptr && d->n > 0 && stats == nullptr) return MO_ERR_INVALID_ARG;
    return run_distill(d, nullptr, nullptr, stats, dlogits, g_dtype, ldg, false, true, stream);
}

int distill_topk_loss_grad(const mo_distill* d, float* loss, void* dlogits, int g_dtype, int64_t ldg,
                           mo_stream_t stream) {
    return run_distill(d, loss, nullptr, nullptr, dlogits, g_dtype, ldg, true, true, stream);
}

}  // extern "C"
