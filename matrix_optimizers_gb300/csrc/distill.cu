// Distillation from a teacher's top logits: per row
//   p = softmax(t / T) over the teacher's present entries,
//   q = softmax(s / T) over the whole vocabulary,
//   loss = w T^2 sum_k p_k (log p_k - log q[idx_k]),
//   d loss / d s_j = g w T (q_j - sum_{k : idx_k = j} p_k).
// A row needs one running maximum and sum over its logits (kept in float32 as
// m = max s and z = sum exp((s - m) / T)); the gradient then is exp again,
// scaled, with the few teacher places corrected afterwards.
#include <cfloat>

#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

constexpr int kMaxTop = 1024;
constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;

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

// m and z of a run of logits, joined pairwise.  m starts at the lowest finite
// value, so that a masked logit (-inf) adds exp(-inf) = 0 and no difference of
// two infinities arises; z == 0 marks a row of -inf only.
struct MaxSum {
    float m, z;
};
__device__ __forceinline__ MaxSum join(const MaxSum& x, const MaxSum& y, float c) {
    MaxSum r;
    r.m = fmaxf(x.m, y.m);
    r.z = x.z * exp2f((x.m - r.m) * c) + y.z * exp2f((y.m - r.m) * c);
    return r;
}

template <typename S>
__device__ __forceinline__ void add_logit(MaxSum& a, float x, float c) {
    const MaxSum one = {fmaxf(x, -FLT_MAX), x == -INFINITY ? 0.f : (x == x ? 1.f : x)};
    a = join(a, one, c);
}

// Logits of [0, vocab) before the first 16-byte boundary.
template <typename S>
__device__ __forceinline__ int64_t row_head(const S* row, int64_t vocab) {
    const int64_t h = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(S);
    return h < vocab ? h : vocab;
}

template <typename S, typename G, bool kLoss, bool kGrad>
__global__ void __launch_bounds__(kRowThreads) distill_row_kernel(const __grid_constant__ DistillArgs a) {
    extern __shared__ float smem[];
    __shared__ float red[kRowWarps + 1];
    __shared__ MaxSum stat;
    const int top = a.d.top;
    Teacher t = {reinterpret_cast<int*>(smem), smem + top, red};
    float* fix = smem + 2 * top;                       // the corrected gradient of each teacher place
    const int64_t row = blockIdx.x, V = a.d.vocab;
    constexpr int kV = Elem<S>::kVec;
    const S* s = static_cast<const S*>(a.d.logits) + row * a.d.ldl;
    G* g = static_cast<G*>(a.grad) + (kGrad ? row * a.ldg : 0);
    const float w = a.d.row_weight != nullptr ? a.d.row_weight[row] : 1.f;
    const bool live = w != 0.f && load_teacher(a, row, t);
    if (!live) {
        if (kLoss && threadIdx.x == 0) {
            a.loss[row] = 0.f;
            if (a.stats_out != nullptr) {
                a.stats_out[2 * row] = 0.f;
                a.stats_out[2 * row + 1] = 1.f;
            }
        }
        if (kGrad)
            for (int64_t j = threadIdx.x; j < V; j += blockDim.x) g[j] = Elem<G>::from_float(0.f);
        return;
    }
    const int64_t head = row_head(s, V), nvec = (V - head) / kV, tail = head + nvec * kV;
    const uint4* sv = reinterpret_cast<const uint4*>(s + head);
    if (kLoss) {
        MaxSum ms = {-FLT_MAX, 0.f};
        for (int64_t j = threadIdx.x; j < head; j += blockDim.x) add_logit<S>(ms, Elem<S>::to_float(s[j]), a.c);
        for (int64_t j = tail + threadIdx.x; j < V; j += blockDim.x) add_logit<S>(ms, Elem<S>::to_float(s[j]), a.c);
        for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
            float v[kV];
            unpack16(sv[j], v);
            float mx = v[0];
#pragma unroll
            for (int k = 1; k < kV; ++k) mx = fmaxf(mx, v[k]);
            mx = fmaxf(mx, ms.m);
            float z = ms.z * exp2f((ms.m - mx) * a.c);
#pragma unroll
            for (int k = 0; k < kV; ++k) z += exp2f((v[k] - mx) * a.c);
            ms.m = mx;
            ms.z = z;
        }
        const float m = block_max(ms.m, red);
        const float z = block_sum(ms.z * exp2f((ms.m - m) * a.c), red);
        if (threadIdx.x == 0) {
            stat = {m, z};
            if (a.stats_out != nullptr) {
                a.stats_out[2 * row] = m;
                a.stats_out[2 * row + 1] = z;
            }
        }
    } else if (threadIdx.x == 0) {
        stat = {a.stats_in[2 * row], a.stats_in[2 * row + 1]};
    }
    __syncthreads();
    const float m = stat.m, z = stat.z;
    const float inv = z == 0.f ? 0.f : 1.f / z;
    if (kLoss) {
        const float log_z = logf(z);
        float part = 0.f;
        for (int k = threadIdx.x; k < top; k += blockDim.x) {
            const float p = t.p[k];
            if (t.at[k] < 0 || p == 0.f) continue;
            const float x = Elem<S>::to_float(s[t.at[k]]);
            // T (log p - log q), with T log q = (x - m) - T log z: finite also where (x - m) / T is not
            part += z == 0.f ? INFINITY : p * (a.d.temperature * (logf(p) + log_z) - (x - m));
        }
        part = block_sum(part, red);
        if (threadIdx.x == 0) a.loss[row] = w * a.d.temperature * part;
    }
    if (kGrad) {
        const float coef = a.d.grad_scale * w * a.d.temperature;
        // a place that several entries name is corrected once, by the first of them
        for (int k = threadIdx.x; k < top; k += blockDim.x) {
            const int at = t.at[k];
            if (at >= 0) {
                float p = 0.f;
                bool first = true;
                for (int q = 0; q < top; ++q) {
                    if (t.at[q] != at) continue;
                    if (q < k) first = false;
                    p += t.p[q];
                }
                const float x = Elem<S>::to_float(s[at]);
                fix[k] = coef * (exp2f((x - m) * a.c) * inv - p);
                reinterpret_cast<int*>(fix + top)[k] = first ? at : -1;
            } else {
                reinterpret_cast<int*>(fix + top)[k] = -1;
            }
        }
        __syncthreads();                               // dlogits may be the logits: all are read before any is written
        const float qs = coef * inv;
        for (int64_t j = threadIdx.x; j < head; j += blockDim.x)
            g[j] = Elem<G>::from_float(exp2f((Elem<S>::to_float(s[j]) - m) * a.c) * qs);
        for (int64_t j = tail + threadIdx.x; j < V; j += blockDim.x)
            g[j] = Elem<G>::from_float(exp2f((Elem<S>::to_float(s[j]) - m) * a.c) * qs);
        const bool wide = (reinterpret_cast<uintptr_t>(g + head) & 15) == 0;
        for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
            float v[kV];
            unpack16(sv[j], v);
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = exp2f((v[k] - m) * a.c) * qs;
            store_run<G, kV>(g + head + j * kV, v, wide);
        }
        __syncthreads();
        for (int k = threadIdx.x; k < top; k += blockDim.x) {
            const int at = reinterpret_cast<const int*>(fix + top)[k];
            if (at >= 0) g[at] = Elem<G>::from_float(fix[k]);
        }
    }
}

template <typename S, typename G>
cudaError_t launch_distill(const DistillArgs& a, bool loss, bool grad, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(a.d.top) * 16;
    const unsigned grid = static_cast<unsigned>(a.d.n);
    if (loss && grad)
        distill_row_kernel<S, G, true, true><<<grid, kRowThreads, smem, s>>>(a);
    else if (loss)
        distill_row_kernel<S, G, true, false><<<grid, kRowThreads, smem, s>>>(a);
    else
        distill_row_kernel<S, G, false, true><<<grid, kRowThreads, smem, s>>>(a);
    return cudaGetLastError();
}

// MO_OK with *none set when there is nothing to do.
int check_distill(const mo_distill* d, bool* none) {
    if (d == nullptr) return MO_ERR_INVALID_ARG;
    *none = false;
    if (d->n < 0 || d->vocab < 0 || d->top < 1 || !op_valid_dtype(d->logits_dtype) ||
        !op_valid_dtype(d->teacher_dtype) || !op_valid_id_dtype(d->idx_dtype) || !(d->temperature > 0.f) ||
        d->temperature > FLT_MAX)
        return MO_ERR_INVALID_ARG;
    if (d->n == 0) {
        *none = true;
        return MO_OK;
    }
    if ((d->vocab > 0 && d->logits == nullptr) || d->idx == nullptr || d->teacher == nullptr || d->ldl < d->vocab)
        return MO_ERR_INVALID_ARG;
    if (d->top > kMaxTop || d->vocab > INT32_MAX || d->n > INT32_MAX) return MO_ERR_UNSUPPORTED;
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
