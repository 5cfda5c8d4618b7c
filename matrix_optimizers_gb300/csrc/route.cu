// Routing of rows to experts: per row the softmax p over the experts and its
// `top` largest logits; over all rows the experts' counts and offsets, each
// choice's place among the rows sorted by (expert, row), and the balance and z
// losses; and the gradient by the logits.
//
// A group of G lanes owns a row, each lane V logits, which stay in registers: the
// softmax and the choices both come from there.
//
// The sort is a counting sort that needs no atomic whose order matters: rows are
// cut into chunks of 32 to 128, a block per chunk, and a bit for each (expert, row)
// of the chunk is set in shared memory.  The count of the bits below a row's own is
// its rank within the chunk; the counts of whole chunks are summed over the chunks
// by a second kernel and added by a third.  A single chunk is finished by the first.
#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

constexpr int kMaxExperts = 1024, kMaxRouteTop = 32;
constexpr int kRouteThreads = 256, kRouteWarps = kRouteThreads / 32;
constexpr int kPerThread = kMaxExperts / kRouteThreads;      // experts per thread in the scans
constexpr unsigned kFull = 0xffffffffu;

struct RouteArgs {
    const void* logits;
    const uint8_t* mask;
    int64_t n, ldl;
    int experts, top, renormalise, rows, words, wide, chunks;   // rows of a chunk, and their 32-bit words
    int32_t *idx, *pos, *order, *offsets, *counts;
    float *gates, *loss;
    int32_t* hist;        // [chunks][experts]: counts of each chunk, then those of the chunks before it
    float* part_p;        // [chunks][experts]: sums of p
    int32_t* total;       // [experts]
    float* sum_p;         // [experts]
    float* part_z;        // [chunks]
    int32_t* part_rows;   // [chunks]
};

// Order-preserving image of a logit: larger key, larger logit; -0 ties with +0.  -inf and NaN
// have the smallest key and are never chosen.
constexpr int kNone = static_cast<int>(0x807FFFFFu);
__device__ __forceinline__ int logit_key(float x) {
    const int u = __float_as_int(fmaxf(x + 0.0f, -INFINITY));
    return u ^ ((u >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_logit(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

template <int G>
__device__ __forceinline__ int group_max(int v) {
    if (G == 32) return __reduce_max_sync(kFull, v);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ int group_min(int v) {
    if (G == 32) return __reduce_min_sync(kFull, v);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// exp(x - top) for x <= top; below 2^-126 it is 0.
__device__ __forceinline__ float exp_below(float x, float top) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((x - top) * 1.44269504088896341f));
    return e;
}
// The largest of a lane's logits, NaN left aside.
template <int V>
__device__ __forceinline__ float lane_top(const float (&x)[V]) {
    float top = fmaxf(x[0], -INFINITY);
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
    return top;
}

// The experts of a lane: runs of W neighbours (16 bytes, or all V), the group's lanes side by side.
template <typename T, int G, int V>
struct Lay {
    static constexpr int W = V < Elem<T>::kVec ? V : Elem<T>::kVec;
    __device__ __forceinline__ static int expert(int sub, int i) { return i / W * (G * W) + sub * W + i % W; }
    // where a value of expert e lies in a row of floats whose lanes' own are G apart (no bank conflicts)
    __device__ __forceinline__ static int place(int e) { return (e / (G * W) * W + e % W) * G + e / W % G; }
};

// A lane's logits; those past the last expert are -inf.
template <typename T, int G, int V>
__device__ __forceinline__ void load_logits(const T* row, int sub, int experts, bool wide, float (&x)[V]) {
    constexpr int W = Lay<T, G, V>::W;
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
        const int c = Lay<T, G, V>::expert(sub, q * W);
        if (wide && c + W <= experts) {
            if constexpr (W * sizeof(T) == 16) {
                float w[W];
                unpack16(*reinterpret_cast<const uint4*>(row + c), w);
#pragma unroll
                for (int i = 0; i < W; ++i) x[q * W + i] = w[i];
            } else {                                                    // four bf16
                const uint2 u = *reinterpret_cast<const uint2*>(row + c);
                x[0] = __uint_as_float(u.x << 16);
                x[1] = __uint_as_float(u.x & 0xFFFF0000u);
                x[2] = __uint_as_float(u.y << 16);
                x[3] = __uint_as_float(u.y & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) x[q * W + i] = c + i < experts ? Elem<T>::to_float(row[c + i]) : -INFINITY;
        }
    }
}

// Sum over the block's threads, the same on every thread and in every run.
template <typename S>
__device__ S block_sum(S v, S* red) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    S sum = 0;
    for (int w = 0; w < kRouteWarps; ++w) sum += red[w];
    return sum;
}

// start[e] = sum of count[0 .. e - 1]; returns the sum of all.
__device__ int scan_counts(const int* count, int* start, int experts, int* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = threadIdx.x * kPerThread;
    int v[kPerThread], own = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        v[i] = e0 + i < experts ? count[e0 + i] : 0;
        own += v[i];
    }
    int below = own;
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFull, below, o);
        if (lane >= o) below += t;
    }
    __syncthreads();
    if (lane == 31) red[warp] = below;
    __syncthreads();
    int all = 0, base = below - own;
    for (int w = 0; w < kRouteWarps; ++w) {
        if (w < warp) base += red[w];
        all += red[w];
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (e0 + i < experts) start[e0 + i] = base;
        base += v[i];
    }
    __syncthreads();
    return all;
}

// What one block writes for all chunks: counts, offsets and the losses.
__device__ void finish_route(const RouteArgs& a, const int* count, const int* start, int all, const float* sum_p, float z,
                             int rows, float* red) {
    float dot = 0.f;
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
        a.counts[e] = count[e];
        a.offsets[e] = start[e];
        if (a.loss != nullptr) dot += static_cast<float>(count[e]) * sum_p[e];
    }
    if (threadIdx.x == 0) {
        a.counts[a.experts] = rows;
        a.offsets[a.experts] = all;
    }
    if (a.loss != nullptr) {
        dot = block_sum(dot, red);
        if (threadIdx.x == 0) {
            const float r = static_cast<float>(rows > 0 ? rows : 1);
            a.loss[0] = static_cast<float>(a.experts) / static_cast<float>(a.top) * (dot / r / r);
            a.loss[1] = z / r;
        }
    }
}

// What a group notes of its row's choices: in shared memory, by the row's place r in the chunk.
struct Choices {
    uint32_t* bits;       // [experts][words]
    float* value;         // [rows][top]: gates
    int16_t* idx;         // [rows][top]
    int top, words;
    __device__ __forceinline__ void note(int r, int j, int expert, float v) const {
        atomicOr(&bits[expert * words + (r >> 5)], 1u << (r & 31));
        idx[r * top + j] = static_cast<int16_t>(expert);
        value[r * top + j] = v;
    }
};
struct RowTop {
    float top, inv;       // the row's largest logit, 1 / sum of exp(logit - top)
    int renormalise;
};

// The largest `top` logits of the group, one a round, of equals the lowest expert.
template <typename T, int G, int V>
__device__ __forceinline__ void choose_in_rounds(const float (&x)[V], const Choices& c, int r, bool there, int sub,
                                                 const RowTop& t) {
    int key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = logit_key(x[i]);
    float chosen = 0.f;
    for (int j = 0; j < c.top; ++j) {
        int best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        const int k = group_max<G>(best);
        const float e = k != kNone ? exp_below(key_logit(k), t.top) : 0.f;
        chosen += e;
        int at = V;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == k) at = i;
        const int mine = at < V ? Lay<T, G, V>::expert(sub, at) : INT32_MAX;
        const int expert = group_min<G>(mine);
        if (mine == expert && k != kNone) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) key[i] = kNone;
            if (there) c.note(r, j, expert, e);
        }
        if (k == kNone && there && sub == 0) {
            c.idx[r * c.top + j] = -1;
            c.value[r * c.top + j] = 0.f;
        }
    }
    __syncwarp();
    const float scale = t.renormalise ? 1.f / chosen : t.inv;
    if (there) {
        for (int j = sub; j < c.top; j += G) {
            const int at = r * c.top + j;
            if (c.idx[at] >= 0) c.value[at] *= scale;
        }
    }
}

// The group's values in descending order, one to a lane (a bitonic network).
template <int G>
__device__ __forceinline__ float sorted_lanes(float v, int sub) {
#pragma unroll
    for (int size = 2; size <= G; size *= 2)
#pragma unroll
        for (int stride = size / 2; stride > 0; stride /= 2) {
            const float other = __shfl_xor_sync(kFull, v, stride);
            const bool larger = ((sub & size) == 0) == ((sub & stride) == 0);            // keeps the larger of the two
            v = larger ? fmaxf(v, other) : fminf(v, other);
        }
    return v;
}

// The top-th largest of the group's values: up to eight in a warp by one maximum after the other (equal ones
// go at once, which makes it the smaller), else out of all of them in order (65536 rows of 512 in bf16: 8
// choices 68 us by maxima, 76 in order; 16 choices 103 and 92).
template <int G>
__device__ __forceinline__ float bound_of(float v, int top, int sub, int group) {
    if (G < 32 || top > 8) return __shfl_sync(kFull, sorted_lanes<G>(v, sub), group * G + top - 1);
    int key = logit_key(v), most = kNone;
    for (int j = 0; j < top; ++j) {
        most = __reduce_max_sync(kFull, key);
        if (key == most) key = kNone;
    }
    return key_logit(most);
}

// The same as choose_in_rounds for up to G choices without rounds over all logits: the top-th largest of the
// lanes' maxima is a bound that at least `top` logits reach and few others do (8 choices of 16 lanes: 10.6 on
// average if the logits are in random order); those that reach it are gathered, one to a lane, and each counts
// the ones before it.  8 of 128 experts for 65536 rows: 37 us forward, 55 by rounds.
//
// gather: `count` of them in `list`; false if a group has more than G, as with many equal logits, or fewer
// than `top` lanes that hold anything.
template <typename T, int G, int V>
__device__ __forceinline__ bool gather(const float (&x)[V], float lane_best, int top, bool live, int sub, int group,
                                       uint64_t* list, int& count) {
    const float least = bound_of<G>(lane_best, top, sub, group);
    const unsigned group_mask = kFull >> (32 - G), below = (1u << sub) - 1;
    count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const unsigned who = (__ballot_sync(kFull, x[i] >= least) >> (group * G)) & group_mask;
        const int at = count + __popc(who & below);
        if (x[i] >= least && at < G)
            list[at] = static_cast<uint64_t>(__float_as_uint(x[i])) << 32 | static_cast<uint32_t>(Lay<T, G, V>::expert(sub, i));
        count += __popc(who);
    }
    const bool good = !__any_sync(kFull, live && (count > G || least == -INFINITY));
    if (!live) count = 0;
    __syncwarp();
    return good;
}
// Notes the `top` first of those.  A row that goes nowhere is noted as such.
template <int G>
__device__ __forceinline__ void choose_from(uint64_t* list, int count, const Choices& c, int r, bool there, bool live, int sub,
                                            const RowTop& t) {
    uint64_t own = 0;
    float value = 0.f;
    int expert = 0;
    if (sub < count) {                               // as one number: the logit's key, then the lowest expert first
        own = list[sub];
        value = __uint_as_float(static_cast<uint32_t>(own >> 32));
        expert = static_cast<int>(static_cast<uint32_t>(own));
        own = static_cast<uint64_t>(static_cast<uint32_t>(logit_key(value)) ^ 0x80000000u) << 32 |
              static_cast<uint32_t>(kMaxExperts - expert);
    }
    list[sub] = own;                                 // (0 past the last: before none)
    __syncwarp();
    int rank = 0;
    const int most = __reduce_max_sync(kFull, count);
    for (int k = 0; k < most; k += 2) {
        const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(list + k);
        rank += (p.x > own) + (p.y > own);
    }
    const bool chosen = sub < count && rank < c.top;
    const float e = chosen ? exp_below(value, t.top) : 0.f;
    const float scale = t.renormalise ? 1.f / group_sum<G>(e) : t.inv;
    if (chosen) c.note(r, rank, expert, e * scale);
    if (there && !live) {
        for (int j = sub; j < c.top; j += G) {
            c.idx[r * c.top + j] = -1;
            c.value[r * c.top + j] = 0.f;
        }
    }
    __syncwarp();                                    // (the list is the next row's, too)
}

// Blocks on an SM: as many as spill little (65536 float32 rows, 8 of 1024: 107 us with two, 157 with one, 159
// with three; of 512 68 us with four, 77 with three; of 256 48 with four, 52 with five, and the gradient 29 and 49).
template <int V>
constexpr int kRouteResident = V <= 16 ? 4 : 2;

template <typename T, int G, int V>
__global__ void __launch_bounds__(kRouteThreads, kRouteResident<V>) route_kernel(RouteArgs a) {
    extern __shared__ uint32_t smem[];
    const int rows_here = a.rows;
    __shared__ __align__(16) uint64_t s_list[kRouteWarps][32];
    uint32_t* bits = smem;                                              // [experts][words]
    float* s_gate = reinterpret_cast<float*>(bits + a.experts * a.words);   // [rows][top]
    float* s_p = s_gate + rows_here * a.top;                            // [experts]
    int* s_count = reinterpret_cast<int*>(s_p + a.experts);             // [experts]
    int* s_start = s_count + a.experts;                                 // [experts]
    int16_t* s_idx = reinterpret_cast<int16_t*>(s_start + a.experts);   // [rows][top]
    __shared__ float red[kRouteWarps];
    __shared__ int red_i[kRouteWarps];
    launch_dependents();

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (G - 1), group = lane / G;
    constexpr int kGroups = 32 / G;                                     // rows of a warp at a time
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_here;
    const int rows = static_cast<int>(min(static_cast<int64_t>(rows_here), a.n - row0));
    const Choices choices = {bits, s_gate, s_idx, a.top, a.words};
    auto load = [&](int r, float (&x)[V]) {                             // -inf for a row that is left out
        if (r < rows && (a.mask == nullptr || a.mask[row0 + r] != 0)) {
            load_logits<T, G, V>(static_cast<const T*>(a.logits) + (row0 + r) * a.ldl, sub, a.experts, a.wide, x);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
    };
    for (int i = threadIdx.x; i < a.experts * a.words; i += kRouteThreads) bits[i] = 0;
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) s_p[e] = 0.f;
    __syncthreads();

    float acc[V] = {}, z = 0.f;
    int live_rows = 0;
    for (int r0 = warp * kGroups; r0 < rows; r0 += kRouteWarps * kGroups) {
        const int r = r0 + group;                                       // within the chunk
        float x[V];
        load(r, x);
        const float lane_best = lane_top<V>(x), found = key_logit(group_max<G>(logit_key(lane_best)));
        const bool live = found > -INFINITY;
        const float top = live ? found : 0.f;                           // (0: the exponentials of such a row are 0)
        int count = 0;
        uint64_t* list = s_list[warp] + group * G;
        const bool gathered = G >= 16 && a.top <= G && gather<T, G, V>(x, lane_best, a.top, live, sub, group, list, count);
        float own[V], sum = 0.f;                                        // (own: in x's registers where that has been used up)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            own[i] = exp_below(x[i], top);
            sum += own[i];
        }
        sum = group_sum<G>(sum);
        const float inv = live ? __fdividef(1.f, sum) : 0.f;            // (sum from 1 to 1024)
        const RowTop t = {top, inv, a.renormalise};
        if (gathered)
            choose_from<G>(list, count, choices, r, r < rows, live, sub, t);
        else
            choose_in_rounds<T, G, V>(x, choices, r, r < rows, sub, t);
        if (live) {
            if (a.loss != nullptr) {
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += own[i] * inv;
                const float lse = top + __logf(sum);
                if (sub == 0) z += lse * lse;
            }
            if (sub == 0) ++live_rows;
        }
    }
    if (a.loss != nullptr) {                                            // sums of p over the chunk, warp after warp
#pragma unroll
        for (int i = 0; i < V; ++i)
            for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
        const int busy = min(kRouteWarps, (rows + kGroups - 1) / kGroups);
        for (int w = 0; w < busy; ++w) {
            if (w == warp && group == 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = Lay<T, G, V>::expert(sub, i);
                    if (e < a.experts) s_p[e] += acc[i];
                }
            }
            __syncthreads();
        }
        z = block_sum(z, red);
    }
    const int chunk_rows = block_sum(live_rows, red_i);                 // (its barriers end the choices, too)
    const bool single = gridDim.x == 1;
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
        int c = 0;
        for (int w = 0; w < a.words; ++w) c += __popc(bits[e * a.words + w]);
        if (single) {
            s_count[e] = c;
        } else {
            a.hist[static_cast<int64_t>(blockIdx.x) * a.experts + e] = c;
            if (a.loss != nullptr) a.part_p[static_cast<int64_t>(blockIdx.x) * a.experts + e] = s_p[e];
        }
    }
    __syncthreads();
    int all = 0;
    if (single) {
        all = scan_counts(s_count, s_start, a.experts, red_i);
        finish_route(a, s_count, s_start, all, s_p, z, chunk_rows, red);
        if (a.order != nullptr)
            for (int64_t i = all + threadIdx.x; i < a.n * a.top; i += kRouteThreads) a.order[i] = -1;
    } else if (threadIdx.x == 0) {
        a.part_z[blockIdx.x] = z;
        a.part_rows[blockIdx.x] = chunk_rows;
    }
    const int items = rows * a.top;
    for (int i = threadIdx.x; i < items; i += kRouteThreads) {
        const int e = s_idx[i], r = i / a.top;
        int rank = -1;
        if (e >= 0) {
            const uint32_t* b = bits + e * a.words;
            rank = __popc(b[r >> 5] & ((1u << (r & 31)) - 1));
            for (int w = 0; w < (r >> 5); ++w) rank += __popc(b[w]);
            if (single) {
                rank += s_start[e];
                if (a.order != nullptr) a.order[rank] = r;
            }
        }
        const int64_t to = row0 * a.top + i;
        a.idx[to] = e;
        a.gates[to] = s_gate[i];
        a.pos[to] = rank;
    }
}

// Per expert: the chunks' counts become those of the chunks before, and totals.  A
// block takes 32 experts, its warps a span of the chunks each.
constexpr int kScanWarps = 32, kScanHeld = 19;      // the counts of 608 chunks are held in registers
__global__ void __launch_bounds__(32 * kScanWarps) route_scan_kernel(RouteArgs a) {
    __shared__ int s_c[kScanWarps][33];
    __shared__ float s_p[kScanWarps][33];
    launch_dependents();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int span = (a.chunks + kScanWarps - 1) / kScanWarps;
    const int c0 = min(warp * span, a.chunks), c1 = min(c0 + span, a.chunks);
    const bool loss = a.loss != nullptr, there = e < a.experts;
    int32_t* h = a.hist + static_cast<int64_t>(c0) * a.experts + e;
    const float* q = a.part_p + static_cast<int64_t>(c0) * a.experts + e;
    int first[kScanHeld], count = 0;                                   // counts of the span's first chunks
    float p = 0.f;
#pragma unroll
    for (int k = 0; k < kScanHeld; ++k) {
        const bool in = there && c0 + k < c1;
        first[k] = in ? h[static_cast<int64_t>(k) * a.experts] : 0;
        p += in && loss ? q[static_cast<int64_t>(k) * a.experts] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kScanHeld; ++k) count += first[k];
    if (there) {
#pragma unroll 4
        for (int c = c0 + kScanHeld; c < c1; ++c) {
            count += h[static_cast<int64_t>(c - c0) * a.experts];
            if (loss) p += q[static_cast<int64_t>(c - c0) * a.experts];
        }
    }
    s_c[warp][lane] = count;
    s_p[warp][lane] = p;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_c[w][lane];
    if (!there) return;
    if (warp == kScanWarps - 1) {
        float all = 0.f;
        for (int w = 0; w < kScanWarps; ++w) all += s_p[w][lane];
        a.total[e] = before + count;
        a.sum_p[e] = all;
    }
#pragma unroll
    for (int k = 0; k < kScanHeld; ++k) {
        if (c0 + k < c1) h[static_cast<int64_t>(k) * a.experts] = before;
        before += first[k];
    }
#pragma unroll 4
    for (int c = c0 + kScanHeld; c < c1; ++c) {
        const int t = h[static_cast<int64_t>(c - c0) * a.experts];
        h[static_cast<int64_t>(c - c0) * a.experts] = before;
        before += t;
    }
}

// For every expert the counts of all chunks and of those before this block's, and (block 0)
// the sums of p: a warp takes every eighth chunk, its lanes the experts.
__device__ void sum_chunks(const RouteArgs& a, int* count, int* before, float* sum_p) {
    __shared__ int part[2][kRouteWarps][32];
    __shared__ float part_p[kRouteWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool want_p = a.loss != nullptr && blockIdx.x == 0;
    constexpr int kBatch = 12;                        // loads in flight
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        int all = 0, low = 0;
        float p = 0.f;
        for (int c0 = warp; c0 < a.chunks; c0 += kBatch * kRouteWarps) {
            int t[kBatch];
            float q[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int c = c0 + k * kRouteWarps;
                const bool in = c < a.chunks && e < a.experts;
                t[k] = in ? a.hist[c * a.experts + e] : 0;
                q[k] = in && want_p ? a.part_p[c * a.experts + e] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                all += t[k];
                low += c0 + k * kRouteWarps < static_cast<int>(blockIdx.x) ? t[k] : 0;
                p += q[k];
            }
        }
        part[0][warp][lane] = all;
        part[1][warp][lane] = low;
        part_p[warp][lane] = p;
        __syncthreads();
        if (warp == 0 && e < a.experts) {
            for (int w = 1; w < kRouteWarps; ++w) {
                all += part[0][w][lane];
                low += part[1][w][lane];
                p += part_p[w][lane];
            }
            count[e] = all;
            before[e] = low;
            sum_p[e] = p;
        }
        __syncthreads();
    }
}

// Ranks within a chunk become places; block 0 writes what concerns all rows.  kScanned: the
// counts were summed over the chunks by route_scan_kernel; else each block sums them itself,
// which saves a launch where they are few (4133 rows over 31 experts, forward and back: 21.7 us
// with the scan, 19.9 without).
constexpr int kPlaceHeld = 4;
// Chunks times experts in full warps: 2 of 8 experts for 8192 rows (128 chunks) 9.7 us, 10.3 with the scan; for
// 16384 11.6 and 11.3, for 65536 21.0 and 15.7.
constexpr int64_t kFewCounts = 1 << 13;
template <bool kScanned>
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(RouteArgs a) {
    __shared__ int s_count[kMaxExperts], s_start[kMaxExperts], s_base[kMaxExperts];
    __shared__ float s_p[kScanned ? 1 : kMaxExperts];
    __shared__ float red[kRouteWarps];
    __shared__ int red_i[kRouteWarps];
    wait_for_previous();
    const int rows_here = a.rows;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_here;
    const int items = static_cast<int>(min(static_cast<int64_t>(rows_here), a.n - row0)) * a.top;
    const int32_t* base = a.hist + static_cast<int64_t>(blockIdx.x) * a.experts;
    int held_e[kPlaceHeld], held_p[kPlaceHeld];                         // the first items, on their way meanwhile
#pragma unroll
    for (int k = 0; k < kPlaceHeld; ++k) {
        const int i = threadIdx.x + k * kRouteThreads;
        held_e[k] = i < items ? a.idx[row0 * a.top + i] : -1;
        held_p[k] = i < items ? a.pos[row0 * a.top + i] : 0;
    }
    if (kScanned) {
        for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
            s_count[e] = a.total[e];
            s_base[e] = base[e];
        }
    } else {
        sum_chunks(a, s_count, s_base, s_p);
    }
    __syncthreads();
    const int all = scan_counts(s_count, s_start, a.experts, red_i);
    auto place = [&](int i, int e, int p) {
        const int64_t at = row0 * a.top + i;
        if (e >= 0) {
            p += s_start[e] + s_base[e];
            a.pos[at] = p;
            if (a.order != nullptr) a.order[p] = static_cast<int32_t>(row0 + i / a.top);
        }
        if (a.order != nullptr && at >= all) a.order[at] = -1;
    };
#pragma unroll
    for (int k = 0; k < kPlaceHeld; ++k)
        if (threadIdx.x + k * kRouteThreads < items) place(threadIdx.x + k * kRouteThreads, held_e[k], held_p[k]);
    for (int i = threadIdx.x + kPlaceHeld * kRouteThreads; i < items; i += kRouteThreads)
        place(i, a.idx[row0 * a.top + i], a.pos[row0 * a.top + i]);
    if (blockIdx.x != 0) return;
    float z = 0.f;
    int rows = 0;
    for (int c = threadIdx.x; c < a.chunks; c += kRouteThreads) {
        if (a.loss != nullptr) z += a.part_z[c];
        rows += a.part_rows[c];
    }
    z = block_sum(z, red);
    rows = block_sum(rows, red_i);
    finish_route(a, s_count, s_start, all, kScanned ? a.sum_p : s_p, z, rows, red);
}

struct RouteGradArgs {
    const void* logits;
    const uint8_t* mask;
    int64_t n, ldl, ldg;
    int experts, top, renormalise, wide, wide_out;
    const int32_t *idx, *counts;
    const float* dgates;
    float balance, z;
    void* grad;
};

// d_e = [chosen: back] + p_e (pull_e - sum p pull) + (2 z / rows) lse p_e
//   renormalised gates g over the chosen:  back = g (dg - sum g dg)
//   otherwise:                             back = g dg, and pull_e includes it: p_e (... - sum g dg)
// with pull_e = balance experts counts[e] / (top rows^2).
template <typename T, typename D, int G, int V>
__global__ void __launch_bounds__(kRouteThreads, kRouteResident<V>) route_grad_kernel(RouteGradArgs a) {
    __shared__ __align__(16) float s_row[kRouteWarps * 32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (G - 1), group = lane / G;
    constexpr int kGroups = 32 / G;
    using L = Lay<T, G, V>;
    float* row_of = s_row + (warp * kGroups + group) * (G * V);         // a value for each expert: exps, then gradients
    const int rows = a.counts[a.experts];
    const float r = static_cast<float>(rows > 0 ? rows : 1);
    float pull[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = L::expert(sub, i);
        const float load = e < a.experts ? static_cast<float>(a.counts[e]) / (static_cast<float>(a.top) * r) : 0.f;
        pull[i] = a.balance != 0.f ? a.balance * static_cast<float>(a.experts) / r * load : 0.f;
    }
    const float zc = 2.f * a.z / r;
    const bool given = a.dgates != nullptr;
    // a row's logits, and of its choices those j = sub, sub + G, ... the first
    auto load = [&](int64_t row, float (&x)[V], int& e, float& dg) {
        const bool there = row < a.n && (a.mask == nullptr || a.mask[row] != 0);
        if (there) {
            load_logits<T, G, V>(static_cast<const T*>(a.logits) + row * a.ldl, sub, a.experts, a.wide, x);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
        const bool choice = there && given && sub < a.top;
        e = choice ? a.idx[row * a.top + sub] : -1;
        dg = choice ? a.dgates[row * a.top + sub] : 0.f;
        if (e >= a.experts) e = -1;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * kGroups;
    int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * kGroups;
    constexpr bool kAhead = V <= 8;                                     // the next row is on its way
    float ahead[V], dg_ahead;
    int e_ahead;
    if (kAhead) load(row0 + group, ahead, e_ahead, dg_ahead);
    for (; row0 < a.n; row0 += step) {
        const int64_t row = row0 + group;
        if (!kAhead) load(row, ahead, e_ahead, dg_ahead);
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = ahead[i];
        const int first = e_ahead;
        const float dg_first = dg_ahead;
        if (kAhead) load(row + step, ahead, e_ahead, dg_ahead);
        const float found = key_logit(group_max<G>(logit_key(lane_top<V>(x))));
        const bool live = found > -INFINITY;
        const float top = live ? found : 0.f;                            // (0: the exponentials of such a row are 0)
        float sum = 0.f, mean = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = exp_below(x[i], top);
            sum += x[i];
            mean += x[i] * pull[i];
            row_of[i * G + sub] = x[i];
        }
        __syncwarp();
        // f(expert, its exp, its dgate) for this lane's choices
        const float v_first = first >= 0 ? row_of[L::place(first)] : 0.f;
        const T* logits = static_cast<const T*>(a.logits) + row * a.ldl;
        auto for_choices = [&](auto&& f) {
            if (first >= 0) f(first, v_first, dg_first);
            if (!live || !given) return;
            for (int j = sub + G; j < a.top; j += G) {
                const int e = a.idx[row * a.top + j];
                if (e >= 0 && e < a.experts) f(e, exp_below(Elem<T>::to_float(logits[e]), top), a.dgates[row * a.top + j]);
            }
        };
        float part = 0.f, part_d = 0.f;                                  // sums of e and e dgate over the chosen
        for_choices([&](int, float v, float dg) {
            part += v;
            part_d += v * dg;
        });
        sum = group_sum<G>(sum);
        mean = group_sum<G>(mean);
        part = group_sum<G>(part);
        part_d = group_sum<G>(part_d);
        const float inv = live ? __fdividef(1.f, sum) : 0.f;             // (sum from 1 to 1024)
        const float scale = a.renormalise ? (part > 0.f ? 1.f / part : 0.f) : inv;
        const float gd = part_d * scale;                                 // sum of gate * dgate
        const float less = a.renormalise ? gd : 0.f;
        float flat = -mean * inv - (a.renormalise ? 0.f : gd);
        if (a.z != 0.f) flat += zc * (top + __logf(sum));
        // the chosen's own parts find their lanes by way of the row in shared memory
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; ++i) row_of[i * G + sub] = 0.f;
        __syncwarp();
        if (live) for_choices([&](int e, float v, float dg) { row_of[L::place(e)] = v * scale * (dg - less); });
        __syncwarp();
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = live ? row_of[i * G + sub] + x[i] * inv * (pull[i] + flat) : 0.f;
        if (row < a.n) {
            D* out = static_cast<D*>(a.grad) + row * a.ldg;
#pragma unroll
            for (int q = 0; q < V / L::W; ++q) {
                const int c = L::expert(sub, q * L::W);
                float w[L::W];
#pragma unroll
                for (int i = 0; i < L::W; ++i) w[i] = d[q * L::W + i];
                if (a.wide_out && c + L::W <= a.experts) {
                    store_run<D, L::W>(out + c, w, true);
                } else {
#pragma unroll
                    for (int i = 0; i < L::W; ++i)
                        if (c + i < a.experts) out[c + i] = Elem<D>::from_float(w[i]);
                }
            }
        }
    }
}

int check_route(const mo_route* r) {
    if (r == nullptr || r->n < 0 || r->experts < 1 || r->top < 1 || r->top > r->experts || r->ldl < r->experts ||
        !op_valid_dtype(r->logits_dtype) || (r->renormalise != 0 && r->renormalise != 1) ||
        (r->n > 0 && r->logits == nullptr))
        return MO_ERR_INVALID_ARG;
    if (r->experts > kMaxExperts || r->top > kMaxRouteTop || r->n >= (int64_t(1) << 31) ||
        r->n * r->top >= (int64_t(1) << 31) - 512)
        return MO_ERR_UNSUPPORTED;
    if (!op_aligned(r->logits, op_elem_size(r->logits_dtype))) return MO_ERR_ALIGNMENT;
    return MO_OK;
}

struct RouteLayout {
    size_t hist, part_p, total, sum_p, part_z, part_rows, bytes;
    int rows, words, chunks;
};

// As many chunks as blocks of up to 512 experts fit on a whole GB300 at once (four on each of 152 SMs; with more
// experts two fit, and the chunks take two turns), of 32 to 128 rows, and of no fewer than a block takes at a time
// (64 with up to 32 experts): 65536 rows of 256 in 586 chunks of 112 take 48 us, in 512 of 128 52 us; of 1024
// 107 and 116 us.  A constant, as the workspace's size is asked for without a device.
constexpr int64_t kMostChunks = 4 * 152;
RouteLayout route_layout(int64_t n, int experts) {
    RouteLayout L;
    const int64_t rows = op_ceil_div(op_ceil_div(n, kMostChunks), kRouteWarps) * kRouteWarps;
    const int64_t least = experts <= 32 ? 64 : 32;
    L.rows = static_cast<int>(rows < least ? least : rows > 128 ? 128 : rows);
    L.words = (L.rows + 31) / 32;
    const int64_t chunks = n > 0 ? op_ceil_div(n, L.rows) : 1;
    L.chunks = static_cast<int>(chunks);
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = op_align_up(o + bytes, 256); return at; };
    const size_t c = static_cast<size_t>(chunks), e = static_cast<size_t>(experts);
    L.hist = take(c * e * 4);
    L.part_p = take(c * e * 4);
    L.total = take(e * 4);
    L.sum_p = take(e * 4);
    L.part_z = take(c * 4);
    L.part_rows = take(c * 4);
    L.bytes = o;
    return L;
}

// (G, V) by the number of experts: eight rows to a warp up to 32 experts, two up to 128, else one.  Two
// rows of 256 to a warp are slower (65536 rows: 52 us forward and 33 back, 48 and 29 with one).
// warps: also up to 128 experts, for choices that half a warp seldom has gathered room for and that are few
// among the experts (12 of 64 for 65536 rows 50 us, 64 with two rows to a warp; 16 of 128 52, 107; but 8 of 128
// 41, 37, and 16 of 64 103, 78).
template <typename F>
cudaError_t with_shape(int experts, bool warps, F&& f) {
    if (experts <= 32) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
    if (experts <= 128 && warps) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
    if (experts <= 64) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    if (experts <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
    if (experts <= 256) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 8>());
    if (experts <= 512) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}

size_t route_smem(const RouteArgs& a) {
    return static_cast<size_t>(a.experts) * (a.words + 3) * 4 + static_cast<size_t>(a.rows) * a.top * 6;
}
// experts * 7 + 128 rows of 32 choices: 28 + 24 KB at most
constexpr size_t kRouteSmemMax = kMaxExperts * 7 * 4 + 128 * kMaxRouteTop * 6;

template <typename T>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    cudaError_t err = with_shape(a.experts, a.top > 8 && a.top * 5 <= a.experts, [&](auto g, auto v) {
        auto kernel = route_kernel<T, decltype(g)::value, decltype(v)::value>;
        static SmemAllowed allowed;                                     // (one for each kernel)
        const size_t smem = route_smem(a);
        if (smem > 40 * 1024) {                                         // 48 KB without asking, static arrays among them
            const cudaError_t e = allowed.allow(kernel, static_cast<int>(kRouteSmemMax));
            if (e != cudaSuccess) return e;
        }
        kernel<<<a.chunks, kRouteThreads, smem, s>>>(a);
        return cudaGetLastError();
    });
    if (err != cudaSuccess || a.chunks == 1) return err;
    if (static_cast<int64_t>(a.chunks) * op_align_up(a.experts, 32) <= kFewCounts)
        return launch_after(route_place_kernel<false>, static_cast<unsigned>(a.chunks), kRouteThreads, s, a);
    err = launch_after(route_scan_kernel, static_cast<unsigned>(op_ceil_div(a.experts, 32)), 32 * kScanWarps, s, a);
    if (err != cudaSuccess) return err;
    return launch_after(route_place_kernel<true>, static_cast<unsigned>(a.chunks), kRouteThreads, s, a);
}

template <typename T, typename D>
cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t s) {
    return with_shape(a.experts, false, [&](auto g, auto v) {
        constexpr int kG = decltype(g)::value;
        const int64_t blocks = op_ceil_div(a.n, kRouteWarps * (32 / kG));
        const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
        route_grad_kernel<T, D, kG, decltype(v)::value>
            <<<static_cast<unsigned>(blocks < most ? blocks : most), kRouteThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int expert_route_workspace_bytes(int64_t n, int experts, int top, size_t* bytes_out) {
    if (bytes_out == nullptr) return MO_ERR_INVALID_ARG;
    mo_route r = {};
    r.n = n;
    r.ldl = r.experts = experts;
    r.top = top;
    r.logits = &r;                                   // (its own checks come with the call)
    const int st = check_route(&r);
    if (st != MO_OK) return st;
    *bytes_out = route_layout(n, experts).bytes;
    return MO_OK;
}

int expert_route(const mo_route* r, int32_t* idx, float* gates, int32_t* pos, int32_t* order, int32_t* offsets,
                 int32_t* counts, float* loss, void* ws, size_t ws_bytes, mo_stream_t stream) {
    int st = check_route(r);
    if (st != MO_OK) return st;
    if (offsets == nullptr || counts == nullptr || (r->n > 0 && (idx == nullptr || gates == nullptr || pos == nullptr)))
        return MO_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(idx), static_cast<const void*>(gates), static_cast<const void*>(pos),
                          static_cast<const void*>(order), static_cast<const void*>(offsets),
                          static_cast<const void*>(counts), static_cast<const void*>(loss)})
        if (!op_aligned(p, 4)) return MO_ERR_ALIGNMENT;
    const RouteLayout L = route_layout(r->n, r->experts);
    if ((st = op_check_ws(ws, ws_bytes, L.bytes)) != MO_OK) return st;
    uint8_t* base = static_cast<uint8_t*>(ws);
    RouteArgs a = {};
    a.logits = r->logits;
    a.mask = r->mask;
    a.n = r->n;
    a.ldl = r->ldl;
    a.experts = r->experts;
    a.top = r->top;
    a.renormalise = r->renormalise;
    a.rows = L.rows;
    a.words = L.words;
    a.chunks = L.chunks;
    a.wide = op_aligned(r->logits, 16) && (r->ldl * op_elem_size(r->logits_dtype)) % 16 == 0;
    a.idx = idx;
    a.pos = pos;
    a.order = order;
    a.offsets = offsets;
    a.counts = counts;
    a.gates = gates;
    a.loss = loss;
    a.hist = reinterpret_cast<int32_t*>(base + L.hist);
    a.part_p = reinterpret_cast<float*>(base + L.part_p);
    a.total = reinterpret_cast<int32_t*>(base + L.total);
    a.sum_p = reinterpret_cast<float*>(base + L.sum_p);
    a.part_z = reinterpret_cast<float*>(base + L.part_z);
    a.part_rows = reinterpret_cast<int32_t*>(base + L.part_rows);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_ROUTE, s, [&] {
        return r->logits_dtype == MO_F32 ? launch_route<float>(a, s) : launch_route<bf16>(a, s);
    }));
}

int expert_route_grad(const mo_route* r, const int32_t* idx, const int32_t* counts, const float* dgates,
                      float balance_coef, float z_coef, void* dlogits, int g_dtype, int64_t ldg, mo_stream_t stream) {
    const int st = check_route(r);
    if (st != MO_OK) return st;
    if (!op_valid_dtype(g_dtype) || ldg < r->experts) return MO_ERR_INVALID_ARG;
    if (r->n == 0) return MO_OK;
    if (idx == nullptr || counts == nullptr || dlogits == nullptr) return MO_ERR_INVALID_ARG;
    if (dlogits == r->logits && (g_dtype != r->logits_dtype || ldg != r->ldl)) return MO_ERR_INVALID_ARG;
    if (!op_aligned(idx, 4) || !op_aligned(counts, 4) || !op_aligned(dgates, 4) ||
        !op_aligned(dlogits, op_elem_size(g_dtype)))
        return MO_ERR_ALIGNMENT;
    RouteGradArgs a = {};
    a.logits = r->logits;
    a.mask = r->mask;
    a.n = r->n;
    a.ldl = r->ldl;
    a.ldg = ldg;
    a.experts = r->experts;
    a.top = r->top;
    a.renormalise = r->renormalise;
    a.wide = op_aligned(r->logits, 16) && (r->ldl * op_elem_size(r->logits_dtype)) % 16 == 0;
    a.wide_out = op_aligned(dlogits, 16) && (ldg * op_elem_size(g_dtype)) % 16 == 0;
    a.idx = idx;
    a.counts = counts;
    a.dgates = dgates;
    a.balance = balance_coef;
    a.z = z_coef;
    a.grad = dlogits;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_ROUTE_GRAD, s, [&] {
        if (r->logits_dtype == MO_F32)
            return g_dtype == MO_F32 ? launch_route_grad<float, float>(a, s) : launch_route_grad<float, bf16>(a, s);
        return g_dtype == MO_F32 ? launch_route_grad<bf16, float>(a, s) : launch_route_grad<bf16, bf16>(a, s);
    }));
}

}  // extern "C"
