// Embedding lookup and its dense gradient.
//
//   out[i, :] = s * W[id_i, :]                       (lookup)
//   dW[v, :]  = s * sum_{i : id_i = v} dY[i, :]      (gradient, in the order of i)
//
// Both only move bytes: the lookup reads each row it needs and writes n rows;
// the gradient reads dY once and writes the whole table once.
//
// The gradient sorts the positions by token (a stable radix sort, so that a
// row's sum runs in the order of i on every call) and reduces the sorted list
// in chunks of kChunk positions: a chunk's threads walk its positions, each
// thread holding 16 bytes of columns, and write a token's row when its run
// ends inside the chunk.  A run that crosses chunks leaves float32 partial
// rows, which the block of the chunk where the run starts adds up in order.
// Equal chunks keep the work balanced when a few tokens make up most of a batch,
// as they do in text.
#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

// ------------------------------------------------------------------- lookup
constexpr int kLookupThreads = 256;

// One 16-byte (or, where a row is not 16-byte aligned, one-element) piece per
// thread and step; consecutive threads take consecutive pieces of a row.
template <typename W, typename O>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const W* __restrict__ w, int64_t vocab, int64_t dim, int64_t ldw, const void* __restrict__ ids,
              int id_dtype, int64_t n, float scale, O* __restrict__ out, int64_t ldo, int wide) {
    constexpr int V = Elem<W>::kVec;
    const int64_t groups = (dim + V - 1) / V;
    const int64_t total = n * groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLookupThreads;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x; t < total; t += step) {
        const int64_t i = t / groups, c = (t - i * groups) * V;
        const int64_t id = load_id(ids, id_dtype, i, vocab);
        const W* src = w + id * ldw + c;
        O* dst = out + i * ldo + c;
        const int nv = static_cast<int>(dim - c < V ? dim - c : V);
        if (nv == V) {
            float v[V];
            if (id < 0) {
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = 0.f;
            } else if (wide) {
                unpack16(__ldg(reinterpret_cast<const uint4*>(src)), v);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = Elem<W>::to_float(src[k]);
            }
            // a padding row is +0 whatever the scale
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = id < 0 ? 0.f : v[k] * scale;
            store_run<O, V>(dst, v, wide);
        } else {
            for (int k = 0; k < nv; ++k)
                dst[k] = Elem<O>::from_float(id < 0 ? 0.f : Elem<W>::to_float(src[k]) * scale);
        }
    }
}

template <typename W, typename O>
cudaError_t launch_lookup(const void* w, int64_t vocab, int64_t dim, int64_t ldw, const void* ids, int id_dtype,
                          int64_t n, float scale, void* out, int64_t ldo, cudaStream_t s) {
    constexpr int V = Elem<W>::kVec;
    const bool wide = op_aligned(w, 16) && (ldw * sizeof(W)) % 16 == 0 && op_aligned(out, V * sizeof(O) < 16 ? 8 : 16) &&
                      (ldo * sizeof(O)) % (V * sizeof(O) < 16 ? 8 : 16) == 0;
    const int64_t blocks = op_ceil_div(n * op_ceil_div(dim, V), kLookupThreads);
    const int grid = static_cast<int>(blocks < 32768 ? blocks : 32768);
    lookup_kernel<W, O><<<grid, kLookupThreads, 0, s>>>(static_cast<const W*>(w), vocab, dim, ldw, ids, id_dtype, n,
                                                        scale, static_cast<O*>(out), ldo, wide);
    return cudaGetLastError();
}

// ------------------------------------------------ stable radix sort by token
// Keys 0 .. vocab - 1, and vocab for a dropped position, in passes of at most
// kDigitBits bits.  A pass counts the digits of each tile of positions, then
// each tile finds where its digits start (all smaller digits of all tiles,
// plus equal digits of earlier tiles) and scatters in order.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

struct SortPass {
    const void* ids;           // the first pass reads the ids, later ones keys_in / pos_in
    int id_dtype;
    const uint32_t* keys_in;
    const uint32_t* pos_in;
    uint32_t* keys_out;
    uint32_t* pos_out;
    uint32_t* counts;          // [tiles][digits]
    int64_t n, vocab;
    int shift, digits, tiles, rounds;   // a tile holds rounds * kSortThreads positions
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, int64_t i) {
    if (p.keys_in != nullptr) return p.keys_in[i];
    const int64_t id = load_id(p.ids, p.id_dtype, i, p.vocab);
    return static_cast<uint32_t>(id < 0 ? p.vocab : id);
}

// Warp w of a tile takes its positions [w * rounds * 32, (w + 1) * rounds * 32),
// 32 at a time, so that position order is warp order, then round, then lane.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortPass p) {
    __shared__ uint32_t hist[kDigits];
    for (int d = threadIdx.x; d < p.digits; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * p.rounds * kSortThreads;
    for (int r = 0; r < p.rounds; ++r) {
        const int64_t i = tile0 + static_cast<int64_t>(r) * kSortThreads + threadIdx.x;
        if (i < p.n) atomicAdd(&hist[(sort_key(p, i) >> p.shift) & (p.digits - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.digits; d += kSortThreads)
        p.counts[static_cast<int64_t>(blockIdx.x) * p.digits + d] = hist[d];
}

__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const __grid_constant__ SortPass p) {
    __shared__ uint32_t hist[kSortWarps][kDigits];   // per warp: digits seen, then where the warp's next one goes
    __shared__ uint32_t base[kDigits];
    __shared__ uint32_t warp_total[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int d = threadIdx.x; d < kSortWarps * kDigits; d += kSortThreads) (&hist[0][0])[d] = 0;
    // where this tile's digit d starts
    uint32_t before = 0, total = 0;
    if (static_cast<int>(threadIdx.x) < p.digits) {
        for (int t = 0; t < p.tiles; ++t) {
            const uint32_t c = p.counts[static_cast<int64_t>(t) * p.digits + threadIdx.x];
            if (t < static_cast<int>(blockIdx.x)) before += c;
            total += c;
        }
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    uint32_t off = 0;
    for (int w = 0; w < warp; ++w) off += warp_total[w];
    base[threadIdx.x] = off + incl - total + before;

    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.rounds * kSortThreads +
                          static_cast<int64_t>(warp) * p.rounds * 32 + lane;
    for (int r = 0; r < p.rounds; ++r) {
        const int64_t i = first + r * 32;
        if (i < p.n) atomicAdd(&hist[warp][(sort_key(p, i) >> p.shift) & (p.digits - 1)], 1u);
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.digits) {
        uint32_t run = base[threadIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = hist[w][threadIdx.x];
            hist[w][threadIdx.x] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int r = 0; r < p.rounds; ++r) {
        const int64_t i = first + r * 32;
        const bool in = i < p.n;
        const uint32_t key = in ? sort_key(p, i) : 0;
        const uint32_t d = in ? (key >> p.shift) & (p.digits - 1) : 0xffffffffu;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const uint32_t rank = __popc(same & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (in) at = hist[warp][d] + rank;
        __syncwarp();
        if (in && rank == 0) hist[warp][d] += __popc(same);
        __syncwarp();
        if (in) {
            p.keys_out[at] = key;
            p.pos_out[at] = p.pos_in != nullptr ? p.pos_in[i] : static_cast<uint32_t>(i);
        }
    }
}

// -------------------------------------------------------- sums of sorted runs
constexpr int kChunk = 64;            // sorted positions per block
constexpr int kGradThreads = 128;     // columns per block: 128 x one 16-byte access
constexpr int kZeroRows = 64;         // table rows per block of the zero fill
constexpr int kAhead = 8;             // rows in flight per thread

struct GradArgs {
    const void* dy;
    int64_t ldy, n, vocab, dim;
    const uint32_t* keys;             // sorted, n
    const uint32_t* pos;
    void* dw;
    int64_t ldw;
    float* part;                      // [chunk][2][dim]: a run's rows in a chunk it enters from before, or leaves
    float scale;
    int accumulate, wide_in, wide_out;
    int64_t chunks, sum_blocks;       // sum_blocks = chunks * column slabs; zero-fill blocks follow
};

template <typename D, int V>
__device__ __forceinline__ void write_row(const GradArgs& a, uint32_t key, int64_t c, int nv, float (&v)[V]) {
    D* dst = static_cast<D*>(a.dw) + static_cast<int64_t>(key) * a.ldw + c;
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] *= a.scale;
    if (a.accumulate) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < nv) v[k] += Elem<D>::to_float(dst[k]);
    }
    if (nv == V) {
        store_run<D, V>(dst, v, a.wide_out);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < nv) dst[k] = Elem<D>::from_float(v[k]);
    }
}

// First sorted position whose key is not below v.
__device__ __forceinline__ int64_t lower_bound_key(const uint32_t* keys, int64_t n, int64_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}

template <typename T, typename D>
__global__ void __launch_bounds__(kGradThreads) grad_sum_kernel(const __grid_constant__ GradArgs a) {
    constexpr int V = Elem<T>::kVec;
    if (blockIdx.x >= a.sum_blocks) {                // rows of absent tokens: zeros
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - a.sum_blocks) * kZeroRows;
        __shared__ uint8_t present[kZeroRows];
        for (int r = threadIdx.x; r < kZeroRows; r += kGradThreads) {
            const int64_t v = r0 + r;
            uint8_t is = 1;
            if (v < a.vocab) {
                const int64_t at = lower_bound_key(a.keys, a.n, v);
                is = at < a.n && a.keys[at] == v;
            }
            present[r] = is;
        }
        __syncthreads();
        constexpr int Z = Elem<D>::kVec;
        for (int r = 0; r < kZeroRows; ++r) {
            if (present[r]) continue;
            D* row = static_cast<D*>(a.dw) + (r0 + r) * a.ldw;
            if (a.wide_out) {
                int64_t c = static_cast<int64_t>(threadIdx.x) * Z;
                for (; c + Z <= a.dim; c += kGradThreads * Z)
                    *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
                for (; c < a.dim; ++c) row[c] = Elem<D>::from_float(0.f);
            } else {
                for (int64_t c = threadIdx.x; c < a.dim; c += kGradThreads) row[c] = Elem<D>::from_float(0.f);
            }
        }
        return;
    }
    __shared__ uint32_t skey[kChunk + 2], spos[kChunk];      // skey[0], skey[len + 1]: the neighbours' keys
    const int64_t chunk = blockIdx.x % a.chunks, slab = blockIdx.x / a.chunks;
    const int64_t p0 = chunk * kChunk;
    const int len = static_cast<int>(a.n - p0 < kChunk ? a.n - p0 : kChunk);
    const uint32_t none = 0xffffffffu, dropped = static_cast<uint32_t>(a.vocab);
    for (int i = threadIdx.x; i < len + 2; i += kGradThreads) {
        const int64_t q = p0 + i - 1;
        skey[i] = q >= 0 && q < a.n ? a.keys[q] : none;
    }
    for (int i = threadIdx.x; i < len; i += kGradThreads) spos[i] = a.pos[p0 + i];
    __syncthreads();
    const int64_t c = (slab * kGradThreads + threadIdx.x) * V;
    if (c >= a.dim) return;
    const int nv = static_cast<int>(a.dim - c < V ? a.dim - c : V);
    const T* dy = static_cast<const T*>(a.dy) + c;
    const bool wide = a.wide_in && nv == V;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    bool from_before = skey[0] == skey[1];
    for (int i0 = 0; i0 < len; i0 += kAhead) {
        float v[kAhead][V];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            const bool on = i < len && skey[i + 1] != dropped;
            const T* src = dy + static_cast<int64_t>(on ? spos[i] : 0) * a.ldy;
            if (on && wide) {
                unpack16(__ldg(reinterpret_cast<const uint4*>(src)), v[u]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) v[u][k] = on && k < nv ? Elem<T>::to_float(src[k]) : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= len || skey[i + 1] == dropped) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += v[u][k];
            const bool last = i + 1 == len;
            if (!last && skey[i + 2] == skey[i + 1]) continue;
            const bool goes_on = last && skey[i + 2] == skey[i + 1];
            if (from_before || goes_on) {
                // slot 0: the run entered from before (and perhaps goes on); slot 1: it starts here and goes on
                float* dst = a.part + ((chunk * 2 + (from_before ? 0 : 1)) * a.dim + c);
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k < nv) dst[k] = acc[k];
            } else {
                write_row<D, V>(a, skey[i + 1], c, nv, acc);
            }
            from_before = false;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
        }
    }
}

// The block of a chunk whose last run goes on adds that run's partial rows, in order.
template <typename T, typename D>
__global__ void __launch_bounds__(kGradThreads) grad_join_kernel(const __grid_constant__ GradArgs a) {
    const int64_t chunk = blockIdx.x, next = (chunk + 1) * kChunk;
    if (next >= a.n) return;
    const uint32_t key = a.keys[next - 1];
    if (key == static_cast<uint32_t>(a.vocab) || a.keys[next] != key) return;
    if (chunk > 0 && a.keys[chunk * kChunk] == key && a.keys[chunk * kChunk - 1] == key) return;   // an earlier chunk's run
    const int64_t end = lower_bound_key(a.keys, a.n, static_cast<int64_t>(key) + 1);   // one past the run
    const int64_t last = (end - 1) / kChunk;
    for (int64_t c = static_cast<int64_t>(blockIdx.y) * kGradThreads + threadIdx.x; c < a.dim;
         c += static_cast<int64_t>(gridDim.y) * kGradThreads) {
        float acc = a.part[(chunk * 2 + 1) * a.dim + c];
        for (int64_t q = chunk + 1; q <= last; q += kAhead) {
            float v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) v[u] = q + u <= last ? a.part[(q + u) * 2 * a.dim + c] : 0.f;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) acc += v[u];
        }
        float one[1] = {acc};
        write_row<D, 1>(a, key, c, 1, one);
    }
}

struct GradLayout {
    size_t keys[2], pos[2], counts, part, total;
    int64_t chunks;
    int passes, digit_bits, tiles, rounds;
};

GradLayout grad_layout(int64_t n, int64_t vocab, int64_t dim) {
    GradLayout L;
    int bits = 1;
    while ((int64_t(1) << bits) <= vocab) ++bits;    // keys 0 .. vocab
    L.passes = (bits + kDigitBits - 1) / kDigitBits;
    L.digit_bits = (bits + L.passes - 1) / L.passes;
    // at most 128 tiles, so that finding the digits' starts stays short
    L.rounds = 2;
    while (op_ceil_div(n, static_cast<int64_t>(L.rounds) * kSortThreads) > 128) L.rounds *= 2;
    L.tiles = static_cast<int>(op_ceil_div(n, static_cast<int64_t>(L.rounds) * kSortThreads));
    L.chunks = op_ceil_div(n, kChunk);
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = op_align_up(o + bytes, 256); return at; };
    for (int k = 0; k < 2; ++k) L.keys[k] = take(static_cast<size_t>(n) * 4);
    for (int k = 0; k < 2; ++k) L.pos[k] = take(static_cast<size_t>(n) * 4);
    L.counts = take((static_cast<size_t>(L.tiles) << L.digit_bits) * 4);
    L.part = take(static_cast<size_t>(L.chunks) * 2 * static_cast<size_t>(dim) * 4);
    L.total = o > 256 ? o : 256;
    return L;
}

template <typename T, typename D>
cudaError_t launch_grad(const GradArgs& a0, cudaStream_t s) {
    GradArgs a = a0;
    constexpr int V = Elem<T>::kVec;
    a.wide_in = op_aligned(a.dy, 16) && (a.ldy * sizeof(T)) % 16 == 0;
    a.wide_out = op_aligned(a.dw, 16) && (a.ldw * sizeof(D)) % 16 == 0;
    const int64_t slabs = op_ceil_div(a.dim, static_cast<int64_t>(kGradThreads) * V);
    a.sum_blocks = a.chunks * slabs;
    const int64_t zero_blocks = a.accumulate ? 0 : op_ceil_div(a.vocab, kZeroRows);
    if (a.sum_blocks + zero_blocks > 0) {
        grad_sum_kernel<T, D><<<static_cast<unsigned>(a.sum_blocks + zero_blocks), kGradThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.chunks > 1) {
        const int64_t by = op_ceil_div(a.dim, kGradThreads);
        grad_join_kernel<T, D><<<dim3(static_cast<unsigned>(a.chunks), static_cast<unsigned>(by < 64 ? by : 64)),
                                 kGradThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxDim = int64_t(1) << 24;

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int embedding_lookup(const void* W, int w_dtype, int64_t vocab, int64_t dim, int64_t ldw, const void* ids,
                     int id_dtype, int64_t n, float scale, void* out, int out_dtype, int64_t ldo,
                     mo_stream_t stream) {
    if (!op_valid_dtype(w_dtype) || !op_valid_dtype(out_dtype) || !op_valid_id_dtype(id_dtype) || vocab < 0 ||
        dim < 0 || n < 0)
        return MO_ERR_INVALID_ARG;
    if (n == 0 || dim == 0) return MO_OK;
    if (out == nullptr || ids == nullptr || (vocab > 0 && W == nullptr) || ldw < dim || ldo < dim)
        return MO_ERR_INVALID_ARG;
    if (vocab > kMaxCount || n > kMaxCount || dim > kMaxDim) return MO_ERR_UNSUPPORTED;
    if (!op_aligned(W, op_elem_size(w_dtype)) || !op_aligned(out, op_elem_size(out_dtype)) ||
        !op_aligned(ids, op_id_size(id_dtype)))
        return MO_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_EMBED, s, [&] {
        auto go = [&](auto w, auto o) {
            return launch_lookup<decltype(w), decltype(o)>(W, vocab, dim, ldw, ids, id_dtype, n, scale, out, ldo, s);
        };
        if (w_dtype == MO_F32) return out_dtype == MO_F32 ? go(float(), float()) : go(float(), bf16());
        return out_dtype == MO_F32 ? go(bf16(), float()) : go(bf16(), bf16());
    }));
}

int embedding_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim, size_t* bytes_out) {
    if (n < 0 || vocab < 0 || dim < 0 || bytes_out == nullptr) return MO_ERR_INVALID_ARG;
    if (vocab >= kMaxCount || n > kMaxCount || dim > kMaxDim) return MO_ERR_UNSUPPORTED;
    // one block for each chunk and column slab, and for each kZeroRows rows: a grid's limit
    if (op_ceil_div(n, kChunk) * op_ceil_div(dim, kGradThreads * 4) + op_ceil_div(vocab, kZeroRows) > kMaxCount)
        return MO_ERR_UNSUPPORTED;
    *bytes_out = grad_layout(n, vocab, dim).total;
    return MO_OK;
}

int embedding_grad(const void* dY, int dy_dtype, int64_t n, int64_t dim, int64_t ldy, const void* ids, int id_dtype,
                   int64_t vocab, float scale, void* dW, int dw_dtype, int64_t ldw, int accumulate, void* ws,
                   size_t ws_bytes, mo_stream_t stream) {
    if (!op_valid_dtype(dy_dtype) || !op_valid_dtype(dw_dtype) || !op_valid_id_dtype(id_dtype) || vocab < 0 ||
        dim < 0 || n < 0 || (accumulate != 0 && accumulate != 1))
        return MO_ERR_INVALID_ARG;
    if (vocab == 0 || dim == 0) return MO_OK;
    if (dW == nullptr || ldw < dim || (n > 0 && (dY == nullptr || ids == nullptr || ldy < dim)))
        return MO_ERR_INVALID_ARG;
    size_t need = 0;
    int st = embedding_grad_workspace_bytes(n, vocab, dim, &need);
    if (st != MO_OK) return st;
    if (!op_aligned(dW, op_elem_size(dw_dtype)) ||
        (n > 0 && (!op_aligned(dY, op_elem_size(dy_dtype)) || !op_aligned(ids, op_id_size(id_dtype)))))
        return MO_ERR_ALIGNMENT;
    if ((st = op_check_ws(ws, ws_bytes, need)) != MO_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const GradLayout L = grad_layout(n, vocab, dim);
    uint8_t* base = static_cast<uint8_t*>(ws);
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(base + L.keys[0]), reinterpret_cast<uint32_t*>(base + L.keys[1])};
    uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(base + L.pos[0]), reinterpret_cast<uint32_t*>(base + L.pos[1])};
    if (n > 0) {
        const cudaError_t e = op_traced(MO_K_EMBED_SORT, s, [&] {
            for (int k = 0; k < L.passes; ++k) {
                SortPass p;
                p.ids = ids;
                p.id_dtype = id_dtype;
                p.keys_in = k == 0 ? nullptr : keys[(k + 1) & 1];
                p.pos_in = k == 0 ? nullptr : pos[(k + 1) & 1];
                p.keys_out = keys[k & 1];
                p.pos_out = pos[k & 1];
                p.counts = reinterpret_cast<uint32_t*>(base + L.counts);
                p.n = n;
                p.vocab = vocab;
                p.shift = k * L.digit_bits;
                p.digits = 1 << L.digit_bits;
                p.tiles = L.tiles;
                p.rounds = L.rounds;
                sort_count_kernel<<<L.tiles, kSortThreads, 0, s>>>(p);
                cudaError_t err = cudaGetLastError();
                if (err != cudaSuccess) return err;
                sort_scatter_kernel<<<L.tiles, kSortThreads, 0, s>>>(p);
                if ((err = cudaGetLastError()) != cudaSuccess) return err;
            }
            return cudaSuccess;
        });
        if (e != cudaSuccess) return MO_ERR_CUDA;
    }
    GradArgs a = {};
    a.dy = dY;
    a.ldy = ldy;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.keys = keys[(L.passes + 1) & 1];
    a.pos = pos[(L.passes + 1) & 1];
    a.dw = dW;
    a.ldw = ldw;
    a.part = reinterpret_cast<float*>(base + L.part);
    a.scale = scale;
    a.accumulate = accumulate;
    a.chunks = L.chunks;
    return op_status(op_traced(MO_K_EMBED_GRAD, s, [&] {
        if (dy_dtype == MO_F32) return dw_dtype == MO_F32 ? launch_grad<float, float>(a, s) : launch_grad<float, bf16>(a, s);
        return dw_dtype == MO_F32 ? launch_grad<bf16, float>(a, s) : launch_grad<bf16, bf16>(a, s);
    }));
}

}  // extern "C"
