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
// in chunks of 8 to 64 positions: a chunk's threads walk its positions, each
// thread holding 16 bytes of columns, and write a token's row when its run
// ends inside the chunk.  A run that crosses chunks leaves float32 partial
// rows, counted as they arrive; the block that brings the last one adds them all up,
// in the chunks' order.
// Equal chunks keep the work balanced when a few tokens make up most of a batch,
// as they do in text.
#include <cooperative_groups.h>

#include <atomic>

#include "train_common.cuh"

namespace mo {

namespace cg = cooperative_groups;

using bf16 = __nv_bfloat16;

namespace {

// ------------------------------------------------------------------- lookup
constexpr int kLookupThreads = 256;

// Eight columns per thread and step, so that a bf16 result leaves in 16-byte
// stores.  A row belongs to 2^row_bits consecutive threads (as many as it has
// such pieces, at most a block), which take its pieces in turn.  kWide: rows start
// on 16-byte boundaries and hold whole pieces, so that a step is loads, multiplies
// and stores alone: with bounds checks in it the instructions, not the bytes, set
// the time (32768 rows of 4096 float32 to bf16 127 us, now 77 us, 79% of the DRAM's
// peak; more rows or pieces in flight per thread cost instructions and were slower).
template <typename W, typename O, bool kWide>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const W* __restrict__ w, int64_t vocab, int dim, int64_t ldw, const void* __restrict__ ids, int id_dtype,
              int64_t n, float scale, O* __restrict__ out, int64_t ldo, int row_bits) {
    constexpr int V = Elem<W>::kVec;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (kLookupThreads >> row_bits) + (threadIdx.x >> row_bits);
    if (i >= n) return;
    const int64_t id = load_id(ids, id_dtype, i, vocab);
    const W* src = w + id * ldw;
    O* dst = out + i * ldo;
    const int step = 8 << row_bits, c0 = static_cast<int>(threadIdx.x & ((1 << row_bits) - 1)) * 8;
    if (id < 0) {                                    // padding: +0 whatever the scale
        for (int c = c0; c < dim; c += step)
            for (int k = 0; k < 8 && c + k < dim; ++k) dst[c + k] = Elem<O>::from_float(0.f);
        return;
    }
    if (kWide) {
#pragma unroll 2
        for (int c = c0; c < dim; c += step) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8 / V; ++q) {
                float x[V];
                unpack16(__ldg(reinterpret_cast<const uint4*>(src + c) + q), x);
#pragma unroll
                for (int k = 0; k < V; ++k) v[q * V + k] = x[k] * scale;
            }
            store_run<O, 8>(dst + c, v, true);
        }
    } else {
        // a thread's eight columns lie apart, so that the row's threads touch neighbours
        // (32768 rows of 4095 float32 to bf16: 166 us, eight in a row 312 us)
        for (int c = c0 / 8; c < dim; c += step) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = c + (k << row_bits);
                if (at < dim) dst[at] = Elem<O>::from_float(Elem<W>::to_float(src[at]) * scale);
            }
        }
    }
}

template <typename W, typename O>
cudaError_t launch_lookup(const void* w, int64_t vocab, int64_t dim, int64_t ldw, const void* ids, int id_dtype,
                          int64_t n, float scale, void* out, int64_t ldo, cudaStream_t s) {
    const bool wide = dim % 8 == 0 && op_aligned(w, 16) && (ldw * sizeof(W)) % 16 == 0 && op_aligned(out, 16) &&
                      (ldo * sizeof(O)) % 16 == 0;
    int row_bits = 0;
    while ((1 << row_bits) < kLookupThreads && (int64_t(8) << row_bits) < dim) ++row_bits;
    const unsigned grid = static_cast<unsigned>(op_ceil_div(n, kLookupThreads >> row_bits));
    auto go = [&](auto kernel) {
        kernel<<<grid, kLookupThreads, 0, s>>>(static_cast<const W*>(w), vocab, static_cast<int>(dim), ldw, ids, id_dtype, n,
                                               scale, static_cast<O*>(out), ldo, row_bits);
        return cudaGetLastError();
    };
    return wide ? go(lookup_kernel<W, O, true>) : go(lookup_kernel<W, O, false>);
}

// ------------------------------------------------ stable radix sort by token
// Keys 0 .. vocab - 1, and vocab for a dropped position, in passes of at most
// kDigitBits bits.  Beyond one cluster's reach (below) a pass counts the digits of each tile of positions, then
// each tile finds where its digits start (all smaller digits of all tiles,
// plus equal digits of earlier tiles) and scatters in order.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

// Every sort also clears the sums' arrival counters (its last step before them in the stream).
__device__ __forceinline__ void clear_counters(uint32_t* arrived, int64_t count) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        arrived[i] = 0;
}

struct SortPass {
    uint32_t* arrived;         // the first pass clears these
    int64_t arrived_count;
    const void* ids;           // the first pass reads the ids, later ones keys_in / pos_in
    int id_dtype;
    const uint32_t* keys_in;
    const uint32_t* pos_in;
    uint32_t* keys_out;
    uint32_t* pos_out;
    uint32_t* counts;          // [tiles][digits]
    int64_t n, vocab;
    int shift, digit_bits, digits, tiles, rounds;   // a tile holds rounds * kSortThreads positions
};

// The lanes with `in` whose digit equals this lane's, by one vote per bit
// (match.any took most of the sort's time).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool in, int bits) {
    uint32_t same = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        const bool set = d >> b & 1u;
        const uint32_t votes = __ballot_sync(0xffffffffu, set);
        if (b < bits) same &= set ? votes : ~votes;
    }
    return same;
}

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, int64_t i) {
    if (p.keys_in != nullptr) return p.keys_in[i];
    const int64_t id = load_id(p.ids, p.id_dtype, i, p.vocab);
    return static_cast<uint32_t>(id < 0 ? p.vocab : id);
}

// Warp w of a tile takes its positions [w * rounds * 32, (w + 1) * rounds * 32),
// 32 at a time, so that position order is warp order, then round, then lane.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortPass p) {
    __shared__ uint32_t hist[kDigits];
    if (p.keys_in == nullptr) clear_counters(p.arrived, p.arrived_count);
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
        const uint32_t d = (key >> p.shift) & (p.digits - 1);
        const uint32_t same = same_digit(d, in, p.digit_bits);
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

// Up to 128 K positions of up to 2^18 - 1 tokens: both passes in one launch of one
// cluster, whose CTAs keep the elements in shared memory and exchange digit counts
// and scattered elements through distributed shared memory.  An element is one
// word, its position with the digit that is still to be sorted by above it; the
// key written out at the end is read again from the ids.  Bound by latency: the
// votes and counter updates of a round, and the scattered words (32768 positions 17 us;
// the passes above 27 us in four launches; 8 CTAs and two words per element 23 us).  From 32768
// positions on a thread holds 4 or 8 of them and spills 20 or 188 bytes of its 64 registers.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;
constexpr int kClusterMax = 16;                      // CTAs of a cluster
constexpr int kClusterRounds = 8;                    // positions per thread, at most
constexpr int kClusterKeys = kClusterThreads * kClusterRounds;
constexpr int kPosBits = 17;
constexpr int64_t kClusterSortMax = static_cast<int64_t>(kClusterMax) * kClusterKeys;
constexpr int64_t kClusterVocabMax = (int64_t(1) << (2 * kDigitBits)) - 1;
static_assert(kClusterSortMax <= (int64_t(1) << kPosBits) && kPosBits + kDigitBits <= 32, "one word per element");

struct ClusterSmem {
    uint32_t elem[kClusterKeys];
    uint16_t hist[kClusterWarps][kDigits];           // digits of each warp, then where the warp's first one goes in the CTA's run
    uint32_t total[kDigits];                         // digits of this CTA
    uint32_t base[kDigits];
    uint32_t scan[kClusterWarps];
};
static_assert(sizeof(ClusterSmem) <= 232448, "shared memory");

template <int kRounds>
__global__ void __launch_bounds__(kClusterThreads, 1)
cluster_sort_kernel(const void* ids, int id_dtype, int n, int64_t vocab, int digit_bits, uint32_t* keys_out,
                    uint32_t* pos_out, uint32_t* arrived, int64_t arrived_count) {
    launch_dependents();
    clear_counters(arrived, arrived_count);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ClusterSmem& sm = *reinterpret_cast<ClusterSmem*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int per = kRounds * kClusterThreads;                    // positions of a CTA: a power of two
    const int mine = min(per, max(0, n - me * per));                  // how many this CTA holds
    const uint32_t digits = 1u << digit_bits, pos_mask = (1u << kPosBits) - 1u;
    auto key_of = [&](uint32_t pos) {
        const int64_t id = load_id(ids, id_dtype, pos, vocab);
        return static_cast<uint32_t>(id < 0 ? vocab : id);
    };
    for (int pass = 0; pass < 2; ++pass) {
        uint32_t* h = reinterpret_cast<uint32_t*>(&sm.hist[0][0]);
        for (int d = threadIdx.x; d < kClusterWarps * kDigits / 2; d += kClusterThreads) h[d] = 0;
        // a warp takes rounds * 32 consecutive elements, 32 at a time: their order is warp, round, lane
        uint32_t key[kRounds];                       // pass 0: the key; pass 1: the element
        uint16_t rank[kRounds];
        const int i0 = warp * kRounds * 32 + lane;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = i0 + r * 32;
            key[r] = 0;
            if (i < mine)
                key[r] = pass == 0 ? key_of(static_cast<uint32_t>(me * per + i)) : sm.elem[i];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const bool in = i0 + r * 32 < mine;
            const uint32_t d = pass == 0 ? key[r] & (digits - 1) : key[r] >> kPosBits;
            const uint32_t same = same_digit(d, in, digit_bits);
            const uint32_t before = __popc(same & ((1u << lane) - 1u));
            const uint16_t seen = in ? sm.hist[warp][d] : 0;
            rank[r] = static_cast<uint16_t>(seen + before);
            __syncwarp();
            if (in && before == 0) sm.hist[warp][d] = static_cast<uint16_t>(seen + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        if (threadIdx.x < kDigits) {
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint16_t c = sm.hist[w][threadIdx.x];
                sm.hist[w][threadIdx.x] = static_cast<uint16_t>(run);
                run += c;
            }
            sm.total[threadIdx.x] = run;
        }
        cluster.sync();
        uint32_t all = 0, before = 0;
        if (threadIdx.x < kDigits) {
#pragma unroll
            for (int c = 0; c < kClusterMax; ++c) {
                const uint32_t t = c < ctas ? cluster.map_shared_rank(&sm.total[0], c)[threadIdx.x] : 0;
                if (c < me) before += t;
                all += t;
            }
        }
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sm.scan[warp] = incl;
        __syncthreads();
        if (threadIdx.x < kDigits) {
            uint32_t off = 0;
#pragma unroll
            for (int w = 0; w < kDigits / 32; ++w) off += w < warp ? sm.scan[w] : 0;
            sm.base[threadIdx.x] = off + incl - all + before;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = i0 + r * 32;
            if (i >= mine) continue;
            const uint32_t d = pass == 0 ? key[r] & (digits - 1) : key[r] >> kPosBits;
            const uint32_t to = sm.base[d] + sm.hist[warp][d] + rank[r];
            if (pass == 0) {
                const uint32_t e = (key[r] >> digit_bits) << kPosBits | static_cast<uint32_t>(me * per + i);
                cluster.map_shared_rank(&sm.elem[0], static_cast<int>(to / per))[to % per] = e;
            } else {
                const uint32_t pos = key[r] & pos_mask;
                keys_out[to] = key_of(pos);
                pos_out[to] = pos;
            }
        }
        // pass 0: the scattered elements have arrived; pass 1: no CTA reads another's counts any more
        if (pass == 0) cluster.sync();
    }
    cluster.sync();
}

template <int kRounds>
cudaError_t launch_cluster_sort(const void* ids, int id_dtype, int64_t n, int64_t vocab, uint32_t* keys, uint32_t* pos,
                                uint32_t* arrived, int64_t arrived_count, cudaStream_t s) {
    // spread over the cluster first, then over rounds
    if (kRounds < kClusterRounds && n > static_cast<int64_t>(kClusterMax) * kRounds * kClusterThreads)
        return launch_cluster_sort<kRounds < kClusterRounds ? 2 * kRounds : kRounds>(ids, id_dtype, n, vocab, keys, pos, arrived,
                                                                                           arrived_count, s);
    static std::atomic<uint64_t> attr_set{0};        // one bit per device ordinal
    const auto kernel = cluster_sort_kernel<kRounds>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(attr_set.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(ClusterSmem));
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit);
    }
    int bits = 2;                                    // keys 0 .. vocab, in two digits
    while ((int64_t(1) << bits) <= vocab) ++bits;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    const unsigned ctas = static_cast<unsigned>(op_ceil_div(n, kRounds * kClusterThreads));
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = sizeof(ClusterSmem);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, ids, id_dtype, static_cast<int>(n), vocab, (bits + 1) / 2, keys, pos, arrived,
                              arrived_count);
}

// Up to 4 K positions: a position's place is the number of smaller keys, plus the
// equal ones before it, counted against every key by a warp; any number of
// blocks can do that side by side.  The gradient's call (512 columns, 5003 rows) for
// 777 / 2048 / 4096 positions: 10.7 / 14.7 / 22.8 us, with eight lanes per position and blocks of
// 1024 threads 13.6 / 20.7 / -, with the cluster's two passes - / - / 23.0 (into 32000 rows 22.8
// against 26.5; 8192 positions 42 against 25).
constexpr int kRankThreads = 512, kRankLanes = 32, kRankKeys = kRankThreads / kRankLanes;   // keys ranked by a block
constexpr int kRankSortMax = 4096;

__global__ void __launch_bounds__(kRankThreads)
rank_sort_kernel(const void* ids, int id_dtype, int n, int64_t vocab, uint32_t* keys_out, uint32_t* pos_out,
                 uint32_t* arrived, int64_t arrived_count) {
    __shared__ __align__(16) uint32_t key[kRankSortMax];
    launch_dependents();
    clear_counters(arrived, arrived_count);
#pragma unroll
    for (int r = 0; r < kRankSortMax / kRankThreads; ++r) {
        const int i = r * kRankThreads + static_cast<int>(threadIdx.x);
        const int64_t id = i < n ? load_id(ids, id_dtype, i, vocab) : -1;
        key[i] = i >= n ? 0xffffffffu : static_cast<uint32_t>(id < 0 ? vocab : id);   // past the end: above every key
    }
    __syncthreads();
    const int i = static_cast<int>(blockIdx.x) * kRankKeys + static_cast<int>(threadIdx.x) / kRankLanes;
    const int sub = static_cast<int>(threadIdx.x) % kRankLanes;
    const uint32_t mine = key[i < n ? i : 0];
    uint32_t rank = 0;
#pragma unroll 4
    for (int j = sub * 4; j < n; j += kRankLanes * 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(key + j);
        rank += (k.x < mine || (k.x == mine && j < i)) + (k.y < mine || (k.y == mine && j + 1 < i)) +
                (k.z < mine || (k.z == mine && j + 2 < i)) + (k.w < mine || (k.w == mine && j + 3 < i));
    }
#pragma unroll
    for (int o = kRankLanes / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (sub == 0 && i < n) {
        keys_out[rank] = mine;
        pos_out[rank] = static_cast<uint32_t>(i);
    }
}

// -------------------------------------------------------- sums of sorted runs
// Bound by the table's write: 128000 x 2048 float32 from 32768 bf16 rows 191 us a call, 174
// of them the bytes at the rate of a copy; the sort takes 17.  A kernel of its own
// for the runs that cross chunks took 201 us, and 335 against 111 us where 8192 positions
// hold one token (1024 columns, 32000 rows).  A separate kernel that zeroes absent
// rows beside the sort gained nothing (204 us a call against 202), one that zeroes all
// of them lost 50 us: the fill hides the sums' latency.  Up to 1024 positions without a
// sort, each block searching the ids for its token's, was faster only without a fill
// (777 x 1024: 10 us against 15) and slower otherwise (777 x 515 into 5003 rows 18 us
// against 14, one token alone 41 us against 21).
constexpr int kMaxChunk = 64;         // sorted positions per block, at most
constexpr int kGradThreads = 128;     // columns per block: 128 x one 16-byte access
constexpr int kMaxZeroRows = 64;      // table rows per block of the zero fill, at most
constexpr int kAhead = 8;             // rows in flight per thread
// Chunks halve (down to 8) until the sums have this many blocks: a small batch is
// bound by the latency of its rows, a large one by their bytes, a frequent token's
// run by its chunks (8192 x 1024, 150 / 300 / 600 blocks: tokens evenly drawn 43 / 39 / 37 us,
// as in text 42 / 41 / 47, one token alone 63 / 111 / 204).
constexpr int64_t kGradBlocks = 300;
constexpr int64_t kZeroBlocks = 2400; // and the zero fill's blocks halve their rows (down to 4) until there are this many

struct GradArgs {
    const void* dy;
    int64_t ldy, n, vocab, dim;
    const uint32_t* keys;             // sorted, n
    const uint32_t* pos;
    void* dw;
    int64_t ldw;
    float* part;                      // [chunk][2][part_ld]: a run's rows in a chunk it enters from before, or leaves
    int64_t part_ld;                  // dim up to whole pieces
    uint32_t* arrived;                // [chunk][column slab]: parts there of the run that leaves that chunk
    float scale;
    int accumulate, wide_out;
    int chunk, zero_rows;             // positions per chunk, table rows per zero-fill block
    int64_t chunks, sum_blocks;       // sum_blocks = chunks * column slabs; zero-fill blocks follow
};

// The old row of an accumulation is read element by element (32768 x 2048 bf16 added into 12.7
// thousand rows of a float32 table: 121 us, 51 of them the bytes).
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

// `valid` elements at p one by one, as the bits of a whole piece (rows off 16-byte boundaries:
// 32768 x 2047 bf16 into 128000 float32 rows 414 us, 2048 columns 192).
template <typename T>
__device__ __forceinline__ uint4 load_elements(const T* p, int valid) {
    constexpr int V = Elem<T>::kVec;
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = k < valid ? Elem<T>::to_float(p[k]) : 0.f;
    return pack16(v);
}

// First sorted position in [lo, hi] whose key is not below v.
__device__ __forceinline__ int64_t lower_bound_key(const uint32_t* keys, int64_t lo, int64_t hi, int64_t v) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}
// The same by a whole warp, 32 probes at a time.
__device__ __forceinline__ int64_t warp_lower_bound_key(const uint32_t* keys, int64_t n, int64_t v) {
    int64_t lo = 0, hi = n;                           // the answer lies in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + (threadIdx.x & 31) * step;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && keys[at] < v);   // a prefix of the lanes
        const int c = __popc(below);
        if (c == 0) return lo;
        const int64_t nlo = lo + (c - 1) * step + 1, nhi = lo + c * step;
        lo = nlo;
        hi = nhi < hi ? nhi : hi;
    }
    return lo;
}

// Seven blocks per SM: 72 registers, of which the bf16 rows' form spills 24 bytes.  With six (80
// registers, no spills) / seven / eight blocks 32768 x 2048 into 128000 rows takes 200 / 193 / 195 us, x 1024 into
// 32000 rows 56 / 60 / 62, 8192 x 1024 of one token 120 / 115 / 123.
template <typename T, typename D, bool kWide>
__global__ void __launch_bounds__(kGradThreads, 7) grad_sum_kernel(const __grid_constant__ GradArgs a) {
    constexpr int V = Elem<T>::kVec;
    wait_for_previous();
    if (blockIdx.x >= a.sum_blocks) {                // rows of absent tokens: zeros
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - a.sum_blocks) * a.zero_rows;
        __shared__ uint8_t present[kMaxZeroRows];
        __shared__ int64_t range[2];
        if (threadIdx.x < 64) {                       // the positions of the block's tokens
            const int w = threadIdx.x >> 5;
            const int64_t at = warp_lower_bound_key(a.keys, a.n, r0 + (w ? a.zero_rows : 0));
            if ((threadIdx.x & 31) == 0) range[w] = at;
        }
        __syncthreads();
        for (int r = threadIdx.x; r < a.zero_rows; r += kGradThreads) {
            const int64_t v = r0 + r;
            uint8_t is = 1;
            if (v < a.vocab) {
                const int64_t at = lower_bound_key(a.keys, range[0], range[1], v);
                is = at < range[1] && a.keys[at] == v;
            }
            present[r] = is;
        }
        __syncthreads();
        constexpr int Z = Elem<D>::kVec;
        for (int r = 0; r < a.zero_rows; ++r) {
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
    __shared__ uint32_t skey[kMaxChunk + 2], spos[kMaxChunk];   // skey[0], skey[len + 1]: the neighbours' keys
    __shared__ int last_here[2];
    __shared__ int64_t span[2][2];
    const int64_t chunk = blockIdx.x % a.chunks, slab = blockIdx.x / a.chunks;
    const int64_t p0 = chunk * a.chunk;
    const int len = static_cast<int>(a.n - p0 < a.chunk ? a.n - p0 : a.chunk);
    const uint32_t none = 0xffffffffu, dropped = static_cast<uint32_t>(a.vocab);
    auto key_at = [&](int64_t q) { return q >= 0 && q < a.n ? a.keys[q] : none; };
    for (int i = threadIdx.x; i < len + 2; i += kGradThreads) skey[i] = key_at(p0 + i - 1);
    // warp 0: the last keys of the 32 chunks before; warp 1: the first keys of the 32 after
    uint32_t edge = none;
    if (threadIdx.x < 64) {
        const int64_t off = static_cast<int64_t>(threadIdx.x & 31) * a.chunk;
        edge = key_at(threadIdx.x < 32 ? p0 - 1 - off : p0 + a.chunk + off);
    }
    for (int i = threadIdx.x; i < len; i += kGradThreads) spos[i] = a.pos[p0 + i];
    __syncthreads();
    const int64_t c = (slab * kGradThreads + threadIdx.x) * V;
    const int nv = static_cast<int>(c >= a.dim ? 0 : a.dim - c < V ? a.dim - c : V);   // this thread's columns
    const T* dy = static_cast<const T*>(a.dy) + c;
    const bool enters = skey[0] == skey[1] && skey[1] != dropped, leaves = skey[len + 1] == skey[len] && skey[len] != dropped;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    bool from_before = enters;
    for (int i0 = 0; i0 < (nv > 0 ? len : 0); i0 += kAhead) {
        uint4 raw[kAhead];
        auto load_rows = [&](auto load) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                raw[u] = make_uint4(0, 0, 0, 0);
                if (i0 + u < len && skey[i0 + u + 1] != dropped)
                    raw[u] = load(dy + static_cast<int64_t>(spos[i0 + u]) * a.ldy);
            }
        };
        // (two loops: the choice inside one keeps the loads from being issued back to back)
        if (kWide && nv == V)
            load_rows([](const T* p) { return __ldg(reinterpret_cast<const uint4*>(p)); });
        else
            load_rows([&](const T* p) { return load_elements(p, nv); });
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= len || skey[i + 1] == dropped) continue;
            float v[V];
            unpack16(raw[u], v);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += v[k];
            const bool last = i + 1 == len;
            if (!last && skey[i + 2] == skey[i + 1]) continue;
            const bool goes_on = last && skey[i + 2] == skey[i + 1];
            if (from_before || goes_on) {
                // slot 0: the run entered from before (and perhaps goes on); slot 1: it starts here and goes on
                store_run<float, V>(a.part + ((chunk * 2 + (from_before ? 0 : 1)) * a.part_ld + c), acc, true);
            } else {
                write_row<D, V>(a, skey[i + 1], c, nv, acc);
            }
            from_before = false;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
        }
    }
    // A run that crosses chunks: the block that brings its last part adds all of
    // them, in the chunks' order whichever block that is.
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {                                       // the run that enters, the one that leaves
        if (side == 0 ? !enters : !leaves || (enters && skey[1] == skey[len])) continue;   // block-uniform
        const uint32_t key = skey[side == 0 ? 1 : len];
        // the run's chunks: as many neighbours as end (begin) with its key; more than 32 are searched for
        const bool from_left = side == 0, to_right = side == 1 || (leaves && skey[len] == key);
        if (threadIdx.x < 64) {
            const bool first = threadIdx.x < 32;
            const uint32_t other = ~__ballot_sync(0xffffffffu, edge == key);
            const int more = __ffs(other) - 1;                                   // -1: all 32
            int64_t q = chunk;
            if (first && from_left)
                q = more >= 0 ? chunk - more : warp_lower_bound_key(a.keys, a.n, key) / a.chunk;
            else if (!first && to_right)
                q = more >= 0 ? chunk + more : (warp_lower_bound_key(a.keys, a.n, static_cast<int64_t>(key) + 1) - 1) / a.chunk;
            if ((threadIdx.x & 31) == 0) span[side][first ? 0 : 1] = q;
        }
        __syncthreads();                                                         // and the block's parts are written
        const int64_t q0 = span[side][0], q1 = span[side][1];
        if (threadIdx.x == 0) {
            __threadfence();
            last_here[side] = atomicAdd(&a.arrived[q0 * (a.sum_blocks / a.chunks) + slab], 1u) == static_cast<uint32_t>(q1 - q0);
            __threadfence();
        }
        __syncthreads();
        if (!last_here[side] || nv == 0) continue;
        constexpr int kRows = 32 / V;                                            // parts in flight per thread
        const float* src = a.part + c;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        for (int64_t q = q0; q <= q1; q += kRows) {
            float v[kRows][V];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const float* row = src + ((q + u) * 2 + (q + u == q0 ? 1 : 0)) * a.part_ld;
#pragma unroll
                for (int k = 0; k < V; k += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (q + u <= q1) x = __ldcg(reinterpret_cast<const float4*>(row + k));   // from L2, where other blocks' parts are
                    v[u][k] = x.x; v[u][k + 1] = x.y; v[u][k + 2] = x.z; v[u][k + 3] = x.w;
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += v[u][k];
        }
        write_row<D, V>(a, key, c, nv, acc);
    }
}

struct GradLayout {
    size_t keys[2], pos[2], counts, part, arrived, total;
    int64_t chunks, part_ld, arrived_count;
    int passes, digit_bits, tiles, rounds, chunk;
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
    L.chunk = kMaxChunk;
    while (L.chunk > 8 && op_ceil_div(n, L.chunk) * op_ceil_div(dim, kGradThreads * 8) < kGradBlocks) L.chunk /= 2;
    L.chunks = op_ceil_div(n, L.chunk);
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = op_align_up(o + bytes, 256); return at; };
    for (int k = 0; k < 2; ++k) L.keys[k] = take(static_cast<size_t>(n) * 4);
    for (int k = 0; k < 2; ++k) L.pos[k] = take(static_cast<size_t>(n) * 4);
    L.counts = take((static_cast<size_t>(L.tiles) << L.digit_bits) * 4);
    L.part_ld = op_ceil_div(dim, 8) * 8;
    L.part = take(static_cast<size_t>(L.chunks) * 2 * static_cast<size_t>(L.part_ld) * 4);
    L.arrived_count = L.chunks * op_ceil_div(dim, kGradThreads * 4);    // column slabs, at most
    L.arrived = take(static_cast<size_t>(L.arrived_count) * 4);
    L.total = o > 256 ? o : 256;
    return L;
}

template <typename T, typename D>
cudaError_t launch_grad(const GradArgs& a0, cudaStream_t s) {
    GradArgs a = a0;
    constexpr int V = Elem<T>::kVec;
    const bool wide_in = op_aligned(a.dy, 16) && (a.ldy * sizeof(T)) % 16 == 0;
    a.wide_out = op_aligned(a.dw, 16) && (a.ldw * sizeof(D)) % 16 == 0;
    const int64_t slabs = op_ceil_div(a.dim, static_cast<int64_t>(kGradThreads) * V);
    a.sum_blocks = a.chunks * slabs;
    a.zero_rows = kMaxZeroRows;
    while (a.zero_rows > 4 && op_ceil_div(a.vocab, a.zero_rows) < kZeroBlocks) a.zero_rows /= 2;
    const int64_t zero_blocks = a.accumulate ? 0 : op_ceil_div(a.vocab, a.zero_rows);
    const unsigned grid = static_cast<unsigned>(a.sum_blocks + zero_blocks);
    if (grid == 0) return cudaSuccess;
    return wide_in ? launch_after(grad_sum_kernel<T, D, true>, grid, kGradThreads, s, a)
                   : launch_after(grad_sum_kernel<T, D, false>, grid, kGradThreads, s, a);
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
    // one block for each chunk and column slab, and for each block of zeroed rows: a grid's limit
    if (op_ceil_div(n, kMaxChunk) * op_ceil_div(dim, kGradThreads * 4) + op_ceil_div(vocab, kMaxZeroRows) > kMaxCount)
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
    uint32_t* arrived = reinterpret_cast<uint32_t*>(base + L.arrived);
    if (n > 0) {
        const cudaError_t e = op_traced(MO_K_EMBED_SORT, s, [&] {
            if (n <= kRankSortMax) {
                rank_sort_kernel<<<static_cast<unsigned>(op_ceil_div(n, kRankKeys)), kRankThreads, 0, s>>>(
                    ids, id_dtype, static_cast<int>(n), vocab, keys[(L.passes + 1) & 1], pos[(L.passes + 1) & 1], arrived,
                    L.arrived_count);
                return cudaGetLastError();
            }
            if (n <= kClusterSortMax && vocab <= kClusterVocabMax) {
                const cudaError_t e = launch_cluster_sort<1>(ids, id_dtype, n, vocab, keys[(L.passes + 1) & 1],
                                                             pos[(L.passes + 1) & 1], arrived, L.arrived_count, s);
                if (e == cudaSuccess) return e;
                (void)cudaGetLastError();              // no room for such a cluster (a part of a GPU): the passes below
            }
            for (int k = 0; k < L.passes; ++k) {
                SortPass p;
                p.arrived = arrived;
                p.arrived_count = L.arrived_count;
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
                p.digit_bits = L.digit_bits;
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
    a.part_ld = L.part_ld;
    a.arrived = arrived;
    a.scale = scale;
    a.accumulate = accumulate;
    a.chunk = L.chunk;
    a.chunks = L.chunks;
    return op_status(op_traced(MO_K_EMBED_GRAD, s, [&] {
        if (dy_dtype == MO_F32) return dw_dtype == MO_F32 ? launch_grad<float, float>(a, s) : launch_grad<float, bf16>(a, s);
        return dw_dtype == MO_F32 ? launch_grad<bf16, float>(a, s) : launch_grad<bf16, bf16>(a, s);
    }));
}

}  // extern "C"
