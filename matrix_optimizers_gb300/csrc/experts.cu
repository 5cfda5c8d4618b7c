// Matrix products grouped by expert on the tensor cores: rows sorted by expert,
// expert e holding rows offsets[e] .. offsets[e + 1] - 1 (device memory).
//   forward  Y[r, :]  = X[r, :] W_e^T
//   dgrad    dX[r, :] = dY[r, :] W_e
//   wgrad    dW_e (+)= sum_r dY[r, :]^T X[r, :]
//
// One persistent CTA per SM walks tiles of D[128, N <= 256] += A B^T.  The 128
// TMEM lanes hold output features and the columns hold tokens (forward,
// dgrad), so that a ragged group costs N rounded up to 16 tokens and not to a
// whole tile; the weight gradient has n on the lanes and k on the columns, and
// its ragged sum over rows ends at a multiple of 16.
//   forward  A = W_e   (K-major),  B = X   (K-major),  sum over k
//   dgrad    A = W_e^T (MN-major), B = dY  (K-major),  sum over n
//   wgrad    A = dY^T  (MN-major), B = X^T (MN-major), sum over the rows
// Every operand comes straight from its row-major home by TMA in 128-byte
// swizzled boxes; no transposed copy is made.
//
// Bound by the tensor cores where the rows are many: 16384 rows, 8 experts of 4096 x 4096,
// forward 294 us (1.87 PFLOP/s, 84% tensor activity), dgrad 294 us, wgrad 295 us (bf16) and
// 324 us (float32, whose sums leave TMEM on the way).  With few rows per expert by the
// weights' bytes, read (forward, dgrad) or written (wgrad: 64 rows per expert, 16 experts
// of 2048 x 2048 float32 49 us, 5.5 TB/s).
//
// Roles (384 threads): warps 0-7 epilogue, warp 8 TMA producer, warp 9 TMEM
// allocation and tcgen05.mma issue into two alternating 256-column accumulators.
// The producer's and the MMA warp's loops run warp-uniform, with one lane elected
// per issue: the same loops inside one lane issued at most 1.48 PFLOP/s of MMAs, these
// 2.2, because the compiler then keeps descriptors and addresses in uniform registers.  Barrier waits are bounded (ptx.cuh); one that gives up raises
// the CTA's abort flag, records a code in the workspace's error word and unwinds.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "ptx.cuh"
#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

enum ExpertMode { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kBM = 128, kBN = 256, kBK = 64;             // lanes, columns and depth of one CTA's tile and stage
constexpr int kABytes = kBM * kBK * 2;                    // 16 KB
constexpr int kRingBytes = 196608;
constexpr int kMaxStages = 9;
// Single CTA (cta_group::1): a stage holds 128 features and up to 256 columns
// (48 KB, four stages).  CTA pair (cta_group::2): 256 features x up to 256
// columns per pair, each CTA holding its 128 features and half the columns
// (32 KB, six stages), its own 128 x 256 accumulator and its own epilogue.
// Few rows per expert: the weights are all there is to read, so tiles of up to 32
// tokens and nine stages of 20 KB keep 144 KB of them in flight per SM instead of 64.
// A weight gradient on single CTAs, which sums few rows and is bound by its stores,
// gives a stage up for wider store blocks, two per epilogue warp.
enum Shape { kSingle = 0, kPairs = 1, kFew = 2 };
constexpr int shape_columns(int shape) { return shape == kFew ? 32 : kBN; }   // of a tile, at most
constexpr int shape_features(int shape) { return shape == kPairs ? 2 * kBM : kBM; }
template <int kMode, int kShape>
struct Geo {
    static constexpr bool kPair = kShape == kPairs, kWideOut = kMode == kWgrad && !kPair;
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kColumns = shape_columns(kShape), kFeatures = shape_features(kShape);
    static constexpr int kStageBytes = kABytes + kColumns / kCtas * kBK * 2;
    static constexpr int kStages = kRingBytes / kStageBytes - (kWideOut ? 1 : 0);
    static constexpr int kOutRow = kWideOut ? 128 : 64;                       // wgrad: bytes of a store block's 32 rows
    static constexpr int kOutBlocks = kWideOut ? 2 : 1;
    static constexpr int kRound = kPair ? 32 : 16;                            // columns of an MMA come in multiples of
    static_assert(kStages <= kMaxStages, "ring depth");
};
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = 32 * (kEpiWarps + 4);            // three warpgroups; two warps of the last have no role
// Registers: the launch gives 168 to every thread; the last warpgroup keeps 56 of
// them and the two epilogue warpgroups, which hold a tile's sums, take 224.
constexpr int kLaunchRegs = 168, kIssueRegs = 56, kEpiRegs = 224;
static_assert(4 * kIssueRegs + kEpiWarps * kEpiRegs <= (kThreads / 32) * kLaunchRegs, "register split");
constexpr int kOutBytes = 2048;                           // one epilogue warp's store block
constexpr int kMaxExperts = 1024;
constexpr int kBoxes = 4;                                 // token boxes of 128, 64, 32 and 16 rows

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
    uint64_t tail[kMaxStages], tail_peer[kMaxStages];     // pair, wgrad: a sum's ragged last block in that stage
    uint32_t tmem_base;
    int abort_flag;
    int32_t cum[kMaxExperts + 1];                         // token tiles before expert e
    int32_t row[kMaxExperts + 1];                         // first row of expert e: not falling, inside [0, rows]
};
constexpr int kCtlBytes = (sizeof(Ctl) + 1023) / 1024 * 1024;
constexpr int kSmemBytes = kRingBytes + kEpiWarps * kOutBytes + kCtlBytes + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

struct ExpertArgs {
    CUtensorMap a;                 // W, or dY (wgrad)
    CUtensorMap b[kBoxes];         // X or dY rows in boxes of 128 >> i; wgrad: b[0] is X
    CUtensorMap o;                 // output stores
    const int32_t* offsets;
    void* out;
    int64_t ldo, stride_o;
    int32_t rows, n, k, experts;
    int32_t group;                 // token tiles that share a sweep over the features, at most
    int32_t f_tiles;               // tiles over the output features
    int32_t width, c_tiles;        // wgrad: columns of a tile, tiles over the k columns
    int32_t splits;                // parts of every sum, each into an output of its own (joined afterwards)
    int32_t chunk;                 // K blocks summed in TMEM before the float32 sum moves on to registers
    int* err;
};

struct Tile {
    int e;
    int f0;                        // first output feature on the lanes (of the pair's first CTA)
    int c0, cn;                    // first column (absolute token row, or k) and how many are real
    int nmma;                      // columns of the MMA: cn rounded up to 16 (pair: 32)
    int r0, depth;                 // wgrad: first row of the sum; length of the sum
    int kb0, kb1;                  // the K blocks (of kBK) of this tile's part of the sum
    int split;
};

// tcgen05 instruction descriptor: bf16 x bf16 -> f32, M x N.
__device__ __forceinline__ uint32_t instr_desc(uint32_t m, uint32_t n, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ int ceil_div_i(int a, int b) { return (a + b - 1) / b; }

// (the host sees to it that tile numbers fit 31 bits)
template <int kMode>
__device__ __forceinline__ int tile_count(const ExpertArgs& p, const Ctl* ctl) {
    return (kMode == kWgrad ? p.experts * p.c_tiles : ctl->cum[p.experts]) * p.f_tiles * p.splits;
}

// Tile u of the walk.  Forward and dgrad go expert by expert, within one in
// groups of token tiles, each sweeping the features with the tokens innermost: a
// group's rows stay in L2 while every weight is read once for the group.
template <int kMode, int kShape>
__device__ __forceinline__ Tile tile_at(const ExpertArgs& p, const Ctl* ctl, int tile) {
    using G = Geo<kMode, kShape>;
    Tile t;
    uint32_t u = static_cast<uint32_t>(tile);
    t.split = 0;
    if (p.splits > 1) {
        t.split = static_cast<int>(u % p.splits);
        u /= p.splits;
    }
    if (kMode == kWgrad) {
        const uint32_t strip = u / p.c_tiles, c = u - strip * p.c_tiles;       // strip: one expert's feature tile
        t.e = static_cast<int>(strip / p.f_tiles);
        t.f0 = static_cast<int>(strip - t.e * p.f_tiles) * G::kFeatures;
        t.c0 = static_cast<int>(c) * p.width;
        t.cn = min(p.width, p.k - t.c0);
        t.r0 = ctl->row[t.e];
        t.depth = ctl->row[t.e + 1] - t.r0;
    } else {
        const int strip = static_cast<int>(u / p.f_tiles);                     // counts token tiles of the experts before
        int lo = 0, hi = p.experts - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ctl->cum[mid] <= strip) lo = mid; else hi = mid - 1;
        }
        t.e = lo;
        const int nt = ctl->cum[lo + 1] - ctl->cum[lo];
        const int group = ceil_div_i(nt, ceil_div_i(nt, p.group));             // equal groups
        const uint32_t v = u - static_cast<uint32_t>(ctl->cum[lo]) * p.f_tiles, per = group * p.f_tiles;
        const int g = static_cast<int>(v / per);
        const uint32_t w = v - g * per, gs = min(group, nt - g * group);
        const int m = ctl->row[lo + 1] - ctl->row[lo], f = static_cast<int>(w / gs);
        const int tok = g * group + static_cast<int>(w - f * gs);
        const int size = (ceil_div_i(m, nt) + G::kRound - 1) / G::kRound * G::kRound;   // equal tiles
        t.f0 = f * G::kFeatures;
        t.c0 = ctl->row[lo] + tok * size;
        t.cn = min(size, m - tok * size);
        t.r0 = 0;
        t.depth = kMode == kFwd ? p.k : p.n;
    }
    t.nmma = (t.cn + G::kRound - 1) / G::kRound * G::kRound;
    t.kb0 = 0;
    t.kb1 = ceil_div_i(t.depth, kBK);
    if (p.splits > 1) {
        const int part = ceil_div_i(t.kb1, p.splits);
        t.kb0 = min(t.split * part, t.kb1);
        t.kb1 = min(t.kb0 + part, t.kb1);
    }
    return t;
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_b32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_b16(uint32_t a, bf16 v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(*reinterpret_cast<unsigned short*>(&v)) : "memory");
}

// A wait that also acquires what the arriving CTA of the cluster wrote.
__device__ __forceinline__ bool mbar_wait_cluster_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                                          int code) {
    const long long t0 = clock64();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort_flag = 1;
            atomicCAS(err, 0, code);
            return false;
        }
    }
}

// A bounded wait by a whole warp; the vote tells the compiler that the outcome
// (and so the control flow and the addresses derived from it) is the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, err, code));
}
// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// One operand box, the pair form counting on an mbarrier of either CTA.
template <bool kPair>
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
    if constexpr (kPair)
        tma_load_2d_pair(dst, m, bar, x, y);
    else
        tma_load_2d(dst, m, bar, x, y);
}
template <bool kPair>
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
    if constexpr (kPair)
        tma_load_3d_pair(dst, m, bar, x, y, z);
    else
        tma_load_3d(dst, m, bar, x, y, z);
}

// The rows from `v` up to the next multiple of 16 of a weight gradient's last
// block belong to another expert (or to none): they become zero in both
// operands, so that not even their infinities or NaN reach the sum.  Called by a
// whole warp after the block's copies landed.
__device__ __forceinline__ void zero_tail(uint32_t stage, int boxes, int v, int lane) {
    const int per = ((v + 15) / 16 * 16 - v) * 8;         // 16-byte pieces per 64-wide box
    for (int i = lane; i < boxes * per; i += 32)
        sts_v4(stage + (i / per) * 8192 + v * 128 + (i % per) * 16, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    __syncwarp();
}

// ---------------------------------------------------------------- epilogues
// Forward and dgrad: the warp holds 32 features (lanes) x 32 tokens (v).  The
// block goes through shared memory so that a token's features are contiguous;
// a full block leaves by one TMA store, a block that ends inside the group by
// plain stores of its real tokens.  A TMA store clips features past the end, but
// in whole 16-byte pieces (measured: it wrote the elements between the end and
// the next 16-byte boundary), so a block with an end inside a piece is stored plainly.
template <bool kF32>
__device__ __forceinline__ void put_tokens(const ExpertArgs& p, int cols, int f, int64_t token, int valid,
                                           const float* v, uint32_t buf, int lane) {
    constexpr int kTok = kF32 ? 16 : 32;               // tokens of one 2 KB block
    constexpr int kRow = kF32 ? 128 : 64;              // bytes of one token's 32 features
    const bool whole = f + 32 <= cols || cols % (kF32 ? 4 : 8) == 0;
#pragma unroll
    for (int h = 0; h < 32 / kTok; ++h) {
        const int nv = min(kTok, valid - h * kTok);
        if (nv <= 0) return;                           // warp-uniform
        if (elect_one()) bulk_wait_read_all();           // the last store has read the block
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            if (kF32)
                sts_b32(buf + t * kRow + lane * 4, __float_as_uint(v[h * kTok + t]));
            else
                sts_b16(buf + t * kRow + lane * 2, __float2bfloat16_rn(v[h * kTok + t]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (nv == kTok && whole) {
            if (elect_one()) {
                tma_store_2d(&p.o, buf, f, static_cast<int>(token + h * kTok));
                bulk_commit();
            }
        } else {
            constexpr int kPieces = kRow / 16, kPer = kF32 ? 4 : 8;     // 16-byte pieces of a row, elements of one
            for (int j = lane; j < nv * kPieces; j += 32) {
                const int t = j / kPieces, q = j % kPieces, c = f + q * kPer;
                if (c >= cols) continue;
                const int64_t at = (token + h * kTok + t) * p.ldo + c;
                const uint32_t src = buf + t * kRow + q * 16;
                if (c + kPer <= cols) {
                    void* dst = kF32 ? static_cast<void*>(static_cast<float*>(p.out) + at)
                                     : static_cast<void*>(static_cast<bf16*>(p.out) + at);
                    *reinterpret_cast<uint4*>(dst) = lds_v4(src);
                } else {
                    const uint4 u = lds_v4(src);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    for (int i = 0; c + i < cols; ++i) {
                        if (kF32)
                            static_cast<float*>(p.out)[at + i] = __uint_as_float(w[i]);
                        else
                            reinterpret_cast<unsigned short*>(p.out)[at + i] =
                                static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
            __syncwarp();
        }
    }
}

// Weight gradient: column group g of a warp's four 32-column groups (pairs of
// groups are neighbours, so that a 128-byte block of bf16 holds two).
__device__ __forceinline__ int wgrad_column(int half, int g) { return (g >> 1) * 128 + half * 64 + (g & 1) * 32; }

// The warp holds 32 rows (lanes) x its four groups.  They leave in blocks of 32
// rows x kRow bytes, staged with the swizzle of the store view (16-byte chunk c of
// row r at c ^ (r & 7) for 128-byte rows, c ^ ((r >> 1) & 3) for 64-byte rows).
template <bool kF32, bool kAcc, int kRow, int kBlocks>
__device__ __forceinline__ void put_weights(const ExpertArgs& p, int e, int row0, int c0, int cn, int half, float (&v)[4][32],
                                            uint32_t buf0, int& block, int lane) {
    constexpr int kCols = kRow / (kF32 ? 4 : 2), kPer = kF32 ? 4 : 8;   // columns of a block, of 16 bytes
#pragma unroll
    for (int b = 0; b < 128 / kCols; ++b) {
        const int g0 = b * kCols / 32, j0 = b * kCols % 32, col = wgrad_column(half, g0) + j0;   // within the tile
        if (col >= cn) continue;                       // warp-uniform
        if (kAcc && row0 + lane < p.n) {               // (each lane its own row, 4 or 2 bytes at a time: 16384 rows, 8
                                                       // experts of 4096 x 4096 float32 737 us, 367 without)
            const int64_t at = e * p.stride_o + static_cast<int64_t>(row0 + lane) * p.ldo + c0 + col;
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                if (col + j < cn)
                    v[g0 + (j0 + j) / 32][(j0 + j) % 32] += kF32 ? static_cast<const float*>(p.out)[at + j]
                                                                 : __bfloat162float(static_cast<const bf16*>(p.out)[at + j]);
        }
        if (c0 + col + kCols > p.k && p.k % kPer != 0) {   // ends inside a 16-byte piece (see put_tokens)
            if (row0 + lane < p.n) {
                const int64_t at = e * p.stride_o + static_cast<int64_t>(row0 + lane) * p.ldo + c0 + col;
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    if (c0 + col + j >= p.k) continue;
                    const float x = v[g0 + (j0 + j) / 32][(j0 + j) % 32];
                    if (kF32)
                        static_cast<float*>(p.out)[at + j] = x;
                    else
                        static_cast<bf16*>(p.out)[at + j] = __float2bfloat16_rn(x);
                }
            }
            continue;
        }
        const uint32_t buf = buf0 + block * (32 * kRow);
        block = block + 1 == kBlocks ? 0 : block + 1;
        if (elect_one())                               // the store that last used the block has read it
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBlocks - 1) : "memory");
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kRow / 16; ++c) {
            float w[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) w[i] = v[g0 + (j0 + c * kPer + i) / 32][(j0 + c * kPer + i) % 32];
            sts_v4(buf + lane * kRow + ((kRow == 128 ? c ^ (lane & 7) : c ^ ((lane >> 1) & 3)) << 4), pack16(w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
            tma_store_3d(&p.o, buf, c0 + col, row0, e);
            bulk_commit();
        }
    }
}

// Arrives on `bar` (in both CTAs of a pair) when the MMAs issued so far are done.
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (kPair)
        umma_commit_pair(bar, 0x3);
    else
        umma_commit(bar);
}

template <int kMode, bool kF32, int kShape, bool kAcc>
__global__ void __launch_bounds__(kThreads, 1) expert_kernel(const __grid_constant__ ExpertArgs p) {
    using G = Geo<kMode, kShape>;
    constexpr bool kPair = G::kPair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + kRingBytes + kEpiWarps * kOutBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    launch_dependents();                               // the next call of these operators may set up while this one ends
    const int cols = kMode == kFwd ? p.n : p.k;        // features of the output
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;   // rank 0 leads the pair
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x) / G::kCtas, units = static_cast<int>(gridDim.x) / G::kCtas;

    if (threadIdx.x < 3) tma_prefetch_desc(threadIdx.x == 0 ? &p.a : threadIdx.x == 1 ? &p.b[kBoxes - 1] : &p.o);
    if (threadIdx.x == kProducerWarp * 32) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&ctl->tfull[a]), 1);
            mbar_init(smem_u32(&ctl->tempty[a]), G::kCtas * kEpiWarps);
        }
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(smem_u32(&ctl->tail[s]), 1);
            mbar_init(smem_u32(&ctl->tail_peer[s]), 1);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) {
            tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&ctl->tmem_base), 512);
            tmem_relinquish();
        }
    }
    wait_for_previous();                               // everything above touches this CTA's own state only
    if (warp == 0) {                                   // the experts' rows and token tiles
        int carry = 0, top = 0;
        if (lane == 0) ctl->cum[0] = 0;
        for (int base = 0; base <= p.experts; base += 32) {
            const int e = base + lane;
            int a = e <= p.experts ? min(max(p.offsets[e], 0), p.rows) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {                              // never below an earlier one
                const int up = __shfl_up_sync(0xffffffffu, a, o);
                if (lane >= o) a = max(a, up);
            }
            a = max(a, top);
            // the expert before ends where this one begins
            int before = __shfl_up_sync(0xffffffffu, a, 1);
            if (lane == 0) before = top;
            int tiles = e > 0 && e <= p.experts ? ceil_div_i(a - before, G::kColumns) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, tiles, o);
                if (lane >= o) tiles += up;
            }
            if (e <= p.experts) {
                ctl->row[e] = a;
                ctl->cum[e] = carry + tiles;                                // of the experts before e
            }
            carry += __shfl_sync(0xffffffffu, tiles, 31);
            top = __shfl_sync(0xffffffffu, a, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();               // both CTAs' barriers exist before any remote signal
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    const int tiles = tile_count<kMode>(p, ctl);

    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == kProducerWarp) {
            int stage = 0;
            uint32_t phase = 0, narmed = 0;
            uint32_t tail_used = 0, tail_phase = 0;         // by stage: ragged last blocks armed, the parity of the last
            bool ok = true;
            for (int u = unit; u < tiles && ok; u += units) {
                const Tile t = tile_at<kMode, kShape>(p, ctl, u);
                // this CTA's features and columns
                const int f0 = t.f0 + static_cast<int>(rank) * kBM;
                const int mine = t.nmma / G::kCtas, c0 = t.c0 + static_cast<int>(rank) * mine;
                const int nb = (mine + 63) / 64;                         // wgrad: 64-wide boxes of X
                const uint32_t bytes = kABytes + (kMode == kWgrad ? nb * 8192 : mine * kBK * 2);
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!warp_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, p.err, 0x201)) {
                        ok = false;
                        break;
                    }
                    // The pair's copies count on the leader's barrier, except that a weight
                    // gradient's ragged last block counts on each CTA's own, because each
                    // zeroes its part before the leader may use it; the stage's full barrier
                    // then only turns its phase over.
                    const bool tail = kPair && kMode == kWgrad && (kb + 1) * kBK > t.depth;
                    if (tail) {
                        tail_phase ^= (tail_used >> stage & 1u) << stage;
                        tail_used |= 1u << stage;
                    }
                    if (elect_one()) {
                        const uint32_t full = smem_u32(&ctl->full[stage]);
                        uint32_t bar = kPair ? mapa_shared(full, 0) : full;
                        if (tail) {
                            if (leader) mbar_arrive(full);
                            bar = smem_u32(&ctl->tail[stage]);
                            mbar_arrive_expect_tx(bar, bytes);
                            bar = mapa_shared(bar, rank);
                        } else if (leader) {
                            mbar_arrive_expect_tx(full, G::kCtas * bytes);
                        }
                        const uint32_t sa = smem_u32(smem + stage * G::kStageBytes);
                        const uint32_t sb = sa + kABytes;
                        const int k0 = kb * kBK;
                        if (kMode == kFwd) {
                            load3<kPair>(sa, &p.a, bar, k0, f0, t.e);
                        } else if (kMode == kDgrad) {
                            load3<kPair>(sa, &p.a, bar, f0, k0, t.e);
                            load3<kPair>(sa + 8192, &p.a, bar, f0 + 64, k0, t.e);
                        } else {
                            load2<kPair>(sa, &p.a, bar, f0, t.r0 + k0);
                            load2<kPair>(sa + 8192, &p.a, bar, f0 + 64, t.r0 + k0);
                            for (int i = 0; i < nb; ++i)
                                load2<kPair>(sb + i * 8192, &p.b[0], bar, c0 + i * 64, t.r0 + k0);
                        }
                        if (kMode != kWgrad) {
                            // the tokens as boxes of 128, 64, 32 and 16 rows
                            int at = 0;
                            if (kShape == kSingle && mine == 256) {
                                load2<kPair>(sb, &p.b[0], bar, k0, c0);
                                at = 128;
                            }
#pragma unroll
                            for (int i = 0; i < kBoxes; ++i) {
                                const int r = 128 >> i;
                                if (mine - at >= r) {
                                    load2<kPair>(sb + at * 128, &p.b[i], bar, k0, c0 + at);
                                    at += r;
                                }
                            }
                        }
                    }
                    __syncwarp();
                    ++narmed;
                    if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            if (lane == 0) {
                // every armed copy lands before the CTA exits, also when the MMA warp gave up
                // first; the leader's barriers also count the peer's copies
                if (leader) {
                    for (int s = 0; s < G::kStages; ++s) {
                        if (narmed <= static_cast<uint32_t>(s)) continue;
                        const uint32_t times = (narmed - 1u - static_cast<uint32_t>(s)) / G::kStages + 1u;
                        const long long t0 = clock64();
                        while (!mbar_try_wait(smem_u32(&ctl->full[s]), (times - 1u) & 1u) && clock64() - t0 < kWaitCycles) {}
                    }
                } else if (!ok) {
                    // copies that count on the leader's barriers: time to land (~2 ms, far above
                    // a copy's latency); the closing cluster barrier keeps this CTA until the leader is done
                    const long long t0 = clock64();
                    while (clock64() - t0 < (1LL << 22)) {}
                }
                for (int s = 0; s < G::kStages; ++s) {
                    if (!(tail_used >> s & 1u)) continue;
                    const long long t0 = clock64();
                    while (!mbar_try_wait(smem_u32(&ctl->tail[s]), tail_phase >> s & 1u) && clock64() - t0 < kWaitCycles) {}
                }
            }
        } else if (warp == kMmaWarp && leader) {
            int stage = 0;
            uint32_t phase = 0, tail_phase = 0;             // tail_phase: by stage
            bool ok = true;
            int q = 0;                                      // chunks so far: accumulator ping-pong
            for (int u = unit; u < tiles && ok; u += units) {
                const Tile t = tile_at<kMode, kShape>(p, ctl, u);
                const uint32_t idesc = instr_desc(G::kFeatures, t.nmma, kMode != kFwd, kMode == kWgrad);
                // K-major operands: 8-row groups 1 KB apart, 32 bytes per 16-wide step.
                // MN-major operands: 64-column blocks 8 KB apart, 8-row K groups 1 KB
                // apart, two of them (2 KB) per step.
                const uint64_t ad0 = kMode == kFwd ? sdesc_sw128(0, 16, 1024) : sdesc_sw128(0, 8192, 1024);
                const uint64_t bd0 = kMode == kWgrad ? sdesc_sw128(0, 8192, 1024) : sdesc_sw128(0, 16, 1024);
                constexpr uint32_t a_step = (kMode == kFwd ? 32 : 2048) >> 4, b_step = (kMode == kWgrad ? 2048 : 32) >> 4;
                int in_chunk = 0;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (in_chunk == 0 &&
                        !warp_wait(smem_u32(&ctl->tempty[q & 1]), ((q >> 1) & 1) ^ 1u, abort_flag, p.err, 0x202)) {
                        ok = false;
                        break;
                    }
                    if (!warp_wait(smem_u32(&ctl->full[stage]), phase, abort_flag, p.err, 0x203)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem_u32(smem + stage * G::kStageBytes), sb = sa + kABytes;
                    int steps = kBK / 16;
                    if (kMode == kWgrad && (kb + 1) * kBK > t.depth) {              // the sum ends inside this block
                        const int v = t.depth - kb * kBK, boxes = 2 + (t.nmma / G::kCtas + 63) / 64;
                        steps = (v + 15) / 16;
                        if (kPair && !warp_wait(smem_u32(&ctl->tail[stage]), tail_phase >> stage & 1u, abort_flag, p.err, 0x205)) {
                            ok = false;
                            break;
                        }
                        zero_tail(sa, boxes, v, lane);
                        if (kPair) {
                            bool there = mbar_wait_cluster_bounded(smem_u32(&ctl->tail_peer[stage]), tail_phase >> stage & 1u,
                                                                   abort_flag, p.err, 0x206);
                            if (!__all_sync(0xffffffffu, there)) {
                                ok = false;
                                break;
                            }
                            tail_phase ^= 1u << stage;
                        }
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t d = tmem + static_cast<uint32_t>((q & 1) * kBN);
                        auto mma = [&](int k) {
                            const uint64_t ad = ad0 + ((sa >> 4) + k * a_step), bd = bd0 + ((sb >> 4) + k * b_step);
                            if constexpr (kPair)
                                umma_bf16_pair(d, ad, bd, idesc, (in_chunk | k) != 0 ? 1u : 0u);
                            else
                                umma_bf16(d, ad, bd, idesc, (in_chunk | k) != 0 ? 1u : 0u);
                        };
                        if (steps == kBK / 16) {
#pragma unroll
                            for (int k = 0; k < kBK / 16; ++k) mma(k);
                        } else {
                            for (int k = 0; k < steps; ++k) mma(k);
                        }
                        commit<kPair>(smem_u32(&ctl->empty[stage]));
                        if (in_chunk + 1 == p.chunk || kb + 1 == t.kb1) commit<kPair>(smem_u32(&ctl->tfull[q & 1]));
                    }
                    __syncwarp();
                    if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
                    if (++in_chunk == p.chunk || kb + 1 == t.kb1) {
                        ++q;
                        in_chunk = 0;
                    }
                }
            }
            if (elect_one()) {                              // all issued MMAs complete before TMEM is released
                commit<kPair>(smem_u32(&ctl->drain));
                const long long t0 = clock64();
                while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && clock64() - t0 < kWaitCycles) {}
            }
        } else if (warp == kMmaWarp) {
            // the pair's second CTA: zeroes its part of each ragged last block
            if (kMode == kWgrad) {
                uint32_t tail_phase = 0;                    // by stage
                int64_t blocks = 0;                         // K blocks so far: the ring's position
                for (int u = unit; u < tiles; u += units) {
                    const Tile t = tile_at<kMode, kShape>(p, ctl, u);
                    blocks += t.kb1 - t.kb0;
                    if (t.kb1 == t.kb0 || t.kb1 * kBK <= t.depth) continue;
                    const int stage = static_cast<int>((blocks - 1) % G::kStages);
                    bool there = true;
                    if (lane == 0)
                        there = mbar_wait_bounded(smem_u32(&ctl->tail[stage]), tail_phase >> stage & 1u, abort_flag, p.err, 0x207);
                    if (!__shfl_sync(0xffffffffu, there, 0)) break;
                    tail_phase ^= 1u << stage;
                    __syncwarp();
                    zero_tail(smem_u32(smem + stage * G::kStageBytes), 2 + (t.nmma / 2 + 63) / 64, t.depth % kBK, lane);
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->tail_peer[stage]), 0));
                }
            }
            if (lane == 0) {                                // the leader's MMAs write this CTA's accumulators
                const long long t0 = clock64();
                while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && clock64() - t0 < kWaitCycles) {}
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t buf = smem_u32(smem + G::kStages * G::kStageBytes + warp * G::kOutBlocks * 32 * G::kOutRow);
        int block = 0;                                  // wgrad: the store block in turn
        if (kMode != kWgrad && p.splits == 1) {         // rows of no expert
            const int head = ctl->row[0], tail = ctl->row[p.experts];
            const int64_t extra = static_cast<int64_t>(head) + (p.rows - tail);
            for (int64_t r = blockIdx.x * kEpiWarps + warp; r < extra; r += static_cast<int64_t>(gridDim.x) * kEpiWarps) {
                const int64_t at = (r < head ? r : tail + (r - head)) * p.ldo;
                for (int c = lane; c < cols; c += 32) {
                    if (kF32)
                        static_cast<float*>(p.out)[at + c] = 0.f;
                    else
                        static_cast<bf16*>(p.out)[at + c] = __float2bfloat16_rn(0.f);
                }
            }
        }
        const uint32_t tempty_leader[2] = {kPair ? mapa_shared(smem_u32(&ctl->tempty[0]), 0) : 0u,
                                           kPair ? mapa_shared(smem_u32(&ctl->tempty[1]), 0) : 0u};
        bool ok = true;
        int q = 0;
        for (int u = unit; u < tiles && ok; u += units) {
            int chunks, nmma;
            {
                const Tile t = tile_at<kMode, kShape>(p, ctl, u);
                chunks = ceil_div_i(t.kb1 - t.kb0, p.chunk);
                nmma = t.nmma;
            }
            float v[4][32];                             // this lane's row of the warp's 32-column groups
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[g][j] = 0.f;
            for (int c = 0; c < chunks; ++c, ++q) {
                ok = mbar_wait_bounded(smem_u32(&ctl->tfull[q & 1]), (q >> 1) & 1, abort_flag, p.err, 0x204);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = kMode == kWgrad ? wgrad_column(half, g) : (2 * g + half) * 32;
                    if (col >= nmma) continue;          // warp-uniform
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                           static_cast<uint32_t>((q & 1) * kBN + col), r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[g][j] += __uint_as_float(r[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(smem_u32(&ctl->tempty[q & 1]));
                    else
                        mbar_arrive_cluster(tempty_leader[q & 1]);
                }
            }
            if (!ok) break;
            int again = u;                              // the tile's place once more: holding it over the sums spills registers
            asm volatile("" : "+r"(again));
            const Tile t = tile_at<kMode, kShape>(p, ctl, again);
            if (kAcc && t.depth == 0) continue;
            const int f = t.f0 + static_cast<int>(rank) * kBM + quarter * 32;
            if (f >= (kMode == kWgrad ? p.n : cols)) continue;
            if constexpr (kMode == kWgrad) {
                put_weights<kF32, kAcc, G::kOutRow, G::kOutBlocks>(p, t.split * p.experts + t.e, f, t.c0, t.cn, half, v, buf, block,
                                                             lane);
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = (2 * g + half) * 32;
                    if (col >= t.cn) continue;
                    put_tokens<kF32>(p, cols, f, static_cast<int64_t>(t.split) * p.rows + t.c0 + col, min(32, t.cn - col),
                                     v[g], buf, lane);
                }
            }
        }
        if (elect_one()) bulk_wait_all();               // no store still reads this CTA's shared memory
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();               // neither CTA leaves while the other may signal it
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (kPair)
            tmem_dealloc_pair(tmem, 512);
        else
            tmem_dealloc(tmem, 512);
    }
}

// Zeros for outputs that no sum reaches (k == 0 or n == 0 in a product, no rows at all in a weight gradient).
__global__ void __launch_bounds__(256) fill_zero_kernel(void* out, int out_f32, int64_t rows, int64_t cols, int64_t ld,
                                                        int64_t stride, int64_t total) {
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
        const int64_t r = i / cols, e = r / rows;
        const int64_t at = e * stride + (r - e * rows) * ld + (i - r * cols);
        if (out_f32)
            static_cast<float*>(out)[at] = 0.f;
        else
            static_cast<bf16*>(out)[at] = __float2bfloat16_rn(0.f);
    }
}

// Adds the parts of split sums in order: out (+)= sum_s part[s], four columns per
// thread.  Rows of no expert (forward, dgrad: row0 .. row1 hold the experts') are zeros.
struct JoinArgs {
    const float* part;             // [splits][rows][ld]
    void* out;
    const int32_t* offsets;        // null for a weight gradient
    int64_t rows, cols, ld, ldo, stride_o, matrix_rows;
    int32_t splits, out_f32, accumulate, experts;
};
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs p) {
    wait_for_previous();
    const int64_t groups = p.ld / 4, total = p.rows * groups;
    int64_t r0 = 0, r1 = p.rows;
    if (p.offsets != nullptr) {
        r0 = min(max(static_cast<int64_t>(p.offsets[0]), int64_t(0)), p.rows);
        r1 = min(max(static_cast<int64_t>(p.offsets[p.experts]), int64_t(0)), p.rows);
    }
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
        const int64_t r = i / groups, c = (i - r * groups) * 4, e = r / p.matrix_rows;
        const int64_t at = e * p.stride_o + (r - e * p.matrix_rows) * p.ldo + c;
        const int nv = static_cast<int>(min(p.cols - c, int64_t(4)));
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (r >= r0 && r < r1)
            for (int s = 0; s < p.splits; ++s) {
                // (an ordinary load: this kernel may start before the parts are written)
                const float4 x = *reinterpret_cast<const float4*>(p.part + (s * p.rows + r) * p.ld + c);
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= nv) continue;
            if (p.accumulate)
                v[k] += p.out_f32 ? static_cast<const float*>(p.out)[at + k]
                                  : __bfloat162float(static_cast<const bf16*>(p.out)[at + k]);
        }
        if (nv == 4) {                                  // rows start on 16-byte boundaries
            if (p.out_f32)
                store_run<float, 4>(static_cast<float*>(p.out) + at, v, true);
            else
                store_run<bf16, 4>(static_cast<bf16*>(p.out) + at, v, true);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= nv) continue;
                if (p.out_f32)
                    static_cast<float*>(p.out)[at + k] = v[k];
                else
                    static_cast<bf16*>(p.out)[at + k] = __float2bfloat16_rn(v[k]);
            }
        }
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encode() {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// `depth` matrices of rows x cols (one: a 2D view): boxes of box_rows x box_cols.
bool encode(CUtensorMap* map, const void* base, int dt, int64_t cols, int64_t rows, int64_t depth, int64_t ld,
            int64_t stride, int rank, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
    const size_t sz = op_elem_size(dt);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * sz), static_cast<cuuint64_t>((depth > 1 ? stride : ld) * sz)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return g_encode(map, dt == MO_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, step,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a call works on, before tensor maps.
struct Request {
    const void* a;                 // rows operand: X (forward), dY (dgrad, wgrad)
    int64_t lda;
    const void* b;                 // W, or X (wgrad)
    int64_t ldb, stride_b;
    void* out;
    int64_t ldo, stride_o;
    const int32_t* offsets;
    int64_t rows, n, k;
    int experts, out_dtype, accumulate;
};

// CTAs of one launch: one per SM, or as many pairs as the device holds at once.
template <int kMode, bool kF32, int kShape, bool kAcc>
cudaError_t prepare_expert(int* ctas) {
    static std::atomic<int> known[64];                  // by device ordinal; 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((*ctas = known[dev & 63].load()) > 0) return cudaSuccess;
    e = cudaFuncSetAttribute(expert_kernel<kMode, kF32, kShape, kAcc>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    *ctas = device_sm_count();
    if (kShape == kPairs) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(*ctas / 2 * 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int pairs = 0;
        e = cudaOccupancyMaxActiveClusters(&pairs, expert_kernel<kMode, kF32, kShape, kAcc>, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorInvalidConfiguration;
        *ctas = std::min(2 * pairs, *ctas / 2 * 2);
    }
    known[dev & 63].store(*ctas);
    return cudaSuccess;
}

template <int kMode, bool kF32, int kShape, bool kAcc = false>
cudaError_t launch_expert(const ExpertArgs& p, int64_t most_tiles, cudaStream_t s) {
    int ctas = 0;
    const cudaError_t e = prepare_expert<kMode, kF32, kShape, kAcc>(&ctas);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(most_tiles * (kShape == kPairs ? 2 : 1), ctas)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (kShape == kPairs) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, expert_kernel<kMode, kF32, kShape, kAcc>, p);
}

template <int kShape>
cudaError_t launch_product(int mode, bool f32, const ExpertArgs& p, int64_t tiles, cudaStream_t s) {
    if (mode == kFwd) return f32 ? launch_expert<kFwd, true, kShape>(p, tiles, s) : launch_expert<kFwd, false, kShape>(p, tiles, s);
    return f32 ? launch_expert<kDgrad, true, kShape>(p, tiles, s) : launch_expert<kDgrad, false, kShape>(p, tiles, s);
}
template <int kShape>
cudaError_t launch_wgrad(bool f32, bool acc, const ExpertArgs& p, int64_t tiles, cudaStream_t s) {
    if (acc)
        return f32 ? launch_expert<kWgrad, true, kShape, true>(p, tiles, s) : launch_expert<kWgrad, false, kShape, true>(p, tiles, s);
    return f32 ? launch_expert<kWgrad, true, kShape>(p, tiles, s) : launch_expert<kWgrad, false, kShape>(p, tiles, s);
}

// -1: chosen by the call's sizes; else a Shape (tests, measurements).
std::atomic<int> g_expert_shape{-1};

// A float32 result's sums leave TMEM every kF32Chunk K blocks (768 terms): the
// tensor core's accumulator drops bits below its last place, always towards zero,
// and adding the pieces in registers (to nearest) keeps that drift from growing
// with the sum.  Measured for a weight gradient over 2048 / 65536 rows (relative
// 2-norm error; plain float32: 3.9e-7 / 4.0e-7): 4 blocks 2.4e-7 / 3.7e-7, 8
// blocks 4.7e-7 / 5.1e-7, 12 blocks 6.7e-7 / 7.5e-7, 16 blocks 1.0e-6 / 1.0e-6,
// never 2.1e-6 / 7.6e-5.  Shorter pieces hold the MMAs up while the epilogue stores:
// 16384 rows, 8 experts of 4096 x 4096: 10 blocks 368 us, 12 blocks 340 us, 16 blocks 327 us.
constexpr int kF32Chunk = 12;
// A bf16 result's sums leave it every kBf16Chunk K blocks (4096 terms), which lose at most
// 256 x 2^-23, a hundredth of the result's own rounding.  Left there, the drift grows with the length:
// 2^20 positive terms came out 6.6e-3 too small on average, now 1.4e-5.  Pieces that long cost
// nothing that shows (16384 rows, 8 experts of 4096 x 11008, forward and dgrad 816 and 851 us before, 822 and 860 now
// in a run whose repeats differ by 20; 65536 rows of one 2048 x 2560 378 and 389, now 377 and 395).
constexpr int kBf16Chunk = 64;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxSide = int64_t(1) << 20;
constexpr size_t kExpertHeader = 256;      // the error word that mo_check_device_status reads

// How a call runs: on CTA pairs or single CTAs, and in how many parts each sum.
struct Plan {
    int shape;
    int splits;
};

// Tiles of a call at most (each expert may end in a tile of its own).
int64_t most_tiles(int mode, int64_t rows, int64_t n, int64_t k, int experts, int shape) {
    const int64_t features = shape_features(shape);
    if (mode == kWgrad) return experts * op_ceil_div(n, features) * op_ceil_div(k, kBN);
    return (rows / shape_columns(shape) + std::min<int64_t>(experts, rows)) * op_ceil_div(mode == kFwd ? n : k, features);
}

constexpr int64_t kSms = 152;
constexpr int64_t kShortSum = 256;         // rows per expert from which a weight gradient runs on pairs
constexpr int64_t kFewRows = 16;           // rows per expert up to which the weights set the time
constexpr int64_t kFewTiles = 228;         // narrow tiles of a product so small that more CTAs help it most
constexpr int64_t kSplitBlocks = 24;       // K blocks that a split has to take off a tile's time
constexpr int64_t kMinSplitBlocks = 4;     // K blocks of a part, at least

// Pairs halve the operand bytes per SM; a weight gradient over few rows is bound by
// its stores instead, which single CTAs issue faster; narrow tiles give small products
// more CTAs.  Measured (us, single / pair / narrow): forward of 16384 rows, 8 experts of
// 4096 x 4096 332 / 294 / -; 4096 rows, 16 experts of 2048 x 2048 44 / 39 / 140; 512 rows, 8
// experts of 1024 x 1024 9.9 / 10.1 / 9.1; 256 rows of one 768 x 768 9.3 / 9.7 / 7.2; 64
// rows, 8 experts of 4096 x 4096 49 / 46 / 47; 16 rows, 16 experts of 2048 x 1024 9.1 / 9.7 /
// 9.1 with the weights in L2.  Weight gradients, float32 and bf16, 16 experts of 2048 x
// 2048 over 1024 rows each 148 / 116 and 130 / 104, over 256 70 / 68 and 55 / 51, over
// 64 49 / 59 and 32 / 42.  The host knows the mean of the rows per expert only, and narrow tiles read an
// expert's weights once for every 32 tokens: 1024 rows, 64 experts of 2048 x 2048, evenly spread 96 / 91 / 88, all
// with one expert 18 / 18 / 42 (256 rows, 16 experts: 31 / 30 / 29 and 17 / 17 / 14).
// Where the tiles leave at least half of the SMs idle and the sums are long, each sum is
// split into parts that are joined in order afterwards (about 3 us more).
Plan plan_call(int mode, int64_t rows, int64_t n, int64_t k, int experts, int forced) {
    const int64_t depth = mode == kFwd ? k : mode == kDgrad ? n : op_ceil_div(rows, experts);
    const int64_t blocks = op_ceil_div(depth, kBK);
    Plan p;
    if (mode == kWgrad)
        p.shape = depth >= kShortSum ? kPairs : kSingle;
    else if (rows <= kFewRows * experts || most_tiles(mode, rows, n, k, experts, kFew) <= kFewTiles)
        p.shape = kFew;
    else
        p.shape = depth > 1024 || most_tiles(mode, rows, n, k, experts, kPairs) > 2 * (kSms / 2) ? kPairs : kSingle;
    if (forced >= 0) p.shape = mode == kWgrad && forced == kFew ? kSingle : forced;
    const int64_t tiles = most_tiles(mode, rows, n, k, experts, p.shape), units = p.shape == kPairs ? kSms / 2 : kSms;
    p.splits = 1;
    if (tiles > 0 && 2 * tiles <= units) {
        const int64_t s = std::min(units / tiles, blocks / kMinSplitBlocks);
        if (s >= 2 && blocks - op_ceil_div(blocks, s) >= kSplitBlocks) p.splits = static_cast<int>(s);
    }
    return p;
}

// Rows and row pitch of one part of a split call's output.
int64_t part_rows(int mode, int64_t rows, int64_t n, int experts) { return mode == kWgrad ? experts * n : rows; }
int64_t part_ld(int mode, int64_t n, int64_t k) { return op_ceil_div(mode == kFwd ? n : k, 4) * 4; }

size_t expert_ws_bytes(int64_t rows, int64_t n, int64_t k, int experts) {
    size_t most = 0;
    for (int mode = kFwd; mode <= kWgrad; ++mode)
        for (int forced = kSingle; forced <= kFew; ++forced) {
            const Plan p = plan_call(mode, rows, n, k, experts, forced);
            if (p.splits > 1)
                most = std::max(most, static_cast<size_t>(p.splits) * static_cast<size_t>(part_rows(mode, rows, n, experts)) *
                                          static_cast<size_t>(part_ld(mode, n, k)) * 4);
        }
    return kExpertHeader + op_align_up(most, 256);
}

int check_sizes(int64_t rows, int64_t n, int64_t k, int experts) {
    if (rows < 0 || n < 0 || k < 0 || experts < 1) return MO_ERR_INVALID_ARG;
    if (rows > kMaxRows || n > kMaxSide || k > kMaxSide || experts > kMaxExperts) return MO_ERR_UNSUPPORTED;
    return MO_OK;
}
// A matrix of `cols` columns; an absent one (no rows) needs no pointer.
int check_matrix(const void* p, int dt, int64_t cols, int64_t ld, bool used) {
    if (!used) return MO_OK;
    if (p == nullptr || ld < cols) return MO_ERR_INVALID_ARG;
    if (!op_aligned(p, 16) || (static_cast<size_t>(ld) * op_elem_size(dt)) % 16 != 0) return MO_ERR_ALIGNMENT;
    return MO_OK;
}
int check_stack(int dt, int64_t rows, int64_t ld, int64_t stride, int experts) {
    if (experts == 1) return MO_OK;
    if (stride < rows * ld) return MO_ERR_INVALID_ARG;
    if ((static_cast<size_t>(stride) * op_elem_size(dt)) % 16 != 0) return MO_ERR_ALIGNMENT;
    return MO_OK;
}

int run_expert(int mode, const Request& q, void* ws, size_t ws_bytes, mo_stream_t stream) {
    if (q.offsets == nullptr) return MO_ERR_INVALID_ARG;
    if (!op_aligned(q.offsets, 4)) return MO_ERR_ALIGNMENT;
    const int st = op_check_ws(ws, ws_bytes, expert_ws_bytes(q.rows, q.n, q.k, q.experts));
    if (st != MO_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t cols = mode == kFwd ? q.n : q.k;      // of the output
    const int64_t depth = mode == kFwd ? q.k : mode == kDgrad ? q.n : q.rows;
    if (depth == 0) {
        if (q.accumulate) return MO_OK;
        const int64_t rows = mode == kWgrad ? q.n : q.rows, total = rows * cols * (mode == kWgrad ? q.experts : 1);
        return op_status(op_traced(MO_K_EXPERT + mode, s, [&] {
            fill_zero_kernel<<<static_cast<unsigned>(std::min<int64_t>(op_ceil_div(total, 256), 16384)), 256, 0, s>>>(
                q.out, q.out_dtype == MO_F32, rows, cols, q.ldo, q.stride_o, total);
            return cudaGetLastError();
        }));
    }
    if (!get_encode()) return MO_ERR_CUDA;
    const Plan plan = plan_call(mode, q.rows, q.n, q.k, q.experts, g_expert_shape.load());
    const bool pair = plan.shape == kPairs;
    const bool split = plan.splits > 1;
    const bool f32 = split || q.out_dtype == MO_F32;    // of what the product kernel writes
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kExpertHeader);
    const int64_t rows_part = part_rows(mode, q.rows, q.n, q.experts), ld_part = part_ld(mode, q.n, q.k);
    void* out = split ? parts : q.out;
    const int out_dtype = f32 ? MO_F32 : MO_BF16;
    const int64_t ldo = split ? ld_part : q.ldo, stride_o = split ? q.n * ld_part : q.stride_o;
    ExpertArgs p;
    const int64_t features = shape_features(plan.shape), tk = op_ceil_div(q.k, kBN);
    // a group's rows take at most 40 MB of L2 (groups of 8 tiles, 16 MB at 4096 columns,
    // read the weights of an expert with 15 tiles twice: 16384 rows over 8 ragged
    // experts of 11008 x 4096 923 us)
    p.group = static_cast<int32_t>(std::max<int64_t>(4, std::min<int64_t>(64, (40 << 20) / (kBN * 2 * depth))));
    p.f_tiles = static_cast<int32_t>(op_ceil_div(mode == kWgrad ? q.n : cols, features));
    // equal tiles of at most kBN columns, in whole store blocks (a block that reached past its tile would overwrite the next one)
    p.width = static_cast<int32_t>(op_ceil_div(op_ceil_div(q.k, tk), 64) * 64);
    p.c_tiles = static_cast<int32_t>(op_ceil_div(q.k, p.width));
    const int64_t tiles = most_tiles(mode, q.rows, q.n, q.k, q.experts, plan.shape) * plan.splits;
    if (tiles > INT32_MAX) return MO_ERR_UNSUPPORTED;
    bool ok;
    constexpr auto k128 = CU_TENSOR_MAP_SWIZZLE_128B;
    if (mode == kWgrad) {
        ok = encode(&p.a, q.a, MO_BF16, q.n, q.rows, 1, q.lda, 0, 2, 64, 64, k128) &&
             encode(&p.b[0], q.b, MO_BF16, q.k, q.rows, 1, q.ldb, 0, 2, 64, 64, k128) &&
             encode(&p.o, out, out_dtype, q.k, q.n, static_cast<int64_t>(q.experts) * plan.splits, ldo, stride_o, 3,
                    (pair ? 64 : 128) / (f32 ? 4 : 2), 32, pair ? CU_TENSOR_MAP_SWIZZLE_64B : k128);
        for (int i = 1; i < kBoxes; ++i) p.b[i] = p.b[0];
    } else {
        ok = encode(&p.a, q.b, MO_BF16, q.k, q.n, q.experts, q.ldb, q.stride_b, 3, 64, mode == kFwd ? 128 : 64, k128) &&
             encode(&p.o, out, out_dtype, cols, q.rows * plan.splits, 1, ldo, 0, 2, 32, f32 ? 16 : 32,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
        for (int i = kBoxes - 1; i >= 0; --i) {         // (boxes that no tile of these rows or this shape takes: not encoded)
            if ((128 >> i) > shape_columns(plan.shape) || ((128 >> i) >= 32 && (128 >> i) >= 2 * q.rows))
                p.b[i] = p.b[i + 1];
            else
                ok = ok && encode(&p.b[i], q.a, MO_BF16, depth, q.rows, 1, q.lda, 0, 2, 64, 128 >> i, k128);
        }
    }
    if (!ok) return MO_ERR_UNSUPPORTED;                 // a stride past what a tensor map holds (2^40 bytes)
    p.offsets = q.offsets;
    p.out = out;
    p.ldo = ldo;
    p.stride_o = stride_o;
    p.rows = static_cast<int32_t>(q.rows);
    p.n = static_cast<int32_t>(q.n);
    p.k = static_cast<int32_t>(q.k);
    p.experts = q.experts;
    p.splits = plan.splits;
    p.chunk = f32 ? kF32Chunk : kBf16Chunk;
    p.err = static_cast<int*>(ws);
    return op_status(op_traced(MO_K_EXPERT + mode, s, [&] {
        const bool acc = !split && q.accumulate;        // (split: the join adds)
        cudaError_t e;
        if (mode == kWgrad)
            e = pair ? launch_wgrad<kPairs>(f32, acc, p, tiles, s) : launch_wgrad<kSingle>(f32, acc, p, tiles, s);
        else
            e = pair                   ? launch_product<kPairs>(mode, f32, p, tiles, s)
                : plan.shape == kFew ? launch_product<kFew>(mode, f32, p, tiles, s)
                                       : launch_product<kSingle>(mode, f32, p, tiles, s);
        if (e != cudaSuccess || !split) return e;
        JoinArgs j;
        j.part = parts;
        j.out = q.out;
        j.offsets = mode == kWgrad ? nullptr : q.offsets;
        j.rows = rows_part;
        j.cols = cols;
        j.ld = ld_part;
        j.ldo = q.ldo;
        j.stride_o = q.stride_o;
        j.matrix_rows = mode == kWgrad ? q.n : q.rows;
        j.splits = plan.splits;
        j.out_f32 = q.out_dtype == MO_F32;
        j.accumulate = q.accumulate;
        j.experts = q.experts;
        const int64_t blocks = op_ceil_div(rows_part * (ld_part / 4), 256);
        return launch_after(join_kernel, static_cast<unsigned>(std::min<int64_t>(blocks, 8 * kSms)), 256, s, j);
    }));
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int mo_debug_set_expert_shape(int shape) {
    if (shape < -1 || shape > kFew) return MO_ERR_INVALID_ARG;
    return g_expert_shape.exchange(shape) + 1;
}

int expert_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k, int experts, size_t* bytes_out) {
    if (bytes_out == nullptr) return MO_ERR_INVALID_ARG;
    const int st = check_sizes(rows, n, k, experts);
    if (st == MO_OK) *bytes_out = expert_ws_bytes(rows, n, k, experts);
    return st;
}

int expert_linear(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t stride_w, const int32_t* offsets,
                  int64_t rows, int64_t n, int64_t k, int experts, void* Y, int y_dtype, int64_t ldy, void* ws,
                  size_t ws_bytes, mo_stream_t stream) {
    int st = check_sizes(rows, n, k, experts);
    if (st != MO_OK) return st;
    if (!op_valid_dtype(y_dtype)) return MO_ERR_INVALID_ARG;
    if (rows == 0 || n == 0) return MO_OK;
    if ((st = check_matrix(X, MO_BF16, k, ldx, k > 0)) != MO_OK) return st;
    if ((st = check_matrix(W, MO_BF16, k, ldw, k > 0)) != MO_OK) return st;
    if ((st = check_stack(MO_BF16, n, ldw, stride_w, experts)) != MO_OK) return st;
    if ((st = check_matrix(Y, y_dtype, n, ldy, true)) != MO_OK) return st;
    const Request a = {X, ldx, W, ldw, stride_w, Y, ldy, 0,
                          offsets, rows, n, k, experts, y_dtype, 0};
    return run_expert(kFwd, a, ws, ws_bytes, stream);
}

int expert_linear_dgrad(const void* dY, int64_t ldy, const void* W, int64_t ldw, int64_t stride_w,
                        const int32_t* offsets, int64_t rows, int64_t n, int64_t k, int experts, void* dX,
                        int dx_dtype, int64_t ldx, void* ws, size_t ws_bytes, mo_stream_t stream) {
    int st = check_sizes(rows, n, k, experts);
    if (st != MO_OK) return st;
    if (!op_valid_dtype(dx_dtype)) return MO_ERR_INVALID_ARG;
    if (rows == 0 || k == 0) return MO_OK;
    if ((st = check_matrix(dY, MO_BF16, n, ldy, n > 0)) != MO_OK) return st;
    if ((st = check_matrix(W, MO_BF16, k, ldw, n > 0)) != MO_OK) return st;
    if ((st = check_stack(MO_BF16, n, ldw, stride_w, experts)) != MO_OK) return st;
    if ((st = check_matrix(dX, dx_dtype, k, ldx, true)) != MO_OK) return st;
    const Request a = {dY, ldy, W, ldw, stride_w, dX, ldx, 0,
                          offsets, rows, n, k, experts, dx_dtype, 0};
    return run_expert(kDgrad, a, ws, ws_bytes, stream);
}

int expert_linear_wgrad(const void* dY, int64_t ldy, const void* X, int64_t ldx, const int32_t* offsets,
                        int64_t rows, int64_t n, int64_t k, int experts, void* dW, int dw_dtype, int64_t lddw,
                        int64_t stride_dw, int accumulate, void* ws, size_t ws_bytes, mo_stream_t stream) {
    int st = check_sizes(rows, n, k, experts);
    if (st != MO_OK) return st;
    if (!op_valid_dtype(dw_dtype) || (accumulate != 0 && accumulate != 1)) return MO_ERR_INVALID_ARG;
    if (n == 0 || k == 0) return MO_OK;
    if ((st = check_matrix(dY, MO_BF16, n, ldy, rows > 0)) != MO_OK) return st;
    if ((st = check_matrix(X, MO_BF16, k, ldx, rows > 0)) != MO_OK) return st;
    if ((st = check_matrix(dW, dw_dtype, k, lddw, true)) != MO_OK) return st;
    if ((st = check_stack(dw_dtype, n, lddw, stride_dw, experts)) != MO_OK) return st;
    const Request a = {dY, ldy, X, ldx, 0, dW, lddw, stride_dw,
                          offsets, rows, n, k, experts, dw_dtype, accumulate};
    return run_expert(kWgrad, a, ws, ws_bytes, stream);
}

}  // extern "C"
