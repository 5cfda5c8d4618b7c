// AdamW over many tensors in one launch, states in float32 or in 8 bits.
//
// The tensors' descriptors travel in the kernel's parameters (no copy, no
// workspace; a captured graph holds them).  Tensors are cut into tiles, numbered
// through; a block walks tiles a grid apart and finds each one's
// tensor by bisection.  A warp takes 256 neighbouring values at a time, eight to a
// lane: one block of the 8-bit states, whose largest value is a maximum over the warp.
//
// Float32 states are bound by their bytes (22 to 28 a value with bf16 or float32 weights and gradients).  8-bit ones are near the
// point where instructions count as much: 16 bytes a value allow about 90.
#include <cmath>

#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 4;
constexpr int kBlockValues = 256;                  // values of one scale
// Blocks of a tile: two to a warp with 8-bit states (one: 560 us instead of 531 for 173 million
// values), one with float32 states (two: 210 us instead of 194 for 53 million, the last tiles being larger).
__host__ __device__ __forceinline__ int tile_blocks(int state_dtype) { return state_dtype == MO_F32 ? kWarps : 2 * kWarps; }

struct Desc {
    int64_t numel;
    void* W;
    const void* g;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    float lr, decay;
    int32_t w_dtype, g_dtype, state_dtype, wide;
    int32_t index;                                  // in the caller's list
    int32_t reserved;
    int64_t tile0;                                  // first tile, counted over the launch's tensors
};

struct Common {
    float beta1, beta2, one_minus1, one_minus2, eps, grad_scale, inv_bc1, inv_bc2;
    const int64_t* step_ptr;
    const float* grad_mul;
    uint32_t key;                                   // hash of seed and step
    uint32_t seed_key;                              // hash of seed, for step_ptr
    int32_t dither, count;
    int64_t tiles;
};

template <int N>
struct Launch {
    Common c;
    Desc d[N];
};

// A 32-bit hash by multiplication and xor-shift; the factors are 2^32 over the golden
// ratio and 2^32 over the square root of 2, both odd.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
    h *= 0x9E3779B1u;
    h = (h ^ (h >> 16)) * 0xB504F333u;
    h = (h ^ (h >> 15)) * 0x9E3779B1u;
    return h ^ (h >> 16);
}

// Eight neighbouring values.  kFull: all of them there, on their natural boundary of 16 bytes
// (8 for codes); else the first `valid`, one by one.
template <bool kFull, typename T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&v)[8]) {
    constexpr int kW = Elem<T>::kVec;
    if (kFull) {
#pragma unroll
        for (int q = 0; q < 8 / kW; ++q) {
            float w[kW];
            unpack16(reinterpret_cast<const uint4*>(p)[q], w);
#pragma unroll
            for (int i = 0; i < kW; ++i) v[q * kW + i] = w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? Elem<T>::to_float(p[i]) : 0.f;
    }
}
template <bool kFull, typename T>
__device__ __forceinline__ void store8(T* p, int valid, const float (&v)[8]) {
    if (kFull) {
        store_run<T, 8>(p, v, true);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = Elem<T>::from_float(v[i]);
    }
}
template <bool kFull>
__device__ __forceinline__ void load8(const void* p, int dt, int64_t at, int valid, float (&v)[8]) {
    if (dt == MO_F32)
        load8<kFull>(static_cast<const float*>(p) + at, valid, v);
    else
        load8<kFull>(static_cast<const bf16*>(p) + at, valid, v);
}
template <bool kFull>
__device__ __forceinline__ void store8(void* p, int dt, int64_t at, int valid, const float (&v)[8]) {
    if (dt == MO_F32)
        store8<kFull>(static_cast<float*>(p) + at, valid, v);
    else
        store8<kFull>(static_cast<bf16*>(p) + at, valid, v);
}

// Two e4m3 codes to floats and back (to nearest, ties to even).
__device__ __forceinline__ void from_e4m3x2(uint32_t codes, float& a, float& b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(a), "=f"(b) : "r"(h));
}
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
    return c;
}

template <bool kFull>
__device__ __forceinline__ void load_codes(const void* p, int64_t at, int valid, float scale, float (&v)[8]) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + at;
    uint2 u = make_uint2(0, 0);
    if (kFull) {
        u = *reinterpret_cast<const uint2*>(q);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < valid) u.x |= static_cast<uint32_t>(q[i]) << (8 * i);
            if (i + 4 < valid) u.y |= static_cast<uint32_t>(q[i + 4]) << (8 * i);
        }
    }
    from_e4m3x2(u.x & 0xFFFF, v[0], v[1]);
    from_e4m3x2(u.x >> 16, v[2], v[3]);
    from_e4m3x2(u.y & 0xFFFF, v[4], v[5]);
    from_e4m3x2(u.y >> 16, v[6], v[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], scale);
}

// A value of |t| < 2^-6, where e4m3 values are 2^-9 apart: to nearest by the conversion
// itself, or below or above by 16 random bits.  kLeast: what is positive stays positive.
template <bool kLeast, bool kDither>
__device__ __noinline__ float small_value(float t, uint32_t bits) {
    if (kDither) {
        const float a = fabsf(t);
        t = copysignf(floorf(__fadd_rn(a * 512.f, static_cast<float>(bits) * 0x1p-16f)) * 0x1p-9f, t);
    }
    return kLeast ? fmaxf(t, 0x1p-9f) : t;
}

// The block's values (eight of them here) as e4m3 codes and a scale.  A dithered value from
// 2^-6 on is the one below (the 20 low bits of its mantissa fall away) or above, by a carry
// out of those bits when the random ones, the low half of `bits` (kLow) or the high, are added.
template <bool kLeast, bool kLow, bool kDither, bool kFull>
__device__ __forceinline__ void store_codes(void* p, float* scale, int64_t at, int valid, const uint32_t (&bits)[8],
                                            const float (&x)[8]) {
    uint32_t most = 0, least = 0xFFFFFFFFu;          // of the magnitudes as integers; infinity and NaN above all others, and 0 left aside
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        most = max(most, a);
        least = min(least, a - 1);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    const bool finite = most < 0x7F800000u, some = most >= 0x00800000u;              // 2^-126
    const float top = __uint_as_float(most);
    const float inv = some ? __frcp_rn(top) : 0.f;
    float t[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = __fmul_rn(__fmul_rn(x[i], inv), 448.f);
        if (kDither) {
            const uint32_t add = kLow ? bits[i] & 0xFFFFu : bits[i] >> 16;
            r[i] = __uint_as_float((__float_as_uint(t[i]) + (add << 4)) & 0xFFF00000u);
        } else {
            r[i] = t[i];
        }
    }
    // |t| < 2^-6 means |x| < 3.5e-5 top: about one value in ten thousand
    if (least <= __float_as_uint(top * (0x1.01p-6f / 448.f))) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(t[i]) < 0x1p-6f && t[i] != 0.f)
                r[i] = small_value<kLeast, kDither>(t[i], kLow ? bits[i] & 0xFFFFu : bits[i] >> 16);
    }
    uint2 u;
    u.x = to_e4m3x2(r[0], r[1]) | to_e4m3x2(r[2], r[3]) << 16;
    u.y = to_e4m3x2(r[4], r[5]) | to_e4m3x2(r[6], r[7]) << 16;
    if (!finite) u = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    uint8_t* q = static_cast<uint8_t*>(p) + at;
    if (kFull) {
        *reinterpret_cast<uint2*>(q) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < valid) q[i] = static_cast<uint8_t>(u.x >> (8 * i));
            if (i + 4 < valid) q[i + 4] = static_cast<uint8_t>(u.y >> (8 * i));
        }
    }
    if ((threadIdx.x & 31) == 0) *scale = finite ? (some ? __fmul_rn(top, 1.f / 448.f) : 0.f) : NAN;
}

struct Step {
    float beta1, beta2, one_minus1, one_minus2, eps, scale, root_inv_bc2, lr, decay;   // lr over its bias correction
    uint32_t key;
};

// A lane's eight values from `at` on, in block `block` of the tensor.
template <bool kCodes, bool kDither, bool kFull>
__device__ __forceinline__ void step_values(const Desc& d, const Step& c, int64_t block, int64_t at, int valid) {
    float w[8], g[8], m[8], v[8], root[8];           // root: of v, what the 8-bit state holds, and the update needs
    load8<kFull>(d.W, d.w_dtype, at, valid, w);
    load8<kFull>(d.g, d.g_dtype, at, valid, g);
    if (kCodes) {
        load_codes<kFull>(d.m, at, valid, d.m_scale[block], m);
        load_codes<kFull>(d.v, at, valid, d.v_scale[block], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
    } else {
        load8<kFull>(static_cast<const float*>(d.m) + at, valid, m);
        load8<kFull>(static_cast<const float*>(d.v) + at, valid, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = __fmul_rn(g[i], c.scale);
        m[i] = __fadd_rn(__fmul_rn(c.beta1, m[i]), __fmul_rn(c.one_minus1, gi));
        v[i] = __fadd_rn(__fmul_rn(c.beta2, v[i]), __fmul_rn(c.one_minus2, __fmul_rn(gi, gi)));
        root[i] = __fsqrt_rn(v[i]);
        const float denom = fmaf(root[i], c.root_inv_bc2, c.eps);
        w[i] = w[i] - c.decay * w[i] - c.lr * __fdividef(m[i], denom);                 // (denom below 2^126, or infinite with v: within 2 u)
    }
    store8<kFull>(d.W, d.w_dtype, at, valid, w);
    if (kCodes) {
        uint32_t bits[8] = {};
        if (kDither) {
#pragma unroll
            for (int i = 0; i < 8; ++i) bits[i] = mix(static_cast<uint32_t>(at + i) ^ c.key);
        }
        store_codes<false, true, kDither, kFull>(d.m, d.m_scale + block, at, valid, bits, m);
        store_codes<true, false, kDither, kFull>(d.v, d.v_scale + block, at, valid, bits, root);
    } else {
        store8<kFull>(static_cast<float*>(d.m) + at, valid, m);
        store8<kFull>(static_cast<float*>(d.v) + at, valid, v);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) adamw_batch_kernel(const __grid_constant__ Launch<N> a) {
    __shared__ float s_bc[2];
    const Common& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float inv_bc1 = c.inv_bc1, inv_bc2 = c.inv_bc2;
    uint32_t key = c.key;
    if (c.step_ptr != nullptr) {
        const int64_t step = *c.step_ptr;
        if (threadIdx.x < 2) {
            const double beta = threadIdx.x == 0 ? c.beta1 : c.beta2;
            s_bc[threadIdx.x] = static_cast<float>(1.0 / (1.0 - pow(beta, static_cast<double>(step))));
        }
        __syncthreads();
        inv_bc1 = s_bc[0];
        inv_bc2 = s_bc[1];
        key = mix(c.seed_key + static_cast<uint32_t>(step));
    }
    Step step;
    step.beta1 = c.beta1;
    step.beta2 = c.beta2;
    step.one_minus1 = c.one_minus1;
    step.one_minus2 = c.one_minus2;
    step.eps = c.eps;
    step.scale = c.grad_mul != nullptr ? c.grad_scale * *c.grad_mul : c.grad_scale;
    step.root_inv_bc2 = sqrtf(inv_bc2);

    for (int64_t tile = blockIdx.x; tile < c.tiles; tile += gridDim.x) {
        int lo = 0, hi = c.count;                   // the last tensor that begins at or before the tile
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.d[mid].tile0 <= tile) lo = mid; else hi = mid;
        }
        const Desc& d = a.d[lo];
        step.lr = d.lr * inv_bc1;
        step.decay = d.decay;
        step.key = mix(key + static_cast<uint32_t>(d.index));
        const bool codes = d.state_dtype != MO_F32, dither = c.dither != 0;
        const int blocks = tile_blocks(d.state_dtype);
        for (int k = warp; k < blocks; k += kWarps) {
            const int64_t block = (tile - d.tile0) * blocks + k, begin = block * kBlockValues, at = begin + lane * 8;
            const int64_t left = d.numel - begin;
            if (left <= 0) break;                   // (the whole warp)
            if (d.wide && left >= kBlockValues) {
                if (!codes)
                    step_values<false, false, true>(d, step, block, at, 8);
                else if (dither)
                    step_values<true, true, true>(d, step, block, at, 8);
                else
                    step_values<true, false, true>(d, step, block, at, 8);
            } else {
                const int valid = static_cast<int>(max(int64_t(0), min(int64_t(8), left - lane * 8)));
                if (!codes)
                    step_values<false, false, false>(d, step, block, at, valid);
                else if (dither)
                    step_values<true, true, false>(d, step, block, at, valid);
                else
                    step_values<true, false, false>(d, step, block, at, valid);
            }
        }
    }
}

template <int N>
cudaError_t launch_batch(const Common& common, const Desc* d, int count, int64_t tiles, cudaStream_t s) {
    Launch<N> a;
    a.c = common;
    a.c.count = count;
    a.c.tiles = tiles;
    for (int i = 0; i < count; ++i) a.d[i] = d[i];
    const int64_t most = static_cast<int64_t>(device_sm_count()) * kBlocksPerSm;
    adamw_batch_kernel<N><<<static_cast<unsigned>(tiles < most ? tiles : most), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

constexpr int kFew = 8, kSome = 64, kMany = 320;   // descriptors of a launch; 320 fill the 32 KB of parameters
constexpr int64_t kMaxNumel = int64_t(1) << 40;
// The update divides by __fdividef, which gives 0 for a divisor above 2^126.  sqrt(v / (1 - beta2^t)) is below 2^76
// (v below 2^128, 1 - beta2 at least 2^-24), so that with such an eps the divisor stays below 2^126.
constexpr float kMaxEps = 0x1p125f;

int check_tensor(const mo_adamw_tensor& t) {
    const bool small = t.state_dtype == MO_E4M3;
    if (t.numel < 0 || !op_valid_dtype(t.w_dtype) || !op_valid_dtype(t.g_dtype) || (t.state_dtype != MO_F32 && !small))
        return MO_ERR_INVALID_ARG;
    if (t.numel == 0) return MO_OK;
    if (t.W == nullptr || t.g == nullptr || t.m == nullptr || t.v == nullptr ||
        (small && (t.m_scale == nullptr || t.v_scale == nullptr)))
        return MO_ERR_INVALID_ARG;
    if (t.numel >= kMaxNumel) return MO_ERR_UNSUPPORTED;
    const size_t state = small ? 1 : 4;
    if (!op_aligned(t.W, op_elem_size(t.w_dtype)) || !op_aligned(t.g, op_elem_size(t.g_dtype)) ||
        !op_aligned(t.m, state) || !op_aligned(t.v, state) ||
        (small && (!op_aligned(t.m_scale, 4) || !op_aligned(t.v_scale, 4))))
        return MO_ERR_ALIGNMENT;
    return MO_OK;
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" int adamw_step_batched(const mo_adamw_tensor* tensors, int count, const mo_adamw_cfg* cfg,
                                  mo_stream_t stream) {
    if (count < 0 || cfg == nullptr || (count > 0 && tensors == nullptr) || (cfg->dither != 0 && cfg->dither != 1) ||
        !(cfg->beta1 >= 0.f && cfg->beta1 < 1.f) || !(cfg->beta2 >= 0.f && cfg->beta2 < 1.f) ||
        !(cfg->eps >= 0.f && cfg->eps <= kMaxEps) ||
        (cfg->step_ptr == nullptr && cfg->step < 1))
        return MO_ERR_INVALID_ARG;
    if (!op_aligned(cfg->step_ptr, 8) || !op_aligned(cfg->grad_mul, 4)) return MO_ERR_ALIGNMENT;
    for (int i = 0; i < count; ++i) {
        const int st = check_tensor(tensors[i]);
        if (st != MO_OK) return st;
    }
    Common c = {};
    c.beta1 = cfg->beta1;
    c.beta2 = cfg->beta2;
    c.one_minus1 = 1.f - cfg->beta1;               // (exact from beta = 0.5 on)
    c.one_minus2 = 1.f - cfg->beta2;
    c.eps = cfg->eps;
    c.grad_scale = cfg->grad_scale;
    c.step_ptr = cfg->step_ptr;
    c.grad_mul = cfg->grad_mul;
    c.dither = cfg->dither;
    c.seed_key = mix(cfg->seed);
    if (cfg->step_ptr == nullptr) {
        const double t = static_cast<double>(cfg->step);
        c.inv_bc1 = static_cast<float>(1.0 / (1.0 - pow(static_cast<double>(cfg->beta1), t)));
        c.inv_bc2 = static_cast<float>(1.0 / (1.0 - pow(static_cast<double>(cfg->beta2), t)));
        c.key = mix(c.seed_key + static_cast<uint32_t>(cfg->step));
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_ADAMW_BATCH, s, [&] {
        Desc d[kMany];
        int held = 0;
        int64_t tiles = 0;
        auto flush = [&] {
            cudaError_t e = cudaSuccess;
            if (held > kSome)
                e = launch_batch<kMany>(c, d, held, tiles, s);
            else if (held > kFew)
                e = launch_batch<kSome>(c, d, held, tiles, s);
            else if (held > 0)
                e = launch_batch<kFew>(c, d, held, tiles, s);
            held = 0;
            tiles = 0;
            return e;
        };
        for (int i = 0; i < count; ++i) {
            const mo_adamw_tensor& t = tensors[i];
            if (t.numel == 0) continue;
            Desc& o = d[held++];
            const bool small = t.state_dtype == MO_E4M3;
            o.numel = t.numel;
            o.W = t.W;
            o.g = t.g;
            o.m = t.m;
            o.v = t.v;
            o.m_scale = t.m_scale;
            o.v_scale = t.v_scale;
            o.lr = t.lr;
            o.decay = static_cast<float>(static_cast<double>(t.lr) * t.weight_decay);
            o.w_dtype = t.w_dtype;
            o.g_dtype = t.g_dtype;
            o.state_dtype = t.state_dtype;
            o.wide = op_aligned(t.W, 16) && op_aligned(t.g, 16) && op_aligned(t.m, small ? 8 : 16) &&
                     op_aligned(t.v, small ? 8 : 16);
            o.index = i;
            o.reserved = 0;
            o.tile0 = tiles;
            tiles += op_ceil_div(t.numel, tile_blocks(t.state_dtype) * kBlockValues);
            if (held == kMany) {
                const cudaError_t e = flush();
                if (e != cudaSuccess) return e;
            }
        }
        return flush();
    }));
}
