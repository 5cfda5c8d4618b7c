// Shared by the training-step operators (embedding, expert products,
// distillation): element access of either type, wide accesses at any
// alignment, and the host-side argument checks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/matrixopt.h"
#include "../../include/matrixopt_debug.h"

namespace mo {

// ------------------------------------------------------------------ host side
inline size_t op_align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t op_ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t op_elem_size(int dt) { return dt == MO_F32 ? 4 : 2; }
inline bool op_valid_dtype(int dt) { return dt == MO_F32 || dt == MO_BF16; }
inline size_t op_id_size(int dt) { return dt == MO_I32 ? 4 : 8; }
inline bool op_valid_id_dtype(int dt) { return dt == MO_I32 || dt == MO_I64; }
inline bool op_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int op_check_ws(const void* ws, size_t have, size_t need) {
    return ws == nullptr || !op_aligned(ws, 256) || have < need ? MO_ERR_WORKSPACE : MO_OK;
}
inline int op_status(cudaError_t e) { return e == cudaSuccess ? MO_OK : MO_ERR_CUDA; }

// Records a CUDA event pair around a launch when the caller's thread traces
// (mo_trace_enable); defined beside the trace itself.
bool trace_begin(cudaStream_t s);
bool trace_end(int kind, cudaStream_t s);
int device_sm_count();

template <typename F>
cudaError_t op_traced(int kind, cudaStream_t s, F&& launch) {
    if (!trace_begin(s)) return cudaErrorUnknown;
    const cudaError_t e = launch();
    if (e != cudaSuccess) return e;
    return trace_end(kind, s) ? cudaSuccess : cudaErrorUnknown;
}

// Kernels of one call that follow each other: the later one's launch overlaps
// the earlier one's end (programmatic dependent launch).  The earlier kernel calls
// launch_dependents() when it starts, the later one wait_for_previous() before its
// first access to anything that the earlier one writes or reads.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- device side
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;                 // elements of one 16-byte access
    __device__ static float to_float(float x) { return x; }
    __device__ static float from_float(float x) { return x; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    // the one rounding of a result, to nearest even
    __device__ static __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// V consecutive floats to V elements of type D: 16-byte stores where `wide`
// (the address is 16-byte aligned and V a multiple of one access), else
// element by element.
template <typename D, int V>
__device__ __forceinline__ void store_run(D* p, const float (&v)[V], bool wide) {
    constexpr int kW = Elem<D>::kVec;
    if (wide && V % kW == 0) {
#pragma unroll
        for (int q = 0; q < V / kW; ++q) {
            float w[kW];
#pragma unroll
            for (int k = 0; k < kW; ++k) w[k] = v[(q * kW + k) % V];
            reinterpret_cast<uint4*>(p)[q] = pack16(w);
        }
    } else if (wide && V == 4 && kW == 8) {        // four bf16: one 8-byte store
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2 % V], v[3 % V]);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) p[k] = Elem<D>::from_float(v[k]);
    }
}

// A token id of either type; -1 stands for any id outside [0, vocab).
__device__ __forceinline__ int64_t load_id(const void* ids, int id_dtype, int64_t i, int64_t vocab) {
    const int64_t v = id_dtype == MO_I32 ? static_cast<const int32_t*>(ids)[i] : static_cast<const int64_t*>(ids)[i];
    return v >= 0 && v < vocab ? v : -1;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace mo
