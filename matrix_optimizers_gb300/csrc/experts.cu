// Matrix products grouped by expert: rows sorted by expert, expert e holding
// rows offsets[e] .. offsets[e + 1] - 1.
//   forward  Y[r, :]  = X[r, :] W_e^T
//   dgrad    dX[r, :] = dY[r, :] W_e
//   wgrad    dW_e (+)= sum_r dY[r, :]^T X[r, :]
#include <algorithm>

#include "train_common.cuh"

namespace mo {

using bf16 = __nv_bfloat16;

namespace {

enum ExpertMode { kFwd = 0, kDgrad = 1, kWgrad = 2 };

struct ExpertArgs {
    const bf16* rows_a;      // X (forward), dY (dgrad, wgrad)
    int64_t lda;
    const bf16* b;           // W, or X (wgrad)
    int64_t ldb, stride_b;
    void* out;
    int64_t ldo, stride_o;
    const int32_t* offsets;
    int64_t rows, n, k;
    int experts, out_dtype, accumulate;
};

// First row of expert e, held inside [0, rows] whatever the caller's array says.
__device__ __forceinline__ int64_t row_begin(const ExpertArgs& a, int e) {
    const int64_t o = a.offsets[e];
    return o < 0 ? 0 : o > a.rows ? a.rows : o;
}

constexpr int kT = 64, kTK = 16;

// 64 x 64 tile of out[i, j] = sum_k A(i, k) B(j, k).
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(FA&& fa, FB&& fb, int64_t depth, float (&acc)[4][4]) {
    __shared__ float sa[kTK][kT + 1], sb[kTK][kT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t k0 = 0; k0 < depth; k0 += kTK) {
        for (int q = threadIdx.x; q < kT * kTK; q += 256) {
            const int i = q / kTK, k = q % kTK;
            sa[k][i] = k0 + k < depth ? fa(i, k0 + k) : 0.f;
            sb[k][i] = k0 + k < depth ? fb(i, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

__device__ __forceinline__ void put(const ExpertArgs& a, int64_t at, float v) {
    if (a.out_dtype == MO_F32) {
        float* p = static_cast<float*>(a.out) + at;
        *p = a.accumulate ? *p + v : v;
    } else {
        bf16* p = static_cast<bf16*>(a.out) + at;
        *p = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*p) + v : v);
    }
}

template <int kMode>
__global__ void __launch_bounds__(256) expert_kernel(const __grid_constant__ ExpertArgs a) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t cols = kMode == kFwd ? a.n : a.k, col0 = static_cast<int64_t>(blockIdx.x) * kT;
    if (kMode == kWgrad) {
        const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kT;
        for (int e = blockIdx.z; e < a.experts; e += gridDim.z) {
            const int64_t r0 = row_begin(a, e), r1 = row_begin(a, e + 1);
            float acc[4][4] = {};
            tile_product([&](int i, int64_t r) { return i0 + i < a.n ? __bfloat162float(a.rows_a[(r0 + r) * a.lda + i0 + i]) : 0.f; },
                         [&](int j, int64_t r) { return col0 + j < a.k ? __bfloat162float(a.b[(r0 + r) * a.ldb + col0 + j]) : 0.f; },
                         r1 > r0 ? r1 - r0 : 0, acc);
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int64_t n = i0 + ty * 4 + i, k = col0 + tx * 4 + j;
                    if (n < a.n && k < a.k) put(a, e * a.stride_o + n * a.ldo + k, acc[i][j]);
                }
        }
        return;
    }
    // row tiles of every expert in turn; e == -1 / experts: the rows of none
    int64_t t = 0;
    for (int e = -1; e <= a.experts; ++e) {
        const int64_t r0 = e < 0 ? 0 : row_begin(a, e);
        const int64_t r1 = e == a.experts ? a.rows : row_begin(a, e + 1);
        for (int64_t i0 = r0; i0 < r1; i0 += kT, ++t) {
            if (t % gridDim.y != blockIdx.y) continue;
            float acc[4][4] = {};
            const int64_t depth = e < 0 || e == a.experts ? 0 : kMode == kFwd ? a.k : a.n;
            const bf16* w = a.b + e * a.stride_b;
            tile_product([&](int i, int64_t k) { return i0 + i < r1 ? __bfloat162float(a.rows_a[(i0 + i) * a.lda + k]) : 0.f; },
                         [&](int j, int64_t k) {
                             if (col0 + j >= cols) return 0.f;
                             return __bfloat162float(kMode == kFwd ? w[(col0 + j) * a.ldb + k] : w[k * a.ldb + col0 + j]);
                         },
                         depth, acc);
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int64_t r = i0 + ty * 4 + i, c = col0 + tx * 4 + j;
                    if (r < r1 && c < cols) put(a, r * a.ldo + c, acc[i][j]);
                }
        }
    }
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxSide = int64_t(1) << 20;
constexpr int kMaxExperts = 1024;
constexpr size_t kExpertHeader = 256;      // the error word that mo_check_device_status reads

size_t expert_ws_bytes() { return kExpertHeader; }

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

int run_expert(int mode, const ExpertArgs& a, void* ws, size_t ws_bytes, mo_stream_t stream) {
    if (a.offsets == nullptr) return MO_ERR_INVALID_ARG;
    if (!op_aligned(a.offsets, 4)) return MO_ERR_ALIGNMENT;
    const int st = op_check_ws(ws, ws_bytes, expert_ws_bytes());
    if (st != MO_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return op_status(op_traced(MO_K_EXPERT + mode, s, [&] {
        const unsigned gx = static_cast<unsigned>(op_ceil_div(mode == kFwd ? a.n : a.k, kT));
        if (mode == kWgrad) {
            const dim3 grid(gx, static_cast<unsigned>(op_ceil_div(a.n, kT)), static_cast<unsigned>(a.experts));
            expert_kernel<kWgrad><<<grid, 256, 0, s>>>(a);
        } else {
            const int64_t tiles = op_ceil_div(a.rows, kT) + a.experts + 2;
            const dim3 grid(gx, static_cast<unsigned>(std::min<int64_t>(tiles, 4096)));
            if (mode == kFwd)
                expert_kernel<kFwd><<<grid, 256, 0, s>>>(a);
            else
                expert_kernel<kDgrad><<<grid, 256, 0, s>>>(a);
        }
        return cudaGetLastError();
    }));
}

}  // namespace
}  // namespace mo

using namespace mo;

extern "C" {

int expert_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k, int experts, size_t* bytes_out) {
    if (bytes_out == nullptr) return MO_ERR_INVALID_ARG;
    const int st = check_sizes(rows, n, k, experts);
    if (st == MO_OK) *bytes_out = expert_ws_bytes();
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
    const ExpertArgs a = {static_cast<const bf16*>(X), ldx, static_cast<const bf16*>(W), ldw, stride_w, Y, ldy, 0,
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
    const ExpertArgs a = {static_cast<const bf16*>(dY), ldy, static_cast<const bf16*>(W), ldw, stride_w, dX, ldx, 0,
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
    const ExpertArgs a = {static_cast<const bf16*>(dY), ldy, static_cast<const bf16*>(X), ldx, 0, dW, lddw, stride_dw,
                          offsets, rows, n, k, experts, dw_dtype, accumulate};
    return run_expert(kWgrad, a, ws, ws_bytes, stream);
}

}  // extern "C"
