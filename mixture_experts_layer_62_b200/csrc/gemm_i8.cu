// Products of the experts in 8-bit integers: for every group e and row r of
// it, with a scale for each token (row) and channel (weight row),
//   PLAIN   out[r][n] = sa_r sb_{e,n} sum_c A[r][c] B_e[n][c]
//   SWIGLU  a, b as PLAIN with B0 and B1; out[r][n] = SiLU(a) b
// The sums are 32-bit integers: at most K 128^2 <= 2^31 - 1 in magnitude for
// K <= 131071, so they are exact and do not depend on the order or on the
// kernel that forms them. The float factors are applied as
// (float(sum) * sa) * sb, every form the same, and the result is rounded once.
//
// This form: 64 x 64 output tiles on CUDA cores (four products an
// instruction), operands staged in shared memory, one block per (column
// tile, group).
#include "ops.cuh"

namespace moe {

namespace {

constexpr int kBT = 64;   // rows and columns of a tile
constexpr int kBK = 64;   // bytes of K a step

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename OutT, bool SWIGLU>
__global__ void __launch_bounds__(256)
i8_simt_kernel(const __grid_constant__ I8Gemm g) {
    __shared__ int32_t sA[kBT][kBK / 4 + 1], sB[SWIGLU ? 2 : 1][kBT][kBK / 4 + 1];
    const int e = blockIdx.y, n0 = blockIdx.x * kBT;
    const int r_lo = g.indptr[e], r_hi = min(g.indptr[e + 1], g.rows);
    if (r_lo < 0) return;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int KW = g.K / 4;   // K % 16 == 0
    const int32_t* A = reinterpret_cast<const int32_t*>(g.A);
    const int32_t* B0 = reinterpret_cast<const int32_t*>(g.B0) + static_cast<size_t>(e) * g.N * KW;
    const int32_t* B1 = SWIGLU ? reinterpret_cast<const int32_t*>(g.B1) + static_cast<size_t>(e) * g.N * KW : nullptr;
    for (int r0 = r_lo; r0 < r_hi; r0 += kBT) {
        int acc[SWIGLU ? 2 : 1][4][4] = {};
        for (int k0 = 0; k0 < KW; k0 += kBK / 4) {
            for (int i = threadIdx.x; i < kBT * (kBK / 4); i += 256) {
                const int r = i / (kBK / 4), c = i % (kBK / 4), kc = k0 + c;
                sA[r][c] = (r0 + r < r_hi && kc < KW) ? A[static_cast<size_t>(r0 + r) * KW + kc] : 0;
                const bool in = n0 + r < g.N && kc < KW;
                sB[0][r][c] = in ? B0[static_cast<size_t>(n0 + r) * KW + kc] : 0;
                if (SWIGLU) sB[SWIGLU ? 1 : 0][r][c] = in ? B1[static_cast<size_t>(n0 + r) * KW + kc] : 0;
            }
            __syncthreads();
#pragma unroll 4
            for (int c = 0; c < kBK / 4; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int w = 0; w < (SWIGLU ? 2 : 1); ++w)
                            acc[w][i][j] = __dp4a(sA[ty * 4 + i][c], sB[w][tx + 16 * j][c], acc[w][i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + ty * 4 + i, n = n0 + tx + 16 * j;
                if (r >= r_hi || n >= g.N) continue;
                const float sa = g.sa[r];
                float v = static_cast<float>(acc[0][i][j]) * sa * g.sb0[static_cast<size_t>(e) * g.N + n];
                if (SWIGLU) {
                    const float b = static_cast<float>(acc[SWIGLU ? 1 : 0][i][j]) * sa * g.sb1[static_cast<size_t>(e) * g.N + n];
                    v = v / (1.f + expf(-v)) * b;
                }
                put(static_cast<OutT*>(g.out) + static_cast<size_t>(r) * g.N + n, v);
            }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *g.status = MOE_OK;
}

template <typename OutT>
cudaError_t launch_t(const I8Gemm& g, cudaStream_t st) {
    const dim3 grid(ceil_div(g.N, kBT), g.E);
    if (g.B1 != nullptr) return launch_k(i8_simt_kernel<OutT, true>, grid, dim3(256), 0, st, g);
    return launch_k(i8_simt_kernel<OutT, false>, grid, dim3(256), 0, st, g);
}

}  // namespace

cudaError_t launch_i8_gemm(const I8Gemm& g, cudaStream_t st) {
    return g.out_dtype == MOE_DTYPE_BF16 ? launch_t<__nv_bfloat16>(g, st) : launch_t<float>(g, st);
}

}  // namespace moe
