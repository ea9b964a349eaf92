// Rows in 8 bits: q_rc is the whole number nearest to 127 x_rc / a_r (ties to
// even) with a_r = max_c |x_rc|, and scale_r = a_r / 127, so x ~ q scale with
// an error of at most half a step a_r / 254. A row whose a_r is below 2^-100
// (where 127 / a could overflow) is a row of zeros with scale 0.
//
// The product x (127 / a) in fp32 is off by at most 127 (2^-24 + 2^-24) =
// 1.6e-5, so only values whose distance to the nearest border m + 1/2 is
// below 1e-4 can round the wrong way; those are decided exactly: the sign of
// 254 x - (2 m + 1) a in fp64, where both products are exact. q is therefore
// a function of x alone, whatever the arithmetic.
#include "ops.cuh"

namespace moe {

namespace {

constexpr float kTinyRow = 7.888609052210118e-31f;   // 2^-100

// 16 consecutive elements of a row
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    uint4 u[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        u[0] = __ldg(reinterpret_cast<const uint4*>(p));
        u[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = reinterpret_cast<const uint32_t*>(u)[i >> 1];
        return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
};
template <> struct Vec16<float> {
    float4 f[4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
    }
    __device__ __forceinline__ float get(int i) const { return reinterpret_cast<const float*>(f)[i]; }
};

template <typename V>
__device__ __forceinline__ float amax16(const V& v, float a) {
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v.get(i)));
    return a;
}

__device__ __noinline__ float border(float x, float a, float v) {
    const float m = floorf(v);
    const double c = 254.0 * static_cast<double>(x) - (2.0 * static_cast<double>(m) + 1.0) * static_cast<double>(a);
    if (c > 0.0) return m + 1.f;
    if (c < 0.0) return m;
    return (static_cast<int>(m) & 1) ? m + 1.f : m;
}

template <typename V>
__device__ __forceinline__ uint4 quant16(const V& x, float a, float inv) {
    constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    float r[16];
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float v = x.get(i) * inv;
        r[i] = (v + kMagic) - kMagic;
        worst = fmaxf(worst, fabsf(v - r[i]));
    }
    if (worst > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = x.get(i) * inv;
            if (fabsf(v - r[i]) > 0.4999f) r[i] = border(x.get(i), a, v);
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = __float_as_uint(r[4 * i + c] + kMagic);   // low byte: the whole number
        w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// TPR threads take a row: up to HOLD 16-element vectors each stay in
// registers between the maximum and the rounding (one read of the row);
// longer rows read the rest twice. SCATTER: the row goes to the k
// destinations pos[row, :] instead of its own place.
constexpr int kHold = 4;
template <typename T, int TPR, bool SCATTER>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
quantize_kernel(const T* __restrict__ x, int rows, int cols, const int32_t* __restrict__ used,
                const int32_t* __restrict__ pos, int k, int out_rows, int8_t* __restrict__ q,
                float* __restrict__ scale) {
    constexpr int BLOCK = TPR < 128 ? 128 : TPR;
    constexpr int RPB = BLOCK / TPR;   // rows a block
    __shared__ float red[BLOCK / 32];
    pdl_wait();
    pdl_launch();
    const int tid = threadIdx.x % TPR;
    const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
    const int n = used != nullptr ? min(rows, *used) : rows;
    if (row >= n) return;   // whole warps (TPR = 32) or the whole block
    const int nv = cols / 16;
    const T* xr = x + static_cast<size_t>(row) * cols;
    Vec16<T> held[kHold];
    float a = 0.f;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int v = tid + h * TPR;
        if (v < nv) held[h].load(xr + static_cast<size_t>(v) * 16);
    }
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if (tid + h * TPR < nv) a = amax16(held[h], a);
    for (int v = tid + kHold * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        a = amax16(w, a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) a = fmaxf(a, red[w]);
    }
    const bool live = a >= kTinyRow;
    const float inv = live ? __fdiv_rn(127.f, a) : 0.f;
    const float sc = live ? __fdiv_rn(a, 127.f) : 0.f;
    auto put = [&](int v, const uint4& w) {
        if constexpr (SCATTER) {
            for (int j = 0; j < k; ++j) {
                const int p = pos[static_cast<size_t>(row) * k + j];
                if (p >= 0 && p < out_rows)
                    *reinterpret_cast<uint4*>(q + static_cast<size_t>(p) * cols + static_cast<size_t>(v) * 16) = w;
            }
        } else {
            *reinterpret_cast<uint4*>(q + static_cast<size_t>(row) * cols + static_cast<size_t>(v) * 16) = w;
        }
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if (tid + h * TPR < nv) put(tid + h * TPR, quant16(held[h], a, inv));
    for (int v = tid + kHold * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        put(v, quant16(w, a, inv));
    }
    if constexpr (SCATTER) {
        if (tid < k) {
            const int p = pos[static_cast<size_t>(row) * k + tid];
            if (p >= 0 && p < out_rows) scale[p] = sc;
        }
    } else if (tid == 0) {
        scale[row] = sc;
    }
}

template <typename T, bool SCATTER>
cudaError_t launch_quant(const T* x, int rows, int cols, const int32_t* used, const int32_t* pos, int k, int out_rows,
                         int8_t* q, float* scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    if (cols <= 32 * 16 * kHold)
        return launch_k(quantize_kernel<T, 32, SCATTER>, dim3(ceil_div(rows, 4)), dim3(128), 0, st, x, rows, cols, used,
                        pos, k, out_rows, q, scale);
    if (cols <= 128 * 16 * kHold)
        return launch_k(quantize_kernel<T, 128, SCATTER>, dim3(rows), dim3(128), 0, st, x, rows, cols, used, pos, k,
                        out_rows, q, scale);
    return launch_k(quantize_kernel<T, 256, SCATTER>, dim3(rows), dim3(256), 0, st, x, rows, cols, used, pos, k,
                    out_rows, q, scale);
}

// Padding rows of the padded layout: zeros, scale 0, no token.
__global__ void __launch_bounds__(256)
pad_rows_i8_kernel(const int32_t* __restrict__ indptr, const void* __restrict__ stats, int E, int nvec,
                   uint4* __restrict__ xq, float* __restrict__ xs, int32_t* __restrict__ row_token) {
    pdl_wait();
    pdl_launch();
    const int e = blockIdx.x;
    const int r0 = indptr[e] + MOE_STATS_KEPT(stats, E)[e], r1 = indptr[e + 1];
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < (r1 - r0) * nvec; i += gridDim.y * blockDim.x)
        xq[static_cast<size_t>(r0 + i / nvec) * nvec + i % nvec] = make_uint4(0u, 0u, 0u, 0u);
    if (blockIdx.y == 0)
        for (int r = r0 + static_cast<int>(threadIdx.x); r < r1; r += blockDim.x) {
            row_token[r] = -1;
            xs[r] = 0.f;
        }
}

}  // namespace

cudaError_t launch_quantize_rows(int dtype, const void* x, int rows, int cols, const int32_t* used, int8_t* q,
                                 float* scale, cudaStream_t st) {
    if (dtype == MOE_DTYPE_BF16)
        return launch_quant<__nv_bfloat16, false>(static_cast<const __nv_bfloat16*>(x), rows, cols, used, nullptr, 0, 0,
                                                  q, scale, st);
    return launch_quant<float, false>(static_cast<const float*>(x), rows, cols, used, nullptr, 0, 0, q, scale, st);
}

cudaError_t launch_quantize_scatter(int dtype, const void* x, const int32_t* pos, int T, int d, int k, int rows,
                                    int8_t* xq, float* xs, cudaStream_t st) {
    if (dtype == MOE_DTYPE_BF16)
        return launch_quant<__nv_bfloat16, true>(static_cast<const __nv_bfloat16*>(x), T, d, nullptr, pos, k, rows, xq,
                                                 xs, st);
    return launch_quant<float, true>(static_cast<const float*>(x), T, d, nullptr, pos, k, rows, xq, xs, st);
}

cudaError_t launch_pad_rows_i8(const int32_t* indptr, const void* stats, int E, int d, int8_t* xq, float* xs,
                               int32_t* row_token, int pad, cudaStream_t st) {
    const int nvec = d / 16;
    const int gy = ceil_div((pad - 1) * nvec, 256 * 4);
    return launch_k(pad_rows_i8_kernel, dim3(E, gy < 1 ? 1 : gy), dim3(256), 0, st, indptr, stats, E, nvec,
                    reinterpret_cast<uint4*>(xq), xs, row_token);
}

}  // namespace moe
