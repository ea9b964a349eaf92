// The way back from the experts with everything that ends the layer in a
// transformer block, and its gradients ("Lecture 21 · LLM: Mixture-of-
// Experts" §3.2 step 4; the residual sum of §2.2):
//   m_t = sum_j g_{t,j} o[pos_{t,j}] (+ s_t),   y_t = residual_t + D(m_t)
//   u = D(dy):  dO[pos_{t,j}] = g_{t,j} u_t,  dgate_{t,j} = <u_t, o[pos_{t,j}]>,  ds = u
// and, with gates 1 and nothing else, the gradient of the permutation
// dx_t = sum_j dXp[pos_{t,j}].
//
// D is dropout whose mask is computed where it is needed and never stored:
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011) at the counter (i / 8, offset) with the seed as key
// gives eight 16-bit numbers, one for each of the elements 8 (i / 8) + 0..7;
// an element stays when its number is at least thr = 65536 p and is then
// scaled by 65536 / (65536 - thr), the exact inverse of the kept share.
// Sixteen bits an element make one generator call serve one 16-byte vector
// of bf16; a dropped element is a selected 0, never a product with 0.
//
// Sums are fp32 in slot order, each result is rounded once, nothing is
// atomic: repeated calls give identical bits.
#include <algorithm>

#include "ops.cuh"

namespace moe {

namespace {

template <typename T> struct Vec8;   // eight consecutive elements
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&v)[8]) {
        uint4 u;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = u;
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ static void store(float* p, const float (&v)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// The eight 16-bit numbers of block b, two to a word (element 2 i in the low half of word i).
__device__ __forceinline__ void philox(unsigned long long seed, unsigned long long offset, unsigned long long b,
                                       uint32_t (&x)[4]) {
    x[0] = static_cast<uint32_t>(b);
    x[1] = static_cast<uint32_t>(b >> 32);
    x[2] = static_cast<uint32_t>(offset);
    x[3] = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long p0 = static_cast<unsigned long long>(x[0]) * 0xD2511F53u;
        const unsigned long long p1 = static_cast<unsigned long long>(x[2]) * 0xCD9E8D57u;
        x[0] = static_cast<uint32_t>(p1 >> 32) ^ x[1] ^ k0;
        x[1] = static_cast<uint32_t>(p1);
        x[2] = static_cast<uint32_t>(p0 >> 32) ^ x[3] ^ k1;
        x[3] = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}
// v -> D(v) for the eight elements of block b
__device__ __forceinline__ void drop8(const Dropout& d, unsigned long long seed, unsigned long long offset,
                                      unsigned long long b, float (&v)[8]) {
    uint32_t x[4];
    philox(seed, offset, b, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = (x[i] & 0xFFFFu) >= d.thr ? v[2 * i] * d.scale : 0.f;
        v[2 * i + 1] = (x[i] >> 16) >= d.thr ? v[2 * i + 1] * d.scale : 0.f;
    }
}

// A block takes a token (or one of a few stretches of its row, for small
// batches): its positions and gates are loaded once, and each thread walks
// vectors of eight columns, the rows of all K slots requested together
// (K: k rounded up to 1, 2, 4, 8 or 16).
constexpr int kMixThreads = 128;
// The threads of a block: a vector of eight columns each, at most kMixThreads. (2876 tokens of d = 152 in fp32, 6 slots,
// both passes: 9.0 us; with 128 threads always 15.3.)
inline unsigned mix_threads(int d) { return static_cast<unsigned>(d >= 8 * kMixThreads ? kMixThreads : (d / 8 + 31) / 32 * 32); }
template <typename T, bool GATED, bool DROP, int K>
__global__ void __launch_bounds__(kMixThreads)
mix_kernel(const __grid_constant__ MixArgs a, int slices) {
    pdl_wait();
    pdl_launch();
    const size_t t = blockIdx.x / slices;
    const int sl = static_cast<int>(blockIdx.x - t * slices), nvec = a.d / 8;
    const int v_lo = static_cast<int>(static_cast<long long>(nvec) * sl / slices);
    const int v_hi = static_cast<int>(static_cast<long long>(nvec) * (sl + 1) / slices);
    int p[K];
    float g[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        p[j] = j < a.k ? a.pos[t * a.k + j] : -1;
        g[j] = GATED && j < a.k ? a.gate[t * a.k + j] : 1.f;
        if (p[j] >= a.rows) p[j] = -1;   // not a row of o: the slot is skipped
    }
    unsigned long long seed = 0, offset = 0;
    if (DROP) {
        seed = a.drop.rng[0];
        offset = a.drop.rng[1];
    }
    const T* o = static_cast<const T*>(a.o);
    for (int v = v_lo + static_cast<int>(threadIdx.x); v < v_hi; v += static_cast<int>(blockDim.x)) {
        const size_t col = static_cast<size_t>(v) * 8, at = t * a.d + col;
        Vec8<T> raw[K], rv, sv;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (p[j] >= 0) raw[j].load(o + static_cast<size_t>(p[j]) * a.d + col);
        if (a.s != nullptr) sv.load(static_cast<const T*>(a.s) + at);
        if (a.residual != nullptr) rv.load(static_cast<const T*>(a.residual) + at);
        float acc[8], x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (p[j] < 0) continue;
            raw[j].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = GATED ? fmaf(g[j], x[e], acc[e]) : acc[e] + x[e];
        }
        if (a.s != nullptr) {
            sv.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
        if (DROP) drop8(a.drop, seed, offset, static_cast<unsigned long long>(at / 8), acc);
        if (a.residual != nullptr) {
            rv.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
        Vec8<T>::store(static_cast<T*>(a.out) + at, acc);
    }
}

// One block per token: a thread takes every blockDim-th vector of dy, forms
// u = D(dy) once and serves all of the token's slots from it; the slots' dot
// products are summed lane by lane, then over the block in a fixed order.
// With padding, the first blocks (`pads`) fill the padding rows of dO with
// zeros: a warp reads the tokens of kPadRows rows at once and writes the rows
// of none (513 tokens of d = 6208, 52 experts padded to 128 rows, both passes:
// 44 us; 32 rows a warp took 54).
constexpr int kPadRows = 8, kMaxPadBlocks = 4 * 148;
template <typename T, bool DROP, int K, int THREADS>   // THREADS: those of the block, 0: any number up to 512
__global__ void __launch_bounds__(THREADS > 0 ? THREADS : 512)
mix_back_kernel(const __grid_constant__ MixBackArgs a, unsigned pads) {
    __shared__ float part[(THREADS > 0 ? THREADS : 512) / 32][K];
    const int threads = THREADS > 0 ? THREADS : static_cast<int>(blockDim.x);
    pdl_wait();
    pdl_launch();
    const int nvec = a.d / 8;
    T* dO = static_cast<T*>(a.dO);
    if (blockIdx.x < pads) {
        const int used = min(a.indptr[a.E], a.rows), lane = threadIdx.x & 31;
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const long long step = static_cast<long long>(kPadRows) * pads * (threads / 32);
        for (long long r0 = kPadRows * (blockIdx.x + static_cast<long long>(pads) * (threadIdx.x >> 5)); r0 < used; r0 += step) {
            const bool none = lane < kPadRows && r0 + lane < used && a.row_token[r0 + lane] < 0;
            for (unsigned m = __ballot_sync(0xffffffffu, none); m != 0; m &= m - 1)
                for (int v = lane; v < nvec; v += 32)
                    Vec8<T>::store(dO + static_cast<size_t>(r0 + __ffs(m) - 1) * a.d + static_cast<size_t>(v) * 8, z);
        }
        return;
    }
    const size_t t = blockIdx.x - pads;
    int p[K];
    float g[K], acc[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        p[j] = j < a.k ? a.pos[t * a.k + j] : -1;
        g[j] = j < a.k ? a.gate[t * a.k + j] : 0.f;
        if (p[j] >= a.rows) p[j] = -1;
        acc[j] = 0.f;
    }
    unsigned long long seed = 0, offset = 0;
    if (DROP) {
        seed = a.drop.rng[0];
        offset = a.drop.rng[1];
    }
    for (int v = threadIdx.x; v < nvec; v += threads) {
        const size_t at = t * a.d + static_cast<size_t>(v) * 8, col = static_cast<size_t>(v) * 8;
        Vec8<T> dyv, ov[K];
        dyv.load(static_cast<const T*>(a.dy) + at);
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (p[j] >= 0) ov[j].load(static_cast<const T*>(a.o) + static_cast<size_t>(p[j]) * a.d + col);
        float u[8];
        dyv.get(u);
        if (DROP) drop8(a.drop, seed, offset, static_cast<unsigned long long>(at / 8), u);
        if (a.ds != nullptr) Vec8<T>::store(static_cast<T*>(a.ds) + at, u);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (p[j] < 0) continue;
            float x[8], w[8];
            ov[j].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[j] = fmaf(u[e], x[e], acc[j]);
                w[e] = g[j] * u[e];
            }
            Vec8<T>::store(dO + static_cast<size_t>(p[j]) * a.d + col, w);
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
        if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
        float s = 0.f;
        for (int w = 0; w < threads / 32; ++w) s += part[w][threadIdx.x];
        a.dgate[t * a.k + threadIdx.x] = s;
    }
}

template <typename T, bool DROP, int K>
cudaError_t mix_back_k(const MixBackArgs& a, cudaStream_t st) {
    // Less than a block's work for every SM: up to four times the threads to a row (one token of d = 4096, with the
    // forward pass, 3.9 us in place of 4.2; 64 tokens of d = 7168 and 8 slots 7.8 in place of 8.6; from 200 tokens on it
    // loses). Blocks of another size than kMixThreads have a kernel of their own, since room for 512 threads leaves each
    // fewer registers: 8192 tokens of 8 slots take 342 us there and 323 here.
    unsigned threads = mix_threads(a.d);
    while (threads < 512 && a.T * threads < 148 * kMixThreads && 8 * threads < static_cast<unsigned>(a.d)) threads *= 2;
    const unsigned rows = kPadRows * (threads / 32);   // rows of a block's turn
    const unsigned pads = a.row_token != nullptr ? std::min((static_cast<unsigned>(a.rows) + rows - 1) / rows, kMaxPadBlocks + 0u) : 0u;
    const dim3 grid(static_cast<unsigned>(a.T) + pads), block(threads);
    if (threads == kMixThreads) return launch_dep(mix_back_kernel<T, DROP, K, kMixThreads>, grid, block, 0, st, a, pads);
    return launch_dep(mix_back_kernel<T, DROP, K, 0>, grid, block, 0, st, a, pads);
}
template <typename T, bool DROP>
cudaError_t mix_back_t(const MixBackArgs& a, cudaStream_t st) {
    if (a.k <= 1) return mix_back_k<T, DROP, 1>(a, st);
    if (a.k <= 2) return mix_back_k<T, DROP, 2>(a, st);
    if (a.k <= 4) return mix_back_k<T, DROP, 4>(a, st);
    if (a.k <= 8) return mix_back_k<T, DROP, 8>(a, st);
    return mix_back_k<T, DROP, 16>(a, st);
}

template <typename T, bool GATED, bool DROP>
cudaError_t mix_d(const MixArgs& a, cudaStream_t st) {
    // fewer tokens than two blocks an SM: stretches of the rows, a pass of the threads at least
    int slices = 1;
    while (a.T * slices < 2 * 148 && slices * kMixThreads < a.d / 8) slices *= 2;
    const dim3 grid(static_cast<unsigned>(a.T) * slices), block(mix_threads(a.d));
    if (a.k <= 1) return launch_dep(mix_kernel<T, GATED, DROP, 1>, grid, block, 0, st, a, slices);
    if (a.k <= 2) return launch_dep(mix_kernel<T, GATED, DROP, 2>, grid, block, 0, st, a, slices);
    if (a.k <= 4) return launch_dep(mix_kernel<T, GATED, DROP, 4>, grid, block, 0, st, a, slices);
    if (a.k <= 8) return launch_dep(mix_kernel<T, GATED, DROP, 8>, grid, block, 0, st, a, slices);
    return launch_dep(mix_kernel<T, GATED, DROP, 16>, grid, block, 0, st, a, slices);
}
template <typename T>
cudaError_t mix_t(const MixArgs& a, cudaStream_t st) {
    if (a.gate == nullptr) return mix_d<T, false, false>(a, st);
    return a.drop.rng == nullptr ? mix_d<T, true, false>(a, st) : mix_d<T, true, true>(a, st);
}

}  // namespace

cudaError_t launch_mix(const MixArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return a.dtype == MOE_DTYPE_BF16 ? mix_t<__nv_bfloat16>(a, st) : mix_t<float>(a, st);
}

cudaError_t launch_mix_back(const MixBackArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool drop = a.drop.rng != nullptr;
    if (a.dtype == MOE_DTYPE_BF16)
        return drop ? mix_back_t<__nv_bfloat16, true>(a, st) : mix_back_t<__nv_bfloat16, false>(a, st);
    return drop ? mix_back_t<float, true>(a, st) : mix_back_t<float, false>(a, st);
}

}  // namespace moe
