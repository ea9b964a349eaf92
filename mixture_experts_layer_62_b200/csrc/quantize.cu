// Rows in 8 bits: q_rc is the whole number nearest to 127 x_rc / a_r (ties to
// even) with a_r = max_c |x_rc|, and scale_r = a_r / 127, so x ~ q scale with
// an error of at most half a step a_r / 254. A row whose a_r is below 2^-100
// (where 127 / a could overflow) is a row of zeros with scale 0.
//
// x inv with inv = 127 / a rounded once is off by at most 127 2^-24 = 7.6e-6,
// and the fused multiply-add that rounds it to a whole number adds nothing to
// that, so only values whose distance to the nearest border m + 1/2 is below
// 1e-4 can go the wrong way; those are decided exactly, by the sign of
// 254 x - (2 m + 1) a in fp64, where both products are exact. q is therefore
// a function of x alone, whatever the arithmetic.
//
// Both users are bound by memory only if the arithmetic stays short: at 6.5
// TB/s an SM takes 9 bf16 elements a clock and has 128 lanes for them. The
// maximum is taken two elements an instruction on the packed bf16 words, and
// rounding, remainder and border test run as two-element fp32 instructions
// (f32x2), about 5 instructions an element in all.
#include "ops.cuh"

namespace moe {

namespace {

constexpr float kTinyRow = 7.888609052210118e-31f;   // 2^-100
constexpr float kMagic = 12582912.f;                 // 1.5 2^23: adding it rounds to a whole number, ties to even

// ---- two-element fp32 arithmetic ----------------------------------------------
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 16 consecutive elements of a row
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ float lo(int i) const { return __uint_as_float(w[i] << 16); }
    __device__ __forceinline__ float hi(int i) const { return __uint_as_float(w[i] & 0xFFFF0000u); }
    __device__ __forceinline__ float amax(float a) const {
        __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
        for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
        const float2 f = __bfloat1622float2(m);
        return fmaxf(a, fmaxf(f.x, f.y));
    }
};
template <> struct Vec16<float> {
    float f[16];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = a.z; f[4 * i + 3] = a.w;
        }
    }
    __device__ __forceinline__ float lo(int i) const { return f[2 * i]; }
    __device__ __forceinline__ float hi(int i) const { return f[2 * i + 1]; }
    __device__ __forceinline__ float amax(float a) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(f[i]));
        return a;
    }
};

// The whole number for a value near a border: r is the fp32 choice, rem the remainder
__device__ __noinline__ float border(float x, float a, float r, float rem) {
    const float m = rem > 0.f ? r : r - 1.f;   // the border is m + 1/2
    const double c = 254.0 * static_cast<double>(x) - (2.0 * static_cast<double>(m) + 1.0) * static_cast<double>(a);
    if (c > 0.0) return m + 1.f;
    if (c < 0.0) return m;
    return (static_cast<int>(m) & 1) ? m + 1.f : m;
}

template <typename V>
__device__ __forceinline__ uint4 quant16(const V& x, float a, float inv) {
    const uint64_t inv2 = pair2(inv, inv), magic2 = pair2(kMagic, kMagic), minus2 = pair2(-kMagic, -kMagic);
    float t[16];   // the low byte of t's bits is the whole number
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t xx = pair2(x.lo(i), x.hi(i));
        const uint64_t tt = fma2(xx, inv2, magic2);
        const uint64_t rem = fma2(xx, inv2, add2(tt, minus2) ^ 0x8000000080000000ull);   // x inv - whole
        float r0, r1;
        split2(rem, r0, r1);
        worst = fmaxf(worst, fmaxf(fabsf(r0), fabsf(r1)));
        split2(tt, t[2 * i], t[2 * i + 1]);
    }
    if (worst > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = i & 1 ? x.hi(i / 2) : x.lo(i / 2), r = t[i] - kMagic, rem = fmaf(v, inv, -r);
            if (fabsf(rem) > 0.4999f) t[i] = border(v, a, r, rem) + kMagic;
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                           __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040), 0x5410);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A row by TPR threads (tid of them): up to kHold 16-element vectors a
// thread stay in registers between the maximum and the rounding, one read of
// the row; a longer row is read twice past that. red: TPR / 32 floats of
// shared memory when TPR > 32, and then all of the block's threads call with
// the same control flow. Returns scale_r; put(v, w) stores vector v.
// hold_row starts the reads (nv = 0: none), quantize_row finishes.
constexpr int kHold = 4;
template <typename T, int TPR>
__device__ __forceinline__ void hold_row(Vec16<T> (&held)[kHold], const T* __restrict__ xr, int nv, int tid) {
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if (tid + h * TPR < nv) held[h].load(xr + static_cast<size_t>(tid + h * TPR) * 16);
}
template <typename T, int TPR, typename Put>
__device__ __forceinline__ float quantize_row(const Vec16<T> (&held)[kHold], const T* __restrict__ xr, int nv, int tid,
                                              float* red, Put put) {
    float a = 0.f;
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if (tid + h * TPR < nv) a = held[h].amax(a);
    for (int v = tid + kHold * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        a = w.amax(a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if constexpr (TPR > 32) {
        if ((tid & 31) == 0) red[tid >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) a = fmaxf(a, red[w]);
    }
    const bool live = a >= kTinyRow;
    const float inv = live ? __fdiv_rn(127.f, a) : 0.f;
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if (tid + h * TPR < nv) put(tid + h * TPR, quant16(held[h], a, inv));
    for (int v = tid + kHold * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        put(v, quant16(w, a, inv));
    }
    return live ? __fdiv_rn(a, 127.f) : 0.f;
}

template <typename T, int TPR>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
quantize_kernel(const T* __restrict__ x, int rows, int cols, const int32_t* __restrict__ used, int8_t* __restrict__ q,
                float* __restrict__ scale) {
    constexpr int RPB = TPR < 128 ? 128 / TPR : 1;   // rows a block
    __shared__ float red[TPR / 32];
    const int tid = threadIdx.x % TPR;
    const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / TPR;
    const int n = used != nullptr ? min(rows, *used) : rows;
    if (row >= n) return;   // whole warps (TPR = 32) or the whole block
    uint4* qr = reinterpret_cast<uint4*>(q + static_cast<size_t>(row) * cols);
    const T* xr = x + static_cast<size_t>(row) * cols;
    Vec16<T> held[kHold];
    hold_row<T, TPR>(held, xr, cols / 16, tid);
    const float sc = quantize_row<T, TPR>(held, xr, cols / 16, tid, red, [&](int v, const uint4& w) { qr[v] = w; });
    if (tid == 0) scale[row] = sc;
}

template <typename T>
cudaError_t quantize_t(const T* x, int rows, int cols, const int32_t* used, int8_t* q, float* scale, cudaStream_t st) {
    if (cols <= 32 * 16 * kHold)
        return launch_k(quantize_kernel<T, 32>, dim3(ceil_div(rows, 4)), dim3(128), 0, st, x, rows, cols, used, q, scale);
    if (cols <= 128 * 16 * kHold)
        return launch_k(quantize_kernel<T, 128>, dim3(rows), dim3(128), 0, st, x, rows, cols, used, q, scale);
    return launch_k(quantize_kernel<T, 256>, dim3(rows), dim3(256), 0, st, x, rows, cols, used, q, scale);
}

// ---- permutation with the rows in 8 bits ------------------------------------------
// TPR threads take a token (a block of 128 four of them, or one): they start
// reading its row, find the destinations of its pairs, write pos and
// row_token, and quantise the row once into all of its destinations. Padding
// rows of the padded layout are shared out over the blocks by expert.
//  FEW (at most kFewPairs pairs): one launch does it all. Every block counts
//  all pairs and scans the experts by itself; a pair's rank is the number of
//  pairs of its expert before it in the drop order. Block 0 writes indptr
//  and the statistics.
//  Otherwise hist_kernel and scan_kernel (permute.cu) have left the chunk
//  bases, indptr and the statistics; a block's tokens lie in one chunk.
struct PermuteArgs {
    const void* x;
    const int32_t* idx;
    const int32_t* blockoff;   // !FEW: [E][kk][NB]
    int32_t* indptr;           // FEW: written here
    void* stats;
    int32_t *pos, *row_token;
    int8_t* xq;
    float* xs;
    int T, d, E, k, kk, capacity, pad, rows, NB;
};
constexpr int kFewPairs = 2048;

template <typename T, int TPR, bool FEW>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
permute_i8_kernel(const __grid_constant__ PermuteArgs a) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR, kTokens = kThreads / TPR;
    __shared__ int s_idx[FEW ? kFewPairs : kChunk * MOE_MAX_K];
    __shared__ int s_cnt[FEW ? MOE_MAX_E : 1], s_ptr[FEW ? MOE_MAX_E + 1 : 1];
    __shared__ int s_pos[kTokens * MOE_MAX_K];
    __shared__ float red[TPR / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int t0 = blockIdx.x * kTokens, nt = min(kTokens, a.T - t0);
    const T* xr = static_cast<const T*>(a.x) + static_cast<size_t>(t0 + sub) * a.d;
    Vec16<T> held[kHold];
    hold_row<T, TPR>(held, xr, sub < nt ? a.d / 16 : 0, tid);
    // the pairs staged: all of them, or the chunk's
    const int c0 = FEW ? 0 : t0 / kChunk * kChunk;
    const int np = (FEW ? a.T : min(kChunk, a.T - c0)) * a.k;
    for (int i = threadIdx.x; i < np; i += kThreads) s_idx[i] = a.idx[static_cast<size_t>(c0) * a.k + i];
    if constexpr (FEW) {
        for (int e = threadIdx.x; e < a.E; e += kThreads) s_cnt[e] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < np; i += kThreads) {
            const int e = s_idx[i];
            if (e >= 0 && e < a.E) atomicAdd(&s_cnt[e], 1);
        }
        __syncthreads();
        if (warp == 0) {
            int base = 0, kept_all = 0, most = 0, all = 0;
            int32_t* counts = MOE_STATS_COUNTS(a.stats, a.E);
            int32_t* keeps = MOE_STATS_KEPT(a.stats, a.E);
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                const int e = e0 + lane;
                const int c = e < a.E ? s_cnt[e] : 0;
                const int kp = a.capacity < 0 ? c : min(c, a.capacity);
                const int held = a.pad > 0 ? (kp + a.pad - 1) / a.pad * a.pad : kp;
                int incl = held;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += u;
                }
                if (e < a.E) {
                    s_ptr[e] = base + incl - held;
                    if (blockIdx.x == 0) {
                        a.indptr[e] = base + incl - held;
                        counts[e] = c;
                        keeps[e] = kp;
                    }
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
                kept_all += kp;
                all += c;
                most = max(most, c);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                kept_all += __shfl_xor_sync(0xffffffffu, kept_all, o);
                all += __shfl_xor_sync(0xffffffffu, all, o);
                most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            if (lane == 0) {
                s_ptr[a.E] = base;
                if (blockIdx.x == 0) {
                    a.indptr[a.E] = base;
                    moe_stats* st = static_cast<moe_stats*>(a.stats);
                    st->status = MOE_OK;
                    st->capacity = a.capacity;
                    st->rows = kept_all;
                    st->dropped = all - kept_all;
                    st->max_count = most;
                    const float mean = static_cast<float>(a.T) * static_cast<float>(a.k) / static_cast<float>(a.E);
                    st->max_over_mean = static_cast<float>(most) / mean;
                    st->reserved[0] = st->reserved[1] = 0;
                }
            }
        }
    } else {
        pdl_wait();   // the chunk bases and indptr come from the scan
    }
    __syncthreads();
    // ranks: a warp a pair, its lanes over the pairs that can stand before it
    const int chunk = c0 / kChunk;
    for (int i = warp; i < nt * a.k; i += kThreads / 32) {
        const int p = (t0 - c0) * a.k + i, j = p % a.k, e = s_idx[p];
        int at = -1;
        if (e >= 0 && e < a.E) {
            int before = 0;
            if (a.kk > 1) {   // slot order: earlier slots first (in the base already when !FEW)
                for (int v = lane; v < np; v += 32) {
                    const int jj = v % a.k;
                    before += s_idx[v] == e && ((FEW && jj < j) || (jj == j && v < p));
                }
            } else {
                for (int v = lane; v < p; v += 32) before += s_idx[v] == e;
            }
            before = __reduce_add_sync(0xffffffffu, before);
            if (!FEW) before += a.blockoff[(static_cast<size_t>(e) * a.kk + (a.kk > 1 ? j : 0)) * a.NB + chunk];
            if (a.capacity < 0 || before < a.capacity) at = (FEW ? s_ptr[e] : a.indptr[e]) + before;
        }
        if (lane == 0) {
            s_pos[i] = at;
            a.pos[static_cast<size_t>(t0) * a.k + i] = at;
            if (at >= 0) a.row_token[at] = t0 + i / a.k;
        }
    }
    if (a.pad > 0) {
        const int nv = a.d / 16;
        for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
            int r0, r1;
            if constexpr (FEW) {
                const int c = s_cnt[e];
                r0 = s_ptr[e] + (a.capacity < 0 ? c : min(c, a.capacity));
                r1 = s_ptr[e + 1];
            } else {
                r0 = a.indptr[e] + MOE_STATS_KEPT(a.stats, a.E)[e];
                r1 = a.indptr[e + 1];
            }
            for (int i = threadIdx.x; i < (r1 - r0) * nv; i += kThreads)
                reinterpret_cast<uint4*>(a.xq + static_cast<size_t>(r0) * a.d)[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int r = r0 + static_cast<int>(threadIdx.x); r < r1; r += kThreads) {
                a.row_token[r] = -1;
                a.xs[r] = 0.f;
            }
        }
    }
    __syncthreads();
    if (sub >= nt) return;   // whole warps: blocks of more than one token have TPR = 32
    int nd = 0;
    for (int j = 0; j < a.k; ++j) nd += s_pos[sub * a.k + j] >= 0;
    if (nd == 0) return;     // the same for all threads of the token
    const float sc = quantize_row<T, TPR>(held, xr, a.d / 16, tid, red, [&](int v, const uint4& w) {
        for (int j = 0; j < a.k; ++j) {
            const int at = s_pos[sub * a.k + j];
            if (at >= 0) reinterpret_cast<uint4*>(a.xq + static_cast<size_t>(at) * a.d)[v] = w;
        }
    });
    if (tid < a.k && s_pos[sub * a.k + tid] >= 0) a.xs[s_pos[sub * a.k + tid]] = sc;
}

template <typename T, bool FEW>
cudaError_t permute_t(const PermuteArgs& a, cudaStream_t st) {
    if (a.d <= 32 * 16 * kHold)
        return launch_k(permute_i8_kernel<T, 32, FEW>, dim3(ceil_div(a.T, 4)), dim3(128), 0, st, a);
    if (a.d <= 128 * 16 * kHold) return launch_k(permute_i8_kernel<T, 128, FEW>, dim3(a.T), dim3(128), 0, st, a);
    return launch_k(permute_i8_kernel<T, 256, FEW>, dim3(a.T), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_quantize_rows(int dtype, const void* x, int rows, int cols, const int32_t* used, int8_t* q,
                                 float* scale, cudaStream_t st) {
    if (dtype == MOE_DTYPE_BF16) return quantize_t(static_cast<const __nv_bfloat16*>(x), rows, cols, used, q, scale, st);
    return quantize_t(static_cast<const float*>(x), rows, cols, used, q, scale, st);
}

cudaError_t launch_permute_i8(const PermuteI8& p, cudaStream_t st) {
    PermuteArgs a = {};
    a.x = p.x; a.idx = p.idx; a.blockoff = p.blockoff; a.indptr = p.indptr; a.stats = p.stats; a.pos = p.pos;
    a.row_token = p.row_token; a.xq = p.xq; a.xs = p.xs;
    a.T = p.T; a.d = p.d; a.E = p.E; a.k = p.k; a.kk = p.kk; a.capacity = p.capacity; a.pad = p.pad; a.rows = p.rows;
    a.NB = ceil_div(p.T, kChunk);
    const bool few = static_cast<long long>(p.T) * p.k <= kFewPairs;
    if (few) return p.dtype == MOE_DTYPE_BF16 ? permute_t<__nv_bfloat16, true>(a, st) : permute_t<float, true>(a, st);
    cudaError_t e = launch_hist(p.idx, p.T, p.k, p.kk, p.E, p.blockcnt, st);
    if (e != cudaSuccess) return e;
    struct Dependent {   // each later launch starts beside the one before and waits for it
        Dependent() { g_pdl = true; }
        ~Dependent() { g_pdl = false; }
    } dependent;
    ScanArgs sa = {};
    sa.T = p.T; sa.k = p.k; sa.E = p.E; sa.capacity = p.capacity; sa.kk = p.kk;
    sa.blockcnt = p.blockcnt; sa.blockoff = p.blockoff;
    sa.indptr = p.indptr; sa.stats = p.stats;
    sa.pad = p.pad;
    e = launch_scan(sa, st);
    if (e != cudaSuccess) return e;
    return p.dtype == MOE_DTYPE_BF16 ? permute_t<__nv_bfloat16, false>(a, st) : permute_t<float, false>(a, st);
}

}  // namespace moe
