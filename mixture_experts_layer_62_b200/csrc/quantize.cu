// Rows in 8 bits: q_rc is the whole number nearest to 127 x_rc / a_r (ties to
// even) with a_r = max_c |x_rc|, and scale_r = a_r / 127, so x ~ q scale with
// an error of at most half a step a_r / 254. A row whose a_r is below 2^-100
// (where 127 / a could overflow) is a row of zeros with scale 0. A row that
// holds an infinity or a NaN gets the scale NaN, so that all that is computed
// from it is NaN: the maxima pass a NaN on (max.NaN, as fast as max). Its q say
// nothing (clearing them too cost the permutation 0.7 to 1 %).
//
// One fused multiply-add rounds x inv, inv = 127 / a in fp32, to a whole
// number; inv is off by 2^-24 relative, so near a border m + 1/2 the wrong
// side could win.
//  * fp32 rows: values closer than 1e-4 to a border (the error is at most 127
//    2^-24 = 7.6e-6) are decided exactly, by the sign of 254 x - (2 m + 1) a in
//    fp64, where both products are exact.
//  * bf16 rows: with x = X 2^i, a = A 2^j, 128 <= X, A <= 255, the distance of
//    v = 127 x / a from a border is |254 X 2^(i-j) - (2 m + 1) A| / (2 A), and
//    that numerator is a multiple of 2^(i-j): if it is not 0 the distance is
//    at least |v| / (254 X) > 1.5e-5 |v|, far above the error 2^-23 |v|, and
//    the product decides. It is 0 only if 127 divides (2 m + 1) A: for A = 254,
//    where inv is a power of two and the product exact, and for m = 63, that
//    is |x| = a / 2, whose even neighbour is 64: inv is taken at or above 127 /
//    a, which sends that one up. No value needs a second look.
// q is a function of x alone either way, whatever the arithmetic.
//
// The arithmetic has to stay short to leave memory the bound: at 6.5 TB/s an
// SM takes 9 bf16 elements a clock and has 128 lanes for them. The maximum
// is taken two elements an instruction on the packed words, the rounding by
// two-element fp32 instructions (f32x2).
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
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 16 consecutive elements of a row, read past L1: each is read once, and a
// kernel that started beside the one that writes its rows must not ask for
// them as constants (so no __restrict__ on what it reads, either)
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p)), b = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ float lo(int i) const { return __uint_as_float(w[i] << 16); }
    __device__ __forceinline__ float hi(int i) const { return __uint_as_float(w[i] & 0xFFFF0000u); }
    __device__ __forceinline__ float amax(float a) const {
        __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
        for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
        const float2 f = __bfloat1622float2(m);
        return max_nan(a, max_nan(f.x, f.y));
    }
};
template <> struct Vec16<float> {
    float f[16];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = a.z; f[4 * i + 3] = a.w;
        }
    }
    __device__ __forceinline__ float lo(int i) const { return f[2 * i]; }
    __device__ __forceinline__ float hi(int i) const { return f[2 * i + 1]; }
    __device__ __forceinline__ float amax(float a) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) a = max_nan(a, fabsf(f[i]));
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

// 127 / a for quant16: for bf16 rows at or above the quotient
__device__ __forceinline__ float inverse(float a, const Vec16<float>*) { return __fdiv_rn(127.f, a); }
__device__ __forceinline__ float inverse(float a, const Vec16<__nv_bfloat16>*) {
    const float r = __fdiv_rn(127.f, a);
    return __fmaf_rn(r, a, -127.f) < 0.f ? __uint_as_float(__float_as_uint(r) + 1u) : r;
}
template <typename V>
__device__ __forceinline__ uint4 quant16(const V& x, float a, float inv) {
    constexpr bool kCheck = sizeof(V) == sizeof(Vec16<float>);   // fp32 rows
    const uint64_t inv2 = pair2(inv, inv), magic2 = pair2(kMagic, kMagic);
    float t[16];   // the low byte of t's bits is the whole number
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t xx = pair2(x.lo(i), x.hi(i));
        const uint64_t tt = fma2(xx, inv2, magic2);
        if constexpr (kCheck) {
            const uint64_t rem = fma2(xx, inv2, fma2(tt, pair2(-1.f, -1.f), magic2));   // x inv - whole
            float r0, r1;
            split2(rem, r0, r1);
            worst = fmaxf(worst, fmaxf(fabsf(r0), fabsf(r1)));
        }
        split2(tt, t[2 * i], t[2 * i + 1]);
    }
    if constexpr (kCheck) {
        if (worst > 0.4999f) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = i & 1 ? x.hi(i / 2) : x.lo(i / 2), r = t[i] - kMagic, rem = fmaf(v, inv, -r);
                if (fabsf(rem) > 0.4999f) t[i] = border(v, a, r, rem) + kMagic;
            }
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
// the row; a longer row is read twice past that. The users walk rows with two
// register buffers, the next row's reads running under this one's arithmetic
// and stores: 75.5 us against 79 with a row a block (11 k rows of 14336 bf16,
// 95 % of the copy bandwidth), 14.8 against 16.0 in the permutation of 4096 rows of 4096.
// hold_row starts the reads, quantize_row finishes. red: TPR / 32 floats of
// shared memory when TPR > 32, another half of it for every other row; the
// row's threads meet at a barrier of their own. Returns scale_r; put(v, w)
// stores vector v.

// The TPR threads of one row meet (a block has block_of(TPR) / TPR rows).
template <int TPR>
__device__ __forceinline__ void row_barrier() {
    if constexpr (TPR == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / TPR), "n"(TPR) : "memory");
}
template <typename T> constexpr int kHold = sizeof(T) == 2 ? 4 : 2;   // registers: 32 a buffer
template <typename T, int TPR>
__device__ __forceinline__ void hold_row(Vec16<T> (&held)[kHold<T>], const T* xr, int nv, int tid) {
#pragma unroll
    for (int h = 0; h < kHold<T>; ++h)
        if (tid + h * TPR < nv) held[h].load(xr + static_cast<size_t>(tid + h * TPR) * 16);
}
template <typename T, int TPR, typename Put>
__device__ __forceinline__ float quantize_row(const Vec16<T> (&held)[kHold<T>], const T* xr, int nv, int tid,
                                              float* red, Put put) {
    float a = 0.f;
#pragma unroll
    for (int h = 0; h < kHold<T>; ++h)
        if (tid + h * TPR < nv) a = held[h].amax(a);
    for (int v = tid + kHold<T> * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        a = w.amax(a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    if constexpr (TPR > 32) {
        if ((tid & 31) == 0) red[tid >> 5] = a;
        row_barrier<TPR>();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) a = max_nan(a, red[w]);
    }
    const bool live = !(a < kTinyRow);
    const float inv = live ? inverse(a, &held[0]) : 0.f;
#pragma unroll
    for (int h = 0; h < kHold<T>; ++h)
        if (tid + h * TPR < nv) put(tid + h * TPR, quant16(held[h], a, inv));
    for (int v = tid + kHold<T> * TPR; v < nv; v += TPR) {
        Vec16<T> w;
        w.load(xr + static_cast<size_t>(v) * 16);
        put(v, quant16(w, a, inv));
    }
    return live ? __fdiv_rn(a, 127.f) + (a - a) : 0.f;   // a - a: 0, or NaN where a is not finite
}
// Threads of a block, and rows it works on at a time
constexpr int block_of(int tpr) { return tpr < 128 ? 128 : tpr; }
// Threads a row: the fewest whose registers hold it
template <typename T> int threads_of(int cols) {
    if (cols <= 32 * 16 * kHold<T>) return 32;
    if (cols <= 64 * 16 * kHold<T>) return 64;
    if (cols <= 128 * 16 * kHold<T>) return 128;
    return sizeof(T) == 2 || cols <= 256 * 16 * kHold<T> ? 256 : 512;
}
// Blocks for `rows` rows: at most the 512 threads an SM that are resident at 125 registers each
inline int grid_of(int rows, int tpr) {
    const int rpb = block_of(tpr) / tpr, sms = device_sm_count();
    const int most = (sms > 0 ? sms : 148) * (512 / block_of(tpr));
    const int need = ceil_div(rows, rpb);
    return need < most ? need : most;
}

template <typename T, int TPR>
__global__ void __launch_bounds__(block_of(TPR))
quantize_kernel(const T* x, int rows, int cols, const int32_t* used, int8_t* q, float* scale) {
    constexpr int RPB = block_of(TPR) / TPR;
    __shared__ float red[RPB][2][TPR / 32];
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR, nv = cols / 16;
    pdl_wait();
    pdl_launch();
    const int step = gridDim.x * RPB;
    int row = blockIdx.x * RPB + sub;
    auto at = [&](int r) { return x + static_cast<size_t>(r) * cols; };
    Vec16<T> A[kHold<T>], B[kHold<T>];
    // the first row's reads start beside that of *used (a row that is not used is read for nothing)
    if (row < rows) hold_row<T, TPR>(A, at(row), nv, tid);
    const int n = used != nullptr ? min(rows, *used) : rows;
    // the threads of a row leave together
    auto one = [&](const Vec16<T> (&cur)[kHold<T>], Vec16<T> (&next)[kHold<T>], int half) {
        if (step < n - row) hold_row<T, TPR>(next, at(row + step), nv, tid);
        uint4* qr = reinterpret_cast<uint4*>(q + static_cast<size_t>(row) * cols);
        const float sc = quantize_row<T, TPR>(cur, at(row), nv, tid, red[sub][half], [&](int v, const uint4& w) { qr[v] = w; });
        if (tid == 0) scale[row] = sc;
        if (step >= n - row) return false;
        row += step;
        return true;
    };
    if (row >= n) return;
    while (one(A, B, 0) && one(B, A, 1)) {}
}

template <typename T>
cudaError_t quantize_t(const T* x, int rows, int cols, const int32_t* used, int8_t* q, float* scale, cudaStream_t st) {
    const int tpr = threads_of<T>(cols);
    const dim3 grid(grid_of(rows, tpr)), block(block_of(tpr));
    if (tpr == 32) return launch_dep(quantize_kernel<T, 32>, grid, block, 0, st, x, rows, cols, used, q, scale);
    if (tpr == 64) return launch_dep(quantize_kernel<T, 64>, grid, block, 0, st, x, rows, cols, used, q, scale);
    if (tpr == 128) return launch_dep(quantize_kernel<T, 128>, grid, block, 0, st, x, rows, cols, used, q, scale);
    if constexpr (sizeof(T) == 4)
        if (tpr == 512) return launch_dep(quantize_kernel<T, 512>, grid, block, 0, st, x, rows, cols, used, q, scale);
    return launch_dep(quantize_kernel<T, 256>, grid, block, 0, st, x, rows, cols, used, q, scale);
}

// ---- permutation with the rows in 8 bits ------------------------------------------
// TPR threads take a token and every so many after it: they start reading its
// row, find the destinations of its pairs, write pos and row_token, and
// quantise the row once into all of its destinations. Padding
// rows of the padded layout are shared out over the blocks by expert.
//  FEW (at most kFewPairs pairs): one launch does it all. Every block counts
//  all pairs and scans the experts by itself; a pair's rank is the number of
//  pairs of its expert before it in the drop order. Block 0 writes indptr
//  and the statistics.
//  Otherwise i8_count_kernel has counted every chunk of kChunk tokens and left
//  each pair's rank in its chunk in pos, and i8_scan_kernel the chunk bases,
//  indptr and the statistics: a destination is three loads and two sums.
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

// the statistics' header of a permutation (P, f and the router's fields stay)
__device__ __forceinline__ void write_header(const PermuteArgs& a, int kept, int all, int most) {
    moe_stats* st = static_cast<moe_stats*>(a.stats);
    st->status = MOE_OK;
    st->capacity = a.capacity;
    st->rows = kept;
    st->dropped = all - kept;
    st->max_count = most;
    st->max_over_mean = static_cast<float>(most) / (static_cast<float>(a.T) * static_cast<float>(a.k) / static_cast<float>(a.E));
    st->reserved[0] = st->reserved[1] = 0;
}

// Expert counts of a chunk (blockcnt [E][kk][NB], as the router leaves them),
// and for every pair the number of pairs before it in the chunk that compete
// for the same rows: the same expert and, under the slot order, the same slot.
constexpr int kCountThreads = 256;
__global__ void __launch_bounds__(kCountThreads)
i8_count_kernel(const int32_t* idx, int T, int k, int kk, int E, int NB, int32_t* blockcnt, int32_t* pos) {
    __shared__ int cnt[kMaxSlotCounts];
    __shared__ int s_idx[kChunk * MOE_MAX_K];
    pdl_wait();
    pdl_launch();
    const int chunk = blockIdx.x, t0 = chunk * kChunk, n = min(kChunk, T - t0) * k;
    for (int i = threadIdx.x; i < E * kk; i += kCountThreads) cnt[i] = 0;
    for (int i = threadIdx.x; i < n; i += kCountThreads) s_idx[i] = idx[static_cast<size_t>(t0) * k + i];
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kCountThreads) {
        const int e = s_idx[i];
        if (e < 0 || e >= E) continue;
        int before = 0;
        if (kk > 1) {
            for (int v = i % k; v < i; v += k) before += s_idx[v] == e;
        } else {
            for (int v = 0; v < i; ++v) before += s_idx[v] == e;
        }
        pos[static_cast<size_t>(t0) * k + i] = before;
        atomicAdd(&cnt[e * kk + (kk > 1 ? i % k : 0)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < E * kk; i += kCountThreads) blockcnt[static_cast<size_t>(i) * NB + chunk] = cnt[i];
}

// One block: the chunk bases of every expert (prefix over its (slot, chunk)
// counts), then capacity, padded row offsets and statistics per expert.
// A warp takes four experts at a time, so that their loads overlap, or one where
// there are no more than warps.
constexpr int kScan8Threads = 1024;
template <int X>   // experts a warp takes at a time
__global__ void __launch_bounds__(kScan8Threads) i8_scan_kernel(const __grid_constant__ PermuteArgs a, const int32_t* blockcnt,
                                                                int32_t* blockoff) {
    __shared__ int s_cnt[MOE_MAX_E], s_held[32], s_red[3][32];
    pdl_wait();
    pdl_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int len = a.kk * a.NB;
    constexpr int U = 4;   // steps of 32 entries in flight
    for (int e0 = warp * X; e0 < a.E; e0 += 32 * X) {
        int carry[X] = {};
        for (int b0 = 0; b0 < len; b0 += 32 * U) {
            int v[X][U];
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = b0 + 32 * u + lane;
                    v[x][u] = e0 + x < a.E && i < len ? blockcnt[static_cast<size_t>(e0 + x) * len + i] : 0;
                }
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    int incl = v[x][u];
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int w = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += w;
                    }
                    const int i = b0 + 32 * u + lane;
                    if (e0 + x < a.E && i < len) blockoff[static_cast<size_t>(e0 + x) * len + i] = carry[x] + incl - v[x][u];
                    carry[x] += __shfl_sync(0xffffffffu, incl, 31);
                }
        }
#pragma unroll
        for (int x = 0; x < X; ++x)
            if (lane == 0 && e0 + x < a.E) s_cnt[e0 + x] = carry[x];
    }
    __syncthreads();
    // experts: one thread each (E <= 512)
    const int e = threadIdx.x;
    const int c = e < a.E ? s_cnt[e] : 0;
    const int kp = a.capacity < 0 ? c : min(c, a.capacity);
    const int held = a.pad > 0 ? (kp + a.pad - 1) / a.pad * a.pad : kp;
    int incl = held;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) s_held[warp] = incl;
    const int kept_w = __reduce_add_sync(0xffffffffu, kp), all_w = __reduce_add_sync(0xffffffffu, c),
              most_w = __reduce_max_sync(0xffffffffu, c);
    if (lane == 0) {
        s_red[0][warp] = kept_w;
        s_red[1][warp] = all_w;
        s_red[2][warp] = most_w;
    }
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += s_held[w];
    if (e < a.E) {
        a.indptr[e] = base + incl - held;
        MOE_STATS_COUNTS(a.stats, a.E)[e] = c;
        MOE_STATS_KEPT(a.stats, a.E)[e] = kp;
        if (e == a.E - 1) a.indptr[a.E] = base + incl;
    }
    if (warp == 0) {
        const int kept = __reduce_add_sync(0xffffffffu, s_red[0][lane]), all = __reduce_add_sync(0xffffffffu, s_red[1][lane]);
        const int most = __reduce_max_sync(0xffffffffu, s_red[2][lane]);
        if (lane == 0) write_header(a, kept, all, most);
    }
}

template <typename T, int TPR, bool FEW>
__global__ void __launch_bounds__(block_of(TPR))
permute_i8_kernel(const __grid_constant__ PermuteArgs a) {
    constexpr int kThreads = block_of(TPR), kTokens = kThreads / TPR;
    __shared__ int s_idx[FEW ? kFewPairs : 1];
    __shared__ int s_cnt[FEW ? MOE_MAX_E : 1], s_ptr[FEW ? MOE_MAX_E + 1 : 1];
    __shared__ int s_pos[2][kTokens][MOE_MAX_K];
    __shared__ float red[kTokens][2][TPR / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR, nv = a.d / 16;
    const int step = gridDim.x * kTokens;
    int t = blockIdx.x * kTokens + sub;
    auto row_of = [&](int tok) { return static_cast<const T*>(a.x) + static_cast<size_t>(tok) * a.d; };
    Vec16<T> A[kHold<T>], B[kHold<T>];
    if constexpr (FEW) pdl_wait();
    if (t < a.T) hold_row<T, TPR>(A, row_of(t), nv, tid);
    // The chunk bases and indptr come from the scan. The first rows need not wait for it: the scan lets this kernel start
    // after the count has ended, which itself has waited for all that came before.
    if constexpr (!FEW) pdl_wait();
    pdl_launch();
    const int np = a.T * a.k;
    if constexpr (FEW) {
        for (int i = threadIdx.x; i < np; i += kThreads) s_idx[i] = a.idx[i];
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
                    write_header(a, kept_all, all, most);
                }
            }
        }
    }
    __syncthreads();
    if (a.pad > 0) {
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
    // !FEW: the first half of a destination (expert and rank in the chunk) is
    // loaded a token ahead
    int e_next = -1, mine_next = 0;
    auto look = [&](int tok) {
        if (!FEW && tid < a.k) {
            const size_t p = static_cast<size_t>(tok) * a.k + tid;
            e_next = a.idx[p];
            mine_next = a.pos[p];
        }
    };
    auto one = [&](const Vec16<T> (&cur)[kHold<T>], Vec16<T> (&next)[kHold<T>], int half) {
        int* dst = s_pos[half][sub];
        const bool more = step < a.T - t;
        if constexpr (FEW) {
            // a warp a pair, its lanes over the pairs that can stand before it
            for (int j = tid >> 5; j < a.k; j += TPR / 32) {
                const int p = t * a.k + j, e = s_idx[p];
                int at = -1;
                if (e >= 0 && e < a.E) {
                    int before = 0;
                    if (a.kk > 1) {   // slot order: earlier slots first
                        for (int v = lane; v < np; v += 32) {
                            const int jj = v % a.k;
                            before += s_idx[v] == e && (jj < j || (jj == j && v < p));
                        }
                    } else {
                        for (int v = lane; v < p; v += 32) before += s_idx[v] == e;
                    }
                    before = __reduce_add_sync(0xffffffffu, before);
                    if (a.capacity < 0 || before < a.capacity) at = s_ptr[e] + before;
                }
                if (lane == 0) {
                    dst[j] = at;
                    a.pos[p] = at;
                    if (at >= 0) a.row_token[at] = t;
                }
            }
        } else if (tid < a.k) {
            int at = -1;
            if (e_next >= 0 && e_next < a.E) {
                const size_t row = static_cast<size_t>(e_next) * a.kk + (a.kk > 1 ? tid : 0);
                const int rank = a.blockoff[row * a.NB + t / kChunk] + mine_next;
                if (a.capacity < 0 || rank < a.capacity) at = a.indptr[e_next] + rank;
            }
            dst[tid] = at;
            a.pos[static_cast<size_t>(t) * a.k + tid] = at;
            if (at >= 0) a.row_token[at] = t;
        }
        if (more) {
            hold_row<T, TPR>(next, row_of(t + step), nv, tid);
            look(t + step);
        }
        row_barrier<TPR>();
        const float sc = quantize_row<T, TPR>(cur, row_of(t), nv, tid, red[sub][half], [&](int v, const uint4& w) {
            for (int j = 0; j < a.k; ++j)
                if (dst[j] >= 0) reinterpret_cast<uint4*>(a.xq + static_cast<size_t>(dst[j]) * a.d)[v] = w;
        });
        if (tid < a.k && dst[tid] >= 0) a.xs[dst[tid]] = sc;
        t += step;
        return more;
    };
    if (t >= a.T) return;   // the threads of a token leave together
    look(t);
    while (one(A, B, 0) && one(B, A, 1)) {}
}

template <typename T, bool FEW>
cudaError_t permute_t(const PermuteArgs& a, cudaStream_t st) {
    const int tpr = threads_of<T>(a.d);
    const dim3 grid(grid_of(a.T, tpr)), block(block_of(tpr));
    if (tpr == 32) return launch_dep(permute_i8_kernel<T, 32, FEW>, grid, block, 0, st, a);
    if (tpr == 64) return launch_dep(permute_i8_kernel<T, 64, FEW>, grid, block, 0, st, a);
    if (tpr == 128) return launch_dep(permute_i8_kernel<T, 128, FEW>, grid, block, 0, st, a);
    if constexpr (sizeof(T) == 4)
        if (tpr == 512) return launch_dep(permute_i8_kernel<T, 512, FEW>, grid, block, 0, st, a);
    return launch_dep(permute_i8_kernel<T, 256, FEW>, grid, block, 0, st, a);
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
    cudaError_t e = launch_dep(i8_count_kernel, dim3(a.NB), dim3(kCountThreads), 0, st, p.idx, p.T, p.k, p.kk, p.E, a.NB,
                             p.blockcnt, p.pos);
    if (e != cudaSuccess) return e;
    e = launch_dep(p.E <= 32 ? i8_scan_kernel<1> : i8_scan_kernel<4>, dim3(1), dim3(kScan8Threads), 0, st, a, static_cast<const int32_t*>(p.blockcnt), p.blockoff);
    if (e != cudaSuccess) return e;
    return p.dtype == MOE_DTYPE_BF16 ? permute_t<__nv_bfloat16, false>(a, st) : permute_t<float, false>(a, st);
}

}  // namespace moe
