// Declarations of the operators beside the layer: products in 8-bit integers
// (quantisation, permutation, grouped products) and the way back with
// dropout, residual and gradients.
#pragma once

#include "common.cuh"

namespace moe {

// Launch as a programmatic dependent of whatever precedes it on the stream:
// the kernel's own launch and prologue overlap the end of the one before,
// and it calls pdl_wait() (which returns when everything before has completed
// and is visible) in every thread before it touches global memory, so calls
// order as ever. The short kernels call pdl_launch() early for the next one;
// the products do not (a next product's first kernel waiting beside them cost
// 1 us of 43 where it should have saved some).
struct DependentLaunch {
    DependentLaunch() : was(g_pdl) { g_pdl = true; }
    ~DependentLaunch() { g_pdl = was; }
    bool was;
};
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dep(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args&&... args) {
    DependentLaunch dependent;
    return launch_k(kernel, grid, block, smem, st, std::forward<Args>(args)...);
}

// ---- 8-bit experts ----------------------------------------------------------

// Byte offsets of moe_int8_workspace_size(p) bytes.
struct I8Layout {
    size_t blockcnt, blockoff;   // permutation: per-chunk expert counts and their scan
    size_t part, sem;            // products: sums and arrival counters of the tail tiles
    int part_rows;               // rows of a tile's sums
    size_t status;               // status word of a call without a statistics block
    size_t total;
};
I8Layout make_i8_layout(const moe_problem& p);

// One product of the experts: out[r][n] over the rows of every group.
enum I8Form { I8_SINGLE = 0, I8_PAIR = 1 };
constexpr int kI8MaxGrid = 160;   // CTAs of the single form at most: sizes the workspace on any host
I8Form i8_form(const moe_problem& p, bool down);
struct I8Gemm {
    int form;
    const int32_t* indptr;   // [E+1] (device)
    int E;
    const int8_t* A;         // [rows, K]
    const float* sa;         // [rows]
    const int8_t* B0;        // [E, N, K]
    const float* sb0;        // [E, N]
    const int8_t* B1;        // second weight of the SwiGLU form, or null
    const float* sb1;
    void* out;               // [rows, N] bf16 or fp32
    int out_dtype;
    int N, K, rows;
    int32_t* status;
    int *part, *sem;         // single form: sums of the tail tiles and their arrival counters
    int part_rows;
};
cudaError_t launch_i8_tc(const I8Gemm& g, cudaStream_t st);

// rows of x -> q, scale; only the first min(rows, *used) rows when used != null
cudaError_t launch_quantize_rows(int dtype, const void* x, int rows, int cols, const int32_t* used, int8_t* q,
                                 float* scale, cudaStream_t st);
// the permutation of moe_permute with the rows in 8 bits
struct PermuteI8 {
    int dtype;
    const void* x;
    const int32_t* idx;
    int32_t *blockcnt, *blockoff;   // workspace: per-chunk expert counts and their scan
    int32_t *pos, *indptr, *row_token;
    int8_t* xq;
    float* xs;
    void* stats;
    int T, d, E, k, kk, capacity, pad, rows;
};
cudaError_t launch_permute_i8(const PermuteI8& a, cudaStream_t st);

// ---- the way back -----------------------------------------------------------

// Dropout of [T, d] values: keep element i = t d + c when the 16-bit half
// i % 8 of the generator's block i / 8 is at least thr; scale = 65536 / (65536 - thr).
struct Dropout {
    const unsigned long long* rng;   // {seed, offset} (device); null: no dropout
    unsigned thr;
    float scale;
};
struct MixArgs {
    int dtype;
    const void* o;           // [rows, d]
    const int32_t* pos;      // [T, k]
    const float* gate;       // [T, k], or null: every gate is 1
    const void* s;           // [T, d] or null
    const void* residual;    // [T, d] or null
    void* out;               // [T, d]
    int T, d, k, rows;
    Dropout drop;
};
cudaError_t launch_mix(const MixArgs& a, cudaStream_t st);

struct MixBackArgs {
    int dtype;
    const void* dy;          // [T, d]
    const void* o;           // [rows, d]
    const int32_t* pos;
    const float* gate;
    void* dO;                // [rows, d]
    float* dgate;            // [T, k]
    void* ds;                // [T, d] or null
    const int32_t* indptr;   // padded layouts: [E+1] and row_token [rows], else null
    const int32_t* row_token;
    int T, d, k, rows, E;
    Dropout drop;
};
cudaError_t launch_mix_back(const MixBackArgs& a, cudaStream_t st);

}  // namespace moe
