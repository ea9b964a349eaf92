// C ABI of the operators beside the layer: argument checks, the workspace of
// the 8-bit experts and the launch sequences. Every launch is asynchronous on
// the caller's stream; the host never waits on the device.
#include <cmath>

#include "ops.cuh"

namespace moe {

I8Layout make_i8_layout(const moe_problem& p) {
    const size_t T = p.T > 0 ? (size_t)p.T : 0, E = (size_t)p.E;
    const size_t NB = (T + kChunk - 1) / kChunk, kk = (size_t)count_slots(p);
    I8Layout L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        size_t o = off;
        off = align_up(off + (bytes > 0 ? bytes : 1), 256);
        return o;
    };
    L.blockcnt = take(E * kk * NB * 4);
    L.blockoff = take(E * kk * NB * 4);
    // sums of up to a grid of tail tiles: 256 channels by the rows of a tile
    const long long rows = permuted_rows(p);
    L.part_rows = (int)(rows < 128 ? (rows + 15) / 16 * 16 : 128);
    L.part = take((size_t)kI8MaxGrid * 256 * L.part_rows * 4);
    L.sem = take((size_t)kI8MaxGrid * 8 * 4);
    L.status = take(4);
    L.total = off;
    return L;
}

// CTA pairs need rows to fill their tiles of 256 x 512 (256 of SWIGLU), K
// blocks to outweigh what a tile costs besides them, channels in 7/10 of their
// tiles' and tiles for 6/10 of the SM pairs; the single form takes the rest.
// Measured, single / pair (us), by rows an expert and K:
//   K = 14336, 4096 channels, 8 experts: 144 rows 133 / 88, 256 rows 135 / 144, 448
//     rows 208 / 162; K = 4096, 2 x 14336 channels: 128 rows 177 / 199, 192 rows
//     221 / 212, 1024 rows 877 / 707
//   K = 2048, 2 x 1408 channels, 64 experts: 352 rows 142 / 154, 448 rows 186 / 167
//   K = 768, 2048 channels, 128 experts: 352 rows 109 / 120, 640 rows 189 / 178
//   K = 2048, 640 channels (5/8 of their tiles), 24 experts: 448 rows 26 / 32
// Over 120 such shapes the choice costs 0.3 % against the better form of each. One border
// serves both products of a K, and near it the other form can be ahead: of the figures
// above, up with 128 rows of K = 4096 (12 %), down with 256 rows of K = 14336 (7 %).
I8Form i8_form(const moe_problem& p, bool down) {
    const long long pairs = (long long)p.T * p.k, E = p.E;
    const int K = down ? p.d_ff : p.d, N = down ? p.d : p.d_ff, wide = down ? 512 : 256;
    if (pairs < (K >= 4096 ? 128 : K > 1024 ? 400 : 640) * E) return I8_SINGLE;
    const long long cols = ceil_div(N, wide);
    if (10ll * N < 7 * cols * wide) return I8_SINGLE;
    const long long blocks2 = pairs / 128 + E;   // blocks of 256 rows, half a block an expert for its ragged end, doubled
    const int sms = device_sm_count();
    return 5 * blocks2 * cols >= 3LL * (sms > 0 ? sms : 148) ? I8_PAIR : I8_SINGLE;
}

}  // namespace moe

using namespace moe;

namespace {

constexpr int kMaxI8K = 131071;   // K 128^2 stays below 2^31

#define CK(expr)                                   \
    do {                                           \
        if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
    } while (0)

bool ok16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// optional pointers: absent, or aligned
bool opt16(const void* p) { return p == nullptr || ok16(p); }

int check_int8(const moe_problem* p) {
    const int rc = check_problem(p);
    if (rc != MOE_OK) return rc;
    if (p->d % 16 || p->d_ff % 16 || p->d_ff_shared || p->d > kMaxI8K || p->d_ff > kMaxI8K) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// 0: dropout of probability prob from rng; MOE_ERR_* otherwise
int make_dropout(float prob, const uint64_t* rng, Dropout* d) {
    if (!(prob >= 0.f) || !(prob < 1.f)) return MOE_ERR_INVALID_ARG;
    const long thr = std::lround((double)prob * 65536.0);
    if (thr > 65535) return MOE_ERR_INVALID_ARG;
    d->rng = nullptr;
    d->thr = (unsigned)thr;
    d->scale = (float)(65536.0 / (65536.0 - (double)thr));
    if (thr == 0) return MOE_OK;
    if (rng == nullptr || (reinterpret_cast<uintptr_t>(rng) & 7u)) return MOE_ERR_INVALID_ARG;
    d->rng = reinterpret_cast<const unsigned long long*>(rng);
    return MOE_OK;
}

int i8_workspace(const moe_problem* p, void* ws, size_t bytes, I8Layout* L) {
    *L = make_i8_layout(*p);
    if (!ws || bytes < L->total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

int run_i8(const moe_problem* p, const int8_t* A, const float* sa, const int32_t* indptr, const int8_t* B0,
           const float* sb0, const int8_t* B1, const float* sb1, void* out, int N, int K, void* stats, void* workspace,
           const I8Layout& L, void* stream) {
    char* ws = static_cast<char*>(workspace);
    I8Gemm g = {};
    g.indptr = indptr; g.E = p->E;
    g.A = A; g.sa = sa; g.B0 = B0; g.sb0 = sb0; g.B1 = B1; g.sb1 = sb1;
    g.out = out; g.out_dtype = p->dtype; g.N = N; g.K = K; g.rows = (int)permuted_rows(*p);
    g.status = stats ? static_cast<int32_t*>(stats) : reinterpret_cast<int32_t*>(ws + L.status);
    g.form = i8_form(*p, B1 == nullptr);
    g.part = reinterpret_cast<int*>(ws + L.part); g.sem = reinterpret_cast<int*>(ws + L.sem); g.part_rows = L.part_rows;
    CK(launch_i8_tc(g, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_int8_workspace_size(const moe_problem* p) {
    if (check_int8(p) != MOE_OK) return 0;
    return make_i8_layout(*p).total;
}

int moe_int8_variant(const moe_problem* p, int down) {
    const int rc = check_int8(p);
    if (rc != MOE_OK) return -rc;
    return i8_form(*p, down != 0) == I8_PAIR ? MOE_INT8_PAIR : MOE_INT8_SINGLE;
}

int moe_quantize_rows(int32_t dtype, const void* x, int32_t rows, int32_t cols, const int32_t* used, int8_t* q,
                      float* scale, void* stream) {
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (cols % 16) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!ok16(x) || !ok16(q) || !ok4(scale) || (used != nullptr && !ok4(used))) return MOE_ERR_INVALID_ARG;
    CK(launch_quantize_rows(dtype, x, rows, cols, used, q, scale, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

int moe_permute_int8(const moe_problem* p, const void* x, const int32_t* idx, int32_t* pos, int32_t* indptr,
                     int32_t* row_token, int8_t* xq, float* xs, void* stats, void* workspace, size_t workspace_bytes,
                     void* stream) {
    int rc = check_int8(p);
    if (rc != MOE_OK) return rc;
    if (!ok4(idx) || !ok4(pos) || !ok4(indptr) || !ok4(row_token) || !ok16(stats) || !ok4(xs)) return MOE_ERR_INVALID_ARG;
    if (!ok16(x) || !ok16(xq)) return MOE_ERR_INVALID_ARG;
    I8Layout L;
    rc = i8_workspace(p, workspace, workspace_bytes, &L);
    if (rc != MOE_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int C = capacity_of(p);
    if (p->T == 0) {
        CK(launch_zero_stats(stats, p->E, C, st));
        CK(cudaMemsetAsync(indptr, 0, sizeof(int32_t) * (size_t)(p->E + 1), st));
        return MOE_OK;
    }
    char* ws = static_cast<char*>(workspace);
    PermuteI8 a = {};
    a.dtype = p->dtype; a.x = x; a.idx = idx;
    a.blockcnt = reinterpret_cast<int32_t*>(ws + L.blockcnt);
    a.blockoff = reinterpret_cast<int32_t*>(ws + L.blockoff);
    a.pos = pos; a.indptr = indptr; a.row_token = row_token; a.xq = xq; a.xs = xs; a.stats = stats;
    a.T = p->T; a.d = p->d; a.E = p->E; a.k = p->k; a.kk = count_slots(*p); a.capacity = C; a.pad = p->pad_rows;
    a.rows = (int)permuted_rows(*p);
    CK(launch_permute_i8(a, st));
    return MOE_OK;
}

int moe_expert_up_int8(const moe_problem* p, const int8_t* xq, const float* xs, const int32_t* indptr,
                       const int8_t* W1, const float* w1s, const int8_t* W3, const float* w3s, void* h, void* stats,
                       void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_int8(p);
    if (rc != MOE_OK) return rc;
    if (!ok16(xq) || !ok16(W1) || !ok16(W3) || !ok16(h) || !ok4(xs) || !ok16(w1s) || !ok16(w3s) || !ok4(indptr) || !opt16(stats))
        return MOE_ERR_INVALID_ARG;
    I8Layout L;
    rc = i8_workspace(p, workspace, workspace_bytes, &L);
    if (rc != MOE_OK) return rc;
    if (p->T == 0) return MOE_OK;
    return run_i8(p, xq, xs, indptr, W1, w1s, W3, w3s, h, p->d_ff, p->d, stats, workspace, L, stream);
}

int moe_expert_down_int8(const moe_problem* p, const int8_t* hq, const float* hs, const int32_t* indptr,
                         const int8_t* W2, const float* w2s, void* o, void* stats, void* workspace,
                         size_t workspace_bytes, void* stream) {
    int rc = check_int8(p);
    if (rc != MOE_OK) return rc;
    if (!ok16(hq) || !ok16(W2) || !ok16(o) || !ok4(hs) || !ok16(w2s) || !ok4(indptr) || !opt16(stats))
        return MOE_ERR_INVALID_ARG;
    I8Layout L;
    rc = i8_workspace(p, workspace, workspace_bytes, &L);
    if (rc != MOE_OK) return rc;
    if (p->T == 0) return MOE_OK;
    return run_i8(p, hq, hs, indptr, W2, w2s, nullptr, nullptr, o, p->d, p->d_ff, stats, workspace, L, stream);
}

int moe_combine_dropout(const moe_problem* p, const void* o, const int32_t* pos, const float* gate, const void* s,
                        const void* residual, float prob, const uint64_t* rng, void* out, void* stream) {
    int rc = check_problem(p);
    if (rc != MOE_OK) return rc;
    MixArgs a = {};
    rc = make_dropout(prob, rng, &a.drop);
    if (rc != MOE_OK) return rc;
    if (p->T == 0) return MOE_OK;
    if (!ok16(o) || !ok4(pos) || !ok4(gate) || !ok16(out) || !opt16(s) || !opt16(residual)) return MOE_ERR_INVALID_ARG;
    a.dtype = p->dtype; a.o = o; a.pos = pos; a.gate = gate; a.s = s; a.residual = residual; a.out = out;
    a.T = p->T; a.d = p->d; a.k = p->k; a.rows = (int)permuted_rows(*p);
    CK(launch_mix(a, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

int moe_combine_backward(const moe_problem* p, const void* dy, const void* o, const int32_t* pos, const float* gate,
                         float prob, const uint64_t* rng, const int32_t* indptr, const int32_t* row_token, void* dO,
                         float* dgate, void* ds, void* stream) {
    int rc = check_problem(p);
    if (rc != MOE_OK) return rc;
    MixBackArgs a = {};
    rc = make_dropout(prob, rng, &a.drop);
    if (rc != MOE_OK) return rc;
    if (p->T == 0) return MOE_OK;
    if (!ok16(dy) || !ok16(o) || !ok4(pos) || !ok4(gate) || !ok16(dO) || !ok4(dgate) || !opt16(ds)) return MOE_ERR_INVALID_ARG;
    if (p->pad_rows > 0) {
        if (!ok4(indptr) || !ok4(row_token)) return MOE_ERR_INVALID_ARG;
        a.indptr = indptr; a.row_token = row_token;
    }
    a.dtype = p->dtype; a.dy = dy; a.o = o; a.pos = pos; a.gate = gate; a.dO = dO; a.dgate = dgate; a.ds = ds;
    a.T = p->T; a.d = p->d; a.k = p->k; a.rows = (int)permuted_rows(*p); a.E = p->E;
    CK(launch_mix_back(a, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

int moe_permute_backward(const moe_problem* p, const void* dxp, const int32_t* pos, void* dx, void* stream) {
    int rc = check_problem(p);
    if (rc != MOE_OK) return rc;
    if (p->T == 0) return MOE_OK;
    if (!ok16(dxp) || !ok4(pos) || !ok16(dx)) return MOE_ERR_INVALID_ARG;
    MixArgs a = {};
    a.dtype = p->dtype; a.o = dxp; a.pos = pos; a.out = dx;
    a.T = p->T; a.d = p->d; a.k = p->k; a.rows = (int)permuted_rows(*p);
    CK(launch_mix(a, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

}  // extern "C"
