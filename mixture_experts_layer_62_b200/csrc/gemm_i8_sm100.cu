// Products of the experts in 8-bit integers on the sm_100a tensor cores
// (tcgen05 kind::i8, 32-bit integer accumulators in TMEM, TMA-fed): for every
// group e and row r of it, with a scale for each token and channel,
//   PLAIN   out[r][n] = S(A, B0) sa_r sb0_{e,n},  S(A, B) = sum_c A[r][c] B_e[n][c]
//   SWIGLU  a = S(A, B0) sa sb0, b = S(A, B1) sa sb1, out = SiLU(a) b
// The integer sums are exact (K 128^2 < 2^31), so no order of K, tile or form
// of the kernel changes a bit of the result; the float factors are applied
// as (float(sum) * sa) * sb and the result is rounded once.
//
// Two forms, both persistent kernels: one warp loads by TMA into a ring of
// 128-byte K blocks (128-byte swizzle), one issues the MMAs, sixteen (or eight)
// read the accumulators back (tcgen05.ld), apply the scales and store: half of
// them to each of the two accumulators, which the tiles take in turn. The tile
// list is formed in each CTA's shared memory from the group offsets. Every wait
// is bounded (moe_set_wait_limit): on expiry the CTA records MOE_ERR_TIMEOUT and
// its warps leave their loops. One that had come to its end before may have left
// copies or MMAs behind that the others no longer wait for, so what was started
// lands after all warps have met: then the CTA frees its tensor memory and returns.
//  * pair: clusters of two CTAs share tiles of 256 rows of A x 512 weight
//    rows (cta_group::2), each CTA loading half of both; groups of many rows.
//    Bound by the tensor pipe and the board's power: 8192 rows, K = 14336,
//    18944 channels run at 3.3 P operations/s, twice the measured bf16 GEMM
//    rate; with K = 4096 (Mixtral-shaped up projection, 8 experts, 690 us, 2.8
//    P/s) the SwiGLU epilogue and the ragged blocks show. What the tile's
//    width buys: with 256 x 256 tiles the L2 has to deliver a third more bytes
//    for the same products, and K = 14336 took 1449 us instead of 1365.
//  * single: one CTA a tile of 256 weight rows and up to 128 rows of A, for
//    groups of few rows. Bound by the weight stream: 24 tokens of the
//    Mixtral-shaped up projection (941 MB) take 141 us, 6.7 TB/s; 256 experts
//    of 64 rows (7.5 GB) 1.19 ms, 98 % of the measured copy bandwidth, with DRAM
//    traffic equal to the bytes of the operands.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "ops.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int BKB = 128;                    // bytes of K a stage: one swizzle row
constexpr int BM = 128;                     // rows of A a CTA
constexpr int A_BYTES = BM * BKB;           // 16 KB
constexpr int BH_BYTES = 128 * BKB;         // 128 weight rows, 16 KB
constexpr int ACC_COLS = 256, TMEM_COLS = 512;
constexpr int P_STAGES = 4, P_STAGE_BYTES = A_BYTES + 2 * BH_BYTES;
constexpr int EPI = 16, NUM_THREADS = 64 + 32 * EPI;   // epilogue warps, threads
constexpr int P_STAGE_FLOATS = 256;                 // pair: stage of an epilogue warp, or its half of a trade [8 rows][32 channels]
constexpr int P_SCALE_FLOATS = 128;                 // pair: the scales of a warp's columns
constexpr int S_STAGES = 4, S_STAGE_BYTES = A_BYTES + 2 * BH_BYTES;
constexpr int S_ROW_FLOATS = 64;                    // single: the row scales of a warp's columns
constexpr long long kBandBytes = 32ll << 20;   // rows of A that a band of M blocks keeps in L2

// kind::i8: A and B signed 8-bit, D signed 32-bit, both operands K-major
constexpr uint32_t idesc_i8(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

struct KP {
    const int32_t* indptr;
    const float *sa, *sb0, *sb1;
    void* out;
    int32_t* status;
    long long timeout_ns, drain_ns;
    int E, N, K, rows, nt, band_m;
    int *part, *sem;   // single form: parts of the tail tiles [slots][part_rows][256] and arrivals [tail][8]
    int part_rows;
};

template <int STAGES>
struct Ctl {
    uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t loaded;          // K blocks that the CTA has requested, written as its loads end
    uint32_t bytes[STAGES];   // pair: what it has requested of the last block in each stage
    int cum[MOE_MAX_E + 1];   // tiles before group g
    int row0[MOE_MAX_E + 1];  // first row of group g
    int most;                 // rows of the tallest tile
};

// Tiles of every group in front of it, by one warp: cum[0..E], row0[0..E]. A
// group whose offsets do not fit in the rows has none.
template <int STAGES>
__device__ __forceinline__ void list_tiles(Ctl<STAGES>* c, const KP& p, int tile_m) {
    const int lane = threadIdx.x & 31;
    int base = 0, most = 0;
    bool bad = false;
    // eight times 32 groups' offsets requested at once: one memory round trip up to 256 experts
    for (int b0 = 0; b0 < p.E; b0 += 256) {
        int lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = b0 + 32 * i + lane;
            lo[i] = g < p.E ? p.indptr[g] : 0;
            hi[i] = g < p.E ? p.indptr[g + 1] : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = b0 + 32 * i + lane;
            if (b0 + 32 * i >= p.E) break;
            const bool ok = lo[i] >= 0 && hi[i] >= lo[i] && hi[i] <= p.rows;
            const int n = ok ? hi[i] - lo[i] : 0;
            bad |= !ok;
            most = max(most, n);
            const int v = (n + tile_m - 1) / tile_m * p.nt;
            int incl = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            if (g < p.E) {
                c->row0[g] = lo[i];
                if (g == p.E - 1) c->row0[p.E] = hi[i];
                c->cum[g] = base + incl - v;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        c->cum[p.E] = base;
        c->most = min(most, tile_m);
    }
    if (kDebugChecks && __any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) debug_record_bounds(p.status);
}

struct Tile {
    int g, rows, row0, m_blk, n_blk;
};
// Tile `id`: M blocks fastest inside a band of band_m M blocks, so that the
// CTAs running together share weight tiles and a band's rows of A stay in L2.
template <int STAGES>
__device__ __forceinline__ Tile tile_of(const Ctl<STAGES>* c, const KP& p, int id, int tile_m) {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c->cum[mid] <= id) lo = mid; else hi = mid;
    }
    Tile t;
    t.g = lo;
    t.row0 = c->row0[lo];
    t.rows = c->row0[lo + 1] - t.row0;
    id -= c->cum[lo];
    const int mt = (t.rows + tile_m - 1) / tile_m;
    int h = mt, m0 = 0;
    if (p.band_m < mt) {
        const int per = p.band_m * p.nt, band = id / per;
        id -= band * per;
        m0 = band * p.band_m;
        h = min(p.band_m, mt - m0);
    }
    t.n_blk = id / h;
    // turned by one from each weight tile to the next, so that a CTA's units
    // (a fixed stride apart) do not meet the short last block every time
    t.m_blk = m0 + (id + t.n_blk) % h;
    return t;
}

template <typename C>
__device__ __forceinline__ bool wait_i8(uint64_t* bar, uint32_t parity, C* ctl, const KP& p, uint32_t peer_abort = 0) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
        if (global_timer_ns() - t0 > static_cast<uint64_t>(p.timeout_ns)) {
            *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
            if (peer_abort) st_shared_remote_u32(peer_abort, 1u);
            atomicExch(p.status, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}
// After a wait gave up: copies and MMAs in flight land before the CTA leaves.
__device__ __forceinline__ void drain_i8(uint64_t* bar, uint32_t parity, const KP& p) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > static_cast<uint64_t>(p.drain_ns)) {
            atomicExch(p.status, MOE_ERR_TIMEOUT);
            return;
        }
}

// The last requests of every stage: block j of `n` completes phase (j / STAGES) % 2 of full[j % STAGES].
template <int STAGES>
__device__ __forceinline__ void drain_loads(Ctl<STAGES>* ctl, uint32_t n, const KP& p) {
#pragma unroll 1
    for (uint32_t j = n > STAGES ? n - STAGES : 0; j < n; ++j) drain_i8(&ctl->full[j % STAGES], (j / STAGES) & 1u, p);
}

// ---- epilogue arithmetic -------------------------------------------------------
// Two fp32 values an instruction (f32x2: each rounded as the scalar form).
__device__ __forceinline__ uint64_t pk(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpk(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kNegLog2e = -1.4426950408889634f;
// SiLU(a) b = (a / (1 + exp(-a))) b. bf16 results: the fast exponential and
// reciprocal (a few 2^-23 off, where the type rounds to 2^-8); fp32 results:
// the accurate exponential, and the reciprocal of one unit in the last place
// with subnormal results kept (a divide in its place: 156 us where this takes
// 100; 3000 rows, K = 64, 11328 channels). Against 64 bits the results of eight
// shapes, K = 64 to 4096, are 1.41 to 1.49 steps of 2^-24 off (rms); with the
// reciprocal corrected by a Newton step 1.39 to 1.48, and up to 6 % later. exp(-a) overflowing gives a 0, as it should.
__device__ __forceinline__ float rcp_full(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float swiglu(float a, float b, float*) {
    return __fmul_rn(__fmul_rn(a, rcp_full(__fadd_rn(1.f, expf(-a)))), b);
}
__device__ __forceinline__ uint64_t swiglu2(uint64_t a, uint64_t b, __nv_bfloat16*) {
    const float2 t = unpk(mul2(a, pk(kNegLog2e, kNegLog2e)));
    const float2 d = unpk(add2(pk(ex2(t.x), ex2(t.y)), pk(1.f, 1.f)));
    return mul2(mul2(a, pk(rcp(d.x), rcp(d.y))), b);
}
__device__ __forceinline__ uint64_t swiglu2(uint64_t a, uint64_t b, float* o) {
    const float2 x = unpk(a), y = unpk(b);
    return pk(swiglu(x.x, y.x, o), swiglu(x.y, y.y, o));
}
// (float(sum) sa) sb for two sums
__device__ __forceinline__ uint64_t scaled2(uint32_t s0, uint32_t s1, uint64_t sa, uint64_t sb) {
    return mul2(mul2(pk(static_cast<float>(static_cast<int>(s0)), static_cast<float>(static_cast<int>(s1))), sa), sb);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// the first n (at most CNT) of v, one under another
template <int CNT, typename OutT>
__device__ __forceinline__ void put_rows(OutT* o, int stride, int n, const float* v) {
    if (n >= CNT) {
#pragma unroll
        for (int j = 0; j < CNT; ++j) put(o + static_cast<size_t>(j) * stride, v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < CNT - 1; ++j)
            if (j < n) put(o + static_cast<size_t>(j) * stride, v[j]);
    }
}

// Stage of a warp: 32 rows of 32 bytes, in the order of a 32-byte swizzle:
// piece p (16 bytes) of a row lies at p ^ ((row / 4) % 2), so that eight lanes
// fall on different banks both here and when rows are read back.
__device__ __forceinline__ uint4* stage_at(uint8_t* st, int row, int p) {
    return reinterpret_cast<uint4*>(st + row * 32 + ((p ^ ((row >> 2) & 1)) << 4));
}
__device__ __forceinline__ void stage_run(uint8_t* st, int row, const float* v, float*) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *stage_at(st, row, i) = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                           __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
}
__device__ __forceinline__ void stage_run(uint8_t* st, int row, const float* v, __nv_bfloat16*) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    *stage_at(st, row, 0) = make_uint4(w[0], w[1], w[2], w[3]);
    *stage_at(st, row, 1) = make_uint4(w[4], w[5], w[6], w[7]);
}
// sixteen consecutive columns of this thread's TMEM lane, at one or two places
__device__ __forceinline__ void tmem_ld16(uint32_t t0, uint32_t (&a)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
          "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
        : "r"(t0)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16x2(uint32_t t0, uint32_t t1, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
          "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]),
          "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]),
          "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
        : "r"(t0), "r"(t1)
        : "memory");
}

// ---- pair form ----------------------------------------------------------------
// Whole tiles: the rows of A are the M operand (rank r holds rows [128 r, 128
// r + 128)), 256 weight rows the N operand (SWIGLU: rank 0 brings 128 rows of
// B0, rank 1 the same of B1, so the accumulator is [128 gates | 128 ups]).
// Short tiles, of at most kShort rows (the ragged end of a group): the
// weights are the M operand and the rows N = 32, 64, .., so they cost what
// they hold. With whole tiles alone a group of 1030 rows pays for 1280: eight
// experts of a random router lost 11 % that way. SWIGLU: rank r's M rows are
// B0's and B1's rows of its 64 channels, so TMEM lanes 0..63 (epilogue warps
// q = 0, 1) hold the gates and lanes 64..127 (q = 2, 3) the up values of the
// same channels; warps q and q + 2 trade halves of every 32 columns through
// shared memory: each sends 16, receives 16, and finishes 16 rows of its 32
// channels. (That trade is why whole tiles are not laid out this way too: it
// made the up projection of 8192 rows take 731 us instead of 710.) kShort
// between 64 and 192 measures the same within 2 %, 255 costs 3 to 5 %.
// Eight warps share an accumulator's epilogue, two to a quarter of the lanes.
// The other accumulator's eight run beside them: with K = 64, where nothing but
// the epilogue takes time, that gave 435 us where the same eight for both took
// 540 and sixteen for each in turn 493.
// The tiles that do not fill a whole wave run as two items of 128 rows each
// when that still fits in one wave.
constexpr int kShort = 192;   // at most 256: an epilogue warp holds the scales of half the rows
struct Work {
    int full, items;
};
__device__ __forceinline__ Work work_of(int units, int nclusters) {
    Work w;
    w.full = units / nclusters * nclusters;
    const int tail = units - w.full;
    w.items = units;
    if (tail > 0 && 2 * tail <= nclusters) w.items = w.full + 2 * tail; else w.full = units;
    return w;
}
struct Item {
    Tile t;
    size_t row0;   // first row of A
    int n;         // rows of A (0: nothing to do)
    bool shrt;     // a short tile: the weights are the M operand
};
template <typename C>
__device__ __forceinline__ Item item_at(const C* c, const KP& p, const Work& w, int v) {
    Item i;
    const int half = v < w.full ? -1 : (v - w.full) & 1;
    i.t = tile_of(c, p, v < w.full ? v : w.full + ((v - w.full) >> 1), 256);
    const int lo = i.t.m_blk * 256 + (half > 0 ? 128 : 0);
    i.n = max(min(i.t.rows - lo, half < 0 ? 256 : 128), 0);
    i.shrt = i.n <= kShort;
    i.row0 = static_cast<size_t>(i.t.row0) + static_cast<size_t>(lo);
    return i;
}
// The two warps of an epilogue pair (64 threads): the logical and of `ok`.
__device__ __forceinline__ bool pair_and(int id, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r) : "r"(ok ? 1u : 0u), "r"(id) : "memory");
    return r != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Epilogues of one set by one warp (half h of its columns).
// Whole tile: a thread is row r, columns are channels from ch0.
// sc: the scales of the warp's columns in shared memory (SWIGLU 64 of B0,
// then 64 of B1). The results go through a 1 KB stage of the warp and leave as
// bulk tensor stores of 32 rows x 32 bytes, which nothing waits for but the
// next use of the stage; the last rows of a group by plain 16-byte stores of
// the same runs. With each lane storing its own row's 16 bytes the stores
// alone cost 36 of 435 us (4096 rows, K = 4096, 18944 channels); staged plain
// stores took 309 us where bulk stores take 304 (8192 rows, K = 14336) and 608
// where they take 540 (33474 rows, K = 64, 11328 channels).
template <bool SWIGLU, typename OutT>
__device__ __forceinline__ void whole_tile(const KP& p, const Item& it, uint32_t tb, int h, int r0, int ch0, float sa,
                                           const float* sc, uint8_t* stage, const CUtensorMap* om, OutT* out) {
    const int lane = threadIdx.x & 31;
    constexpr int HALF = SWIGLU ? 64 : 128;
    constexpr int RUN = 32 / sizeof(OutT);   // channels of a run
    constexpr int PER = 16 / sizeof(OutT);   // channels of a piece
    const uint64_t sa2 = pk(sa, sa);
    const bool whole = r0 + 32 <= it.n;   // all 32 rows are the tile's: one bulk store a run
#pragma unroll 1
    for (int c = 0; c < HALF; c += 16) {
        uint32_t a[16], b[SWIGLU ? 16 : 1];
        __syncwarp();   // the loads are the warp's: all lanes come to them together
        if constexpr (SWIGLU) tmem_ld16x2(tb + HALF * h + c, tb + 128 + HALF * h + c, a, b);
        else tmem_ld16(tb + HALF * h + c, a);
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const ulonglong2 s0 = *reinterpret_cast<const ulonglong2*>(sc + c + i);
            uint64_t y0 = scaled2(a[i], a[i + 1], sa2, s0.x), y1 = scaled2(a[i + 2], a[i + 3], sa2, s0.y);
            if constexpr (SWIGLU) {
                const ulonglong2 s1 = *reinterpret_cast<const ulonglong2*>(sc + 64 + c + i);
                y0 = swiglu2(y0, scaled2(b[i], b[i + 1], sa2, s1.x), out);
                y1 = swiglu2(y1, scaled2(b[i + 2], b[i + 3], sa2, s1.y), out);
            }
            const float2 f0 = unpk(y0), f1 = unpk(y1);
            v[i] = f0.x; v[i + 1] = f0.y; v[i + 2] = f1.x; v[i + 3] = f1.y;
        }
#pragma unroll
        for (int e = 0; e < 16; e += RUN) {
            if (lane == 0) bulk_wait_read<0>();   // the run before has left the stage
            __syncwarp();
            stage_run(stage, lane, v + e, out);
            const int ch = ch0 + HALF * h + c + e;   // N is a multiple of 16: runs are in or out
            if (whole) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && ch < p.N) tma_store_2d(om, smem_u32(stage), ch, static_cast<int>(it.row0) + r0);
                if (lane == 0) bulk_commit();
            } else {
                __syncwarp();
                if (ch < p.N) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = i * 16 + (lane >> 1);
                        if (r0 + row < it.n)
                            *reinterpret_cast<uint4*>(out + (it.row0 + r0 + row) * p.N + ch + (lane & 1) * PER) =
                                *stage_at(stage, row, lane & 1);
                    }
                }
                __syncwarp();
            }
        }
    }
}
// Short tile: a thread is channel ch with scale f, columns are rows of A; sc:
// the scales of the warp's rows, 32 of every 64, in shared memory.
template <typename OutT>
__device__ __forceinline__ void short_plain(const KP& p, const Item& it, uint32_t tb, int h, int ch, float f, const float* sc,
                                            OutT* out) {
    const uint64_t f2 = pk(f, f);
#pragma unroll 1
    for (int i = 0; i < kShort / 2; i += 16) {
        const int c = 32 * h + (i & 16) + (i & ~31) * 2;
        if (c >= it.n) continue;
        uint32_t v[16];
        __syncwarp();
        tmem_ld16(tb + c, v);
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sc + i + j);
            const float2 u0 = unpk(scaled2(v[j], v[j + 1], s.x, f2)), u1 = unpk(scaled2(v[j + 2], v[j + 3], s.y, f2));
            y[j] = u0.x; y[j + 1] = u0.y; y[j + 2] = u1.x; y[j + 3] = u1.y;
        }
        if (ch < p.N) put_rows<16>(out + (it.row0 + c) * p.N + ch, p.N, it.n - c, y);
    }
}
template <typename OutT>
__device__ __forceinline__ void short_swiglu(const KP& p, const Item& it, uint32_t tb, int h, bool gate, int pid, float* mine,
                                             const float* other, int ch, float f, const float* sc, OutT* out) {
    const int lane = threadIdx.x & 31;
    const uint64_t f2 = pk(f, f);
#pragma unroll 1
    for (int i = 0; i < kShort / 2; i += 16) {
        const int c = 32 * h + (i & 16) + (i & ~31) * 2;
        if (c >= it.n) continue;
        uint32_t v[16];
        __syncwarp();
        tmem_ld16(tb + c, v);
        float keep[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {   // rows 0..7 are the gate warp's to finish, 8..15 the up warp's
            const float2 lo = unpk(scaled2(v[j], v[j + 1], *reinterpret_cast<const uint64_t*>(sc + i + j), f2));
            const float2 hi = unpk(scaled2(v[8 + j], v[9 + j], *reinterpret_cast<const uint64_t*>(sc + i + 8 + j), f2));
            keep[j] = gate ? lo.x : hi.x;
            keep[j + 1] = gate ? lo.y : hi.y;
            mine[j * 32 + lane] = gate ? hi.x : lo.x;
            mine[(j + 1) * 32 + lane] = gate ? hi.y : lo.y;
        }
        pair_sync(pid);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = other[j * 32 + lane];
        pair_sync(pid);   // both have read: the buffers are free
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t k2 = pk(keep[j], keep[j + 1]), o2 = pk(y[j], y[j + 1]);
            const float2 u = unpk(gate ? swiglu2(k2, o2, out) : swiglu2(o2, k2, out));
            y[j] = u.x;
            y[j + 1] = u.y;
        }
        const int c0 = c + (gate ? 0 : 8);
        if (ch < p.N) put_rows<8>(out + (it.row0 + c0) * p.N + ch, p.N, it.n - c0, y);
    }
}

template <bool SWIGLU, typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
i8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
               const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmA32,
               const __grid_constant__ CUtensorMap tmO, const KP p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* xch = reinterpret_cast<float*>(smem + P_STAGES * P_STAGE_BYTES);
    using C = Ctl<P_STAGES>;
    C* ctl = reinterpret_cast<C*>(xch + EPI * (P_STAGE_FLOATS + P_SCALE_FLOATS));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const uint32_t peer_abort = mapa_shared(smem_u32(&ctl->abort_flag), rank ^ 1u);
    const int cluster = static_cast<int>(blockIdx.x >> 1), nclusters = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&ctl->tfull[a], 1);
            mbar_init(&ctl->tempty[a], EPI);   // of both CTAs, half the epilogue warps each
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&tmA); prefetch_map(&tmB0); prefetch_map(&tmB1);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&ctl->tmem_base)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    if (warp == 2) list_tiles(ctl, p, 256);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Work work = work_of(ctl->cum[p.E], nclusters);
    const int num_kb = (p.K + BKB - 1) / BKB;
    constexpr int SET = SWIGLU ? 128 : 256;   // channels of one of a tile's two sets
    auto sets_of = [&](const Item& it) { return it.t.n_blk * 2 * SET + SET < p.N ? 2 : 1; };

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, loaded = 0;
            bool aborted = false;
            auto full_of = [&](int st) { return mapa_shared(smem_u32(&ctl->full[st]), 0u); };
            for (int u = cluster; u < work.items && !aborted; u += nclusters) {
                const Item it = item_at(ctl, p, work, u);
                if (it.n == 0) continue;
                const int sets = sets_of(it);
                // this rank's rows of A: 128 in one box, or of a short tile half of its N columns in boxes of 32
                const int half_n = (it.n + 31) / 32 * 16;
                const int arow = static_cast<int>(it.row0) + rank * (it.shrt ? half_n : BM);
                const int boxes = it.shrt ? (half_n + 31) / 32 : 0;
                // its two 64-row boxes of weights of each set
                const int b0 = it.t.g * p.N + it.t.n_blk * 2 * SET + (SWIGLU ? (it.shrt ? rank * 64 : 0) : rank * 128);
                const int b1 = SWIGLU && it.shrt ? b0 : b0 + 64;
                const CUtensorMap* m0 = SWIGLU && !it.shrt && rank ? &tmB1 : &tmB0;
                const CUtensorMap* m1 = SWIGLU && it.shrt ? &tmB1 : m0;
                const uint32_t bytes = (it.shrt ? boxes * 32 * BKB : A_BYTES) + sets * BH_BYTES;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!wait_i8(&ctl->empty[s], ph ^ 1u, ctl, p, peer_abort)) { aborted = true; break; }
                    const uint32_t sa = smem_u32(smem + s * P_STAGE_BYTES);
                    if (leader) mbar_arrive_expect_tx(&ctl->full[s], 2 * bytes);
                    ctl->bytes[s] = bytes;
                    if (it.shrt) {
                        for (int q = 0; q < boxes; ++q)
                            tma_load_2d_pair(sa + q * 32 * BKB, &tmA32, full_of(s), kb * BKB, arow + 32 * q);
                    } else {
                        tma_load_2d_pair(sa, &tmA, full_of(s), kb * BKB, arow);
                    }
                    for (int z = 0; z < sets; ++z) {
                        const uint32_t sw = sa + A_BYTES + z * BH_BYTES;
                        tma_load_2d_pair(sw, m0, full_of(s), kb * BKB, b0 + z * SET);
                        tma_load_2d_pair(sw + BH_BYTES / 2, m1, full_of(s), kb * BKB, b1 + z * SET);
                    }
                    ++loaded;
                    if (++s == P_STAGES) { s = 0; ph ^= 1u; }
                }
            }
            ctl->loaded = loaded;
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            int s = 0;
            uint32_t ph = 0, aph[2] = {0u, 0u}, first_acc = 0;   // the accumulators take the sets in turn
            bool aborted = false;
            for (int u = cluster; u < work.items && !aborted; u += nclusters) {
                const Item it = item_at(ctl, p, work, u);
                if (it.n == 0) continue;
                const int sets = sets_of(it);
                const uint32_t id = idesc_i8(256, it.shrt ? (it.n + 31) / 32 * 32 : 256);
                // the K blocks [kb, kb + cnt) of set z; the last set of an item releases the stages
                auto run = [&](int kb, int cnt, int z, int st, uint32_t p0) {
                    for (int i = 0; i < cnt; ++i) {
                        if (z == 0 && !wait_i8(&ctl->full[st], p0, ctl, p, peer_abort)) return false;
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + st * P_STAGE_BYTES);
                        const uint64_t xd = sw128_desc(sa), wd = sw128_desc(sa + A_BYTES + z * BH_BYTES);
                        const uint64_t md = it.shrt ? wd : xd, nd = it.shrt ? xd : wd;
                        const uint32_t d = tmem_base + ((first_acc + z) & 1u) * ACC_COLS;
#pragma unroll
                        for (int kk = 0; kk < BKB / 32; ++kk)
                            mma_i8_pair(d, md + 2u * kk, nd + 2u * kk, id, (kb + i) | kk ? 1u : 0u);
                        if (z == sets - 1) tc_commit_pair_mc(&ctl->empty[st], 0x3);
                        if (++st == P_STAGES) { st = 0; p0 ^= 1u; }
                    }
                    return true;
                };
                auto full_acc = [&](int z) { tc_commit_pair_mc(&ctl->tfull[(first_acc + z) & 1u], 0x3); };
                auto step = [&](int cnt) {
                    s += cnt;
                    if (s >= P_STAGES) { s -= P_STAGES; ph ^= 1u; }
                };
                auto free_acc = [&](int z) {
                    const uint32_t acc = (first_acc + z) & 1u;
                    const bool ok = wait_i8(&ctl->tempty[acc], aph[acc] ^ 1u, ctl, p, peer_abort);
                    aph[acc] ^= 1u;
                    tc_fence_after();
                    return ok;
                };
                // With two sets the first and last P_STAGES K blocks go set by set: set 0
                // starts while the epilogue still reads set 1 of the tile before, and is
                // complete while set 1 still runs.
                const int first = min(P_STAGES, num_kb), last = sets == 2 ? min(P_STAGES, num_kb - first) : 0;
                bool ok = free_acc(0) && run(0, first, 0, s, ph);
                if (ok && first == num_kb) full_acc(0);
                if (ok && sets == 2) ok = free_acc(1) && run(0, first, 1, s, ph);
                if (ok) step(first);
                for (int kb = first; ok && kb < num_kb - last; ++kb) {
                    ok = run(kb, 1, 0, s, ph);
                    if (ok && sets == 2) ok = run(kb, 1, 1, s, ph);
                    if (ok) step(1);
                }
                if (ok && first < num_kb) {
                    ok = run(num_kb - last, last, 0, s, ph);
                    if (ok) full_acc(0);
                    if (ok && sets == 2) ok = run(num_kb - last, last, 1, s, ph);
                    if (ok) step(last);
                }
                if (ok && sets == 2) full_acc(1);
                first_acc += sets;
                aborted = !ok;
            }
        }
    } else {
        const int q = warp & 3;
        const bool gate = q < 2;                      // short SWIGLU tiles: this warp's accumulators
        const int h = ((warp - 2) >> 2) & 1;          // which half of a set's columns
        const int acc = (warp - 2) >> 3;              // which accumulator
        const int pid = 1 + (q & 1) + 2 * h + 4 * acc;   // barrier of the warp pair
        // whole tiles stage in the 1 KB in which the warp sends its half of a short one (read by the partner before
        // the barrier that ends every trade)
        float* trade = xch + 2 * (pid - 1) * P_STAGE_FLOATS;
        float* mine_st = trade + (gate ? 0 : P_STAGE_FLOATS);
        const float* other_st = trade + (gate ? P_STAGE_FLOATS : 0);
        uint8_t* stage = reinterpret_cast<uint8_t*>(mine_st);
        float* scales = xch + EPI * P_STAGE_FLOATS + (warp - 2) * P_SCALE_FLOATS;
        const uint32_t tempty0 = mapa_shared(smem_u32(&ctl->tempty[acc]), 0u);
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * ACC_COLS);
        OutT* out = static_cast<OutT*>(p.out);
        uint32_t aph = 0;
        // This accumulator's set to come, with its scales already on the way: they are fetched
        // while the set before is finished. 32 items are decoded at once, one a lane.
        struct Next {
            Item it;
            int z, sets;
            float sa, sc[4] = {};
        } nx;
        Item mine;
        int cnt = 0, seen = 0;   // items and sets so far
        nx.z = nx.sets = 0;
        auto fetch = [&]() {   // false past the last
            do {
                if (++nx.z >= nx.sets) {
                    do {
                        if ((cnt & 31) == 0) {
                            const long long u = cluster + static_cast<long long>(cnt + lane) * nclusters;
                            mine.n = -1;
                            if (u < work.items) mine = item_at(ctl, p, work, static_cast<int>(u));
                        }
                        const int from = cnt++ & 31;
                        nx.it.n = __shfl_sync(0xffffffffu, mine.n, from);
                        if (nx.it.n < 0) return false;
                        nx.it.t.g = __shfl_sync(0xffffffffu, mine.t.g, from);
                        nx.it.t.n_blk = __shfl_sync(0xffffffffu, mine.t.n_blk, from);
                        nx.it.row0 = __shfl_sync(0xffffffffu, static_cast<int>(mine.row0), from);
                    } while (nx.it.n == 0);
                    nx.it.shrt = nx.it.n <= kShort;
                    nx.z = 0;
                    nx.sets = sets_of(nx.it);
                }
            } while ((seen++ & 1) != acc);
            const int ch0 = nx.it.t.n_blk * 2 * SET + nx.z * SET;
            const size_t gsb = static_cast<size_t>(nx.it.t.g) * p.N;
            const float* sap = p.sa + nx.it.row0;
            if (nx.it.shrt) {   // sa: the thread's channel; sc: rows 32 h .. 32 h + 31 of every 64
                const int ch = ch0 + lane + (SWIGLU ? rank * 64 + (q & 1) * 32 : rank * 128 + q * 32);
                nx.sa = ch < p.N ? (SWIGLU && !gate ? p.sb1 : p.sb0)[gsb + ch] : 0.f;
#pragma unroll
                for (int v = 0; v < 3; ++v) {
                    const int r = 64 * v + 32 * h + lane;
                    nx.sc[v] = r < nx.it.n ? sap[r] : 0.f;
                }
            } else {            // sa: the thread's row; sc: the warp's channels
                const int r = rank * BM + q * 32 + lane;
                nx.sa = r < nx.it.n ? sap[r] : 0.f;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int ch = ch0 + (SWIGLU ? 64 * h + 32 * (v & 1) : 128 * h + 32 * v) + lane;
                    nx.sc[v] = ch < p.N ? (SWIGLU && v >= 2 ? p.sb1 : p.sb0)[gsb + ch] : 0.f;
                }
            }
            return true;
        };
        bool met = false;
        for (bool more = fetch(); more;) {
            const Item it = nx.it;
            const int r0 = rank * BM + q * 32, ch0 = it.t.n_blk * 2 * SET + nx.z * SET;
            const float sa = nx.sa;
#pragma unroll
            for (int v = 0; v < 4; ++v) scales[32 * v + lane] = nx.sc[v];
            __syncwarp();
            more = fetch();
            const bool ok = __all_sync(0xffffffffu, wait_i8(&ctl->tfull[acc], aph, ctl, p, peer_abort));   // one answer a warp
            aph ^= 1u;
            // The warps of a pair leave together, so that neither waits for the other: on the word of both at a
            // short tile, else after the loop, where one that has left early answers the other's last question.
            if (SWIGLU && it.shrt) {
                met = !pair_and(pid, ok);
                if (met) break;
            } else if (!ok) {
                break;
            }
            tc_fence_after();
            if (SWIGLU && it.shrt) {   // the stage is the trade's buffer too
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
            }
            if (!it.shrt) whole_tile<SWIGLU, OutT>(p, it, tb, h, r0, ch0, sa, scales, stage, &tmO, out);
            else if (SWIGLU) short_swiglu<OutT>(p, it, tb, h, gate, pid, mine_st, other_st, ch0 + rank * 64 + (q & 1) * 32 + lane, sa, scales, out);
            else short_plain<OutT>(p, it, tb, h, ch0 + rank * 128 + q * 32 + lane, sa, scales, out);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(&ctl->tempty[acc]);
                else mbar_arrive_remote(tempty0);
            }
        }
        __syncwarp();
        if (SWIGLU && !met) pair_and(pid, false);
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    // A wait gave up (both CTAs carry the flag): the leader's barriers count both CTAs' copies, so it
    // waits for all of them. Where one CTA has requested more blocks than the other, the bytes that will
    // not come are taken off the leader's phase, or the phase is armed for the other CTA's alone.
    if (__builtin_expect(*reinterpret_cast<volatile int*>(&ctl->abort_flag), 0)) {
        if (cluster_ctarank() == 0 && threadIdx.x == 0) {
            auto other = [](const uint32_t* v) { return ld_shared_remote_u32(mapa_shared(smem_u32(v), 1u)); };
            const uint32_t n0 = ctl->loaded, n1 = other(&ctl->loaded);
            const uint32_t hi = max(n0, n1);
#pragma unroll 1
            for (uint32_t j = min(n0, n1); j < hi; ++j) {
                if (n0 > n1) mbar_complete_tx(&ctl->full[j % P_STAGES], ctl->bytes[j % P_STAGES]);
                else mbar_arrive_expect_tx(&ctl->full[j % P_STAGES], other(&ctl->bytes[j % P_STAGES]));
            }
            drain_loads(ctl, hi, p);
        } else if (cluster_ctarank() == 0 && threadIdx.x == 32) {
            tc_commit_pair(&ctl->drain);
            drain_i8(&ctl->drain, 0, p);
        }
        __syncwarp();
        tc_fence_before();
        cluster_sync_all();
        tc_fence_after();
    }
    if (threadIdx.x >> 5 == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(ctl->tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

// ---- single form ----------------------------------------------------------------
// The weights are the M operand: a tile is 256 weight rows (two MMAs of M =
// 128: SWIGLU 128 channels of B0 and the same of B1, PLAIN 256 channels of
// B0) against up to 128 rows of A as N = 16, 32, .. 128, so a group of few
// rows costs few tensor cycles and few bytes beside its weights, and a
// thread of the epilogue owns a channel: its two scales are loaded once and
// every store of a warp is 32 consecutive channels of one row. H warps share a
// quarter of the channels of an accumulator, 16 rows of every 16 H each.
//
// Units: the tiles that fill whole waves of the grid run one to a CTA, in
// order, over all of K. The tail tiles are cut along K into equal shares for
// all CTAs and run first, so that joining their parts hides under the whole
// tiles: each part is added to the tile's accumulators in the workspace
// (integer additions in L2, whose order does not matter), and the warp that
// arrives last applies the scales and stores.
struct Unit {
    int tile, kb0, kb1;
    int parts;        // contributors of the tile
    int tail;         // index of the tile among the tail tiles
};
struct Units {
    int whole, tail, nkb, grid, n;   // whole tiles of a CTA; tail tiles; K blocks a tile; CTAs; CTAs sharing the tail
    __device__ __forceinline__ int lo(int b) const {
        return static_cast<int>(static_cast<long long>(tail) * nkb * b / n);
    }
    __device__ __forceinline__ int owner(int r) const {   // the b with lo(b) <= r < lo(b + 1)
        return static_cast<int>((static_cast<long long>(r + 1) * n - 1) / (static_cast<long long>(tail) * nkb));
    }
};
// Whether the tail is cut: shares of kMinShare K blocks or more, one to a CTA,
// if that shortens the tail by more K blocks than joining costs. Joining is
// two passes over each part's sums in L2 and the zeros before: about as long
// as 4 K blocks and one for every 10 rows of the tallest tile. Measured cut /
// not cut: 46 rows of K = 11264 (down, 8 experts, N = 4096) 85 / 85 us and with 2
// experts of one row 34 / 50; 128 rows, K = 1408, 96 tiles 27 / 16; 128 rows, K =
// 8400, 20 tiles 48 / 62; 36 rows, K = 1792, 76 tiles in the tail 34 / 22.
// A tail of more than three quarters of the CTAs is not cut: so many draw the
// weights as fast as all (128 tiles, K = 14336: 6 rows 82 / 80 us, 32 rows 89 / 82,
// 64 rows 95 / 83).
constexpr int kMinShare = 4;
__device__ __forceinline__ Units units_of(int tiles, int most, int nkb, int grid) {
    Units u;
    u.grid = grid;
    u.nkb = nkb;
    u.whole = tiles / grid;
    u.tail = tiles - u.whole * grid;
    const long long blocks = static_cast<long long>(u.tail) * nkb;
    const int shares = static_cast<int>(min((blocks + kMinShare - 1) / kMinShare, static_cast<long long>(grid)));
    u.n = max(shares, max(u.tail, 1));
    const int share = static_cast<int>((blocks + u.n - 1) / u.n);
    if (nkb - share <= 4 + most / 10 || 4 * u.tail > 3 * grid) u.n = max(u.tail, 1);
    return u;
}
// Unit i of CTA b; false past the last.
__device__ __forceinline__ bool unit_at(const Units& u, int b, int i, Unit& o) {
    if (u.tail > 0 && b < u.n) {
        const int r0 = u.lo(b), r1 = u.lo(b + 1), t0 = r0 / u.nkb;
        const int cnt = r1 > r0 ? (r1 - 1) / u.nkb - t0 + 1 : 0;
        if (i < cnt) {
            const int t = t0 + i;
            o.tail = t;
            o.tile = u.whole * u.grid + t;
            o.kb0 = max(r0 - t * u.nkb, 0);
            o.kb1 = min(r1 - t * u.nkb, u.nkb);
            o.parts = u.owner((t + 1) * u.nkb - 1) - u.owner(t * u.nkb) + 1;
            return true;
        }
        i -= cnt;
    }
    if (i >= u.whole) return false;
    o.tile = b + i * u.grid; o.kb0 = 0; o.kb1 = u.nkb; o.parts = 1; o.tail = 0;
    return true;
}

__device__ __forceinline__ void red_add(int* p, uint32_t v) {
    asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <bool SWIGLU, typename OutT, int H>
__global__ void __launch_bounds__(64 + 256 * H, 1)
i8_single_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmB0h,
                 const __grid_constant__ CUtensorMap tmB1h, const KP p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using C = Ctl<S_STAGES>;
    float* rows_sa = reinterpret_cast<float*>(smem + S_STAGES * S_STAGE_BYTES);
    C* ctl = reinterpret_cast<C*>(rows_sa + 8 * H * S_ROW_FLOATS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = static_cast<int>(blockIdx.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S_STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&ctl->tfull[a], 1);
            mbar_init(&ctl->tempty[a], 4 * H);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&tmA); prefetch_map(&tmB0); prefetch_map(&tmB1);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&ctl->tmem_base)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    if (warp == 2) list_tiles(ctl, p, BM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Units un = units_of(ctl->cum[p.E], ctl->most, (p.K + BKB - 1) / BKB, static_cast<int>(gridDim.x));

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, loaded = 0;
            bool aborted = false;
            Unit w;
            for (int i = 0; !aborted && unit_at(un, b, i, w); ++i) {
                const Tile t = tile_of(ctl, p, w.tile, BM);
                const int arow = t.row0 + t.m_blk * BM;
                const int boxes = (min(t.rows - t.m_blk * BM, BM) + 31) / 32;
                // each half's weight rows in one box of 128, or of 64 where the expert has no more left: a 128-row
                // box costs what it holds, two of 64 in its place 4 % (256 experts of 64 rows, 1158 -> 1203 us)
                const int n0 = SWIGLU ? t.n_blk * 128 : t.n_blk * 256, n1 = SWIGLU ? n0 : n0 + 128;
                const int brow = t.g * p.N + n0, brow1 = t.g * p.N + n1;
                const CUtensorMap* m0 = p.N - n0 > 64 ? &tmB0 : &tmB0h;
                const CUtensorMap* m1 = p.N - n1 > 64 ? (SWIGLU ? &tmB1 : &tmB0) : (SWIGLU ? &tmB1h : &tmB0h);
                const bool two = n1 < p.N;
                const uint32_t bytes = boxes * 32 * BKB + (p.N - n0 > 64 ? BH_BYTES : BH_BYTES / 2) +
                                       (p.N - n1 > 64 ? BH_BYTES : two ? BH_BYTES / 2 : 0);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_i8(&ctl->empty[s], ph ^ 1u, ctl, p)) { aborted = true; break; }
                    const uint32_t sa = smem_u32(smem + s * S_STAGE_BYTES);
                    mbar_arrive_expect_tx(&ctl->full[s], bytes);
                    tma_load_2d(sa + A_BYTES, m0, &ctl->full[s], kb * BKB, brow);
                    if (two) tma_load_2d(sa + A_BYTES + BH_BYTES, m1, &ctl->full[s], kb * BKB, brow1);
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(sa + q * 32 * BKB, &tmA, &ctl->full[s], kb * BKB, arow + 32 * q);
                    ++loaded;
                    if (++s == S_STAGES) { s = 0; ph ^= 1u; }
                }
            }
            ctl->loaded = loaded;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool aborted = false;
            Unit w;
            for (int i = 0; !aborted && unit_at(un, b, i, w); ++i) {
                const Tile t = tile_of(ctl, p, w.tile, BM);
                const bool two = SWIGLU || t.n_blk * 256 + 128 < p.N;   // the tile has channels in its second half
                const uint32_t id = idesc_i8(BM, (min(t.rows - t.m_blk * BM, BM) + 15) / 16 * 16);
                if (!wait_i8(&ctl->tempty[acc], aph ^ 1u, ctl, p)) { aborted = true; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * ACC_COLS);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_i8(&ctl->full[s], ph, ctl, p)) { aborted = true; break; }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + s * S_STAGE_BYTES);
                    const uint64_t xd = sw128_desc(sa), w0 = sw128_desc(sa + A_BYTES), w1 = sw128_desc(sa + A_BYTES + BH_BYTES);
#pragma unroll
                    for (int kk = 0; kk < BKB / 32; ++kk) {
                        const uint32_t accum = kb != w.kb0 || kk != 0 ? 1u : 0u;
                        mma_i8(d, w0 + 2u * kk, xd + 2u * kk, id, accum);
                        if (two) mma_i8(d + 128u, w1 + 2u * kk, xd + 2u * kk, id, accum);
                    }
                    tc_commit(&ctl->empty[s]);
                    if (++s == S_STAGES) { s = 0; ph ^= 1u; }
                }
                if (aborted) break;
                tc_commit(&ctl->tfull[acc]);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
        }
    } else {
        const int q = warp & 3, r = q * 32 + lane;   // this thread's channel of each half
        const int h = ((warp - 2) >> 2) % H;         // rows 16 h .. 16 h + 15 of every 16 H are this warp's
        const int acc = (warp - 2) / (4 * H);        // units acc, acc + 2, .. are its accumulator's
        float* my_sa = rows_sa + (warp - 2) * S_ROW_FLOATS;
        uint32_t aph = 0;
        OutT* out = static_cast<OutT*>(p.out);
        // What the epilogue needs of a unit, with its scales already on the
        // way: fetched while the unit before it is finished.
        struct Next {
            Unit w;
            Tile t;
            bool some;
            float f0, f1, s0, s1;
        } nx;
        auto fetch = [&](int i) {
            nx.some = unit_at(un, b, i, nx.w);
            if (!nx.some) return;
            nx.t = tile_of(ctl, p, nx.w.tile, BM);
            const int n0 = (SWIGLU ? nx.t.n_blk * 128 : nx.t.n_blk * 256) + r, n1 = SWIGLU ? n0 : n0 + 128;
            const size_t sc = static_cast<size_t>(nx.t.g) * p.N;
            nx.f0 = n0 < p.N ? p.sb0[sc + n0] : 0.f;
            nx.f1 = n1 < p.N ? (SWIGLU ? p.sb1 : p.sb0)[sc + n1] : 0.f;
            // lane l: the l-th and the (l + 32)-th of the warp's rows
            const int n = nx.t.rows - nx.t.m_blk * BM, c = (lane & 16) * H + 16 * h + (lane & 15);
            const float* sap = p.sa + nx.t.row0 + static_cast<size_t>(nx.t.m_blk) * BM;
            nx.s0 = c < min(n, BM) ? sap[c] : 0.f;
            nx.s1 = c + 32 * H < min(n, BM) ? sap[c + 32 * H] : 0.f;
        };
        fetch(acc);
        for (int i = acc; nx.some;) {
            const Unit w = nx.w;
            const Tile t = nx.t;
            int nrow = min(t.rows - t.m_blk * BM, BM);
            const size_t row0 = static_cast<size_t>(t.row0) + static_cast<size_t>(t.m_blk) * BM;
            const int ch0 = (SWIGLU ? t.n_blk * 128 : t.n_blk * 256) + r, ch1 = SWIGLU ? ch0 : ch0 + 128;
            const bool two = SWIGLU || t.n_blk * 256 + 128 < p.N;
            const uint64_t f0 = pk(nx.f0, nx.f0), f1 = pk(nx.f1, nx.f1);
            my_sa[lane] = nx.s0;
            my_sa[32 + lane] = nx.s1;
            __syncwarp();
            i += 2;
            fetch(i);
            if (!__all_sync(0xffffffffu, wait_i8(&ctl->tfull[acc], aph, ctl, p))) break;   // one answer a warp
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * ACC_COLS);
            int* sums = p.part + static_cast<size_t>(w.tail) * 256 * p.part_rows + r;   // [row][256 channels]
            if (w.parts > 1) {
#pragma unroll 1
                for (int c = 16 * h; c < nrow; c += 16 * H) {
                    uint32_t lo[16], hi[16];
                    __syncwarp();
                    tmem_ld16x2(tb + c, tb + 128 + c, lo, hi);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < nrow) {
                            red_add(sums + (c + j) * 256, lo[j]);
                            if (two) red_add(sums + (c + j) * 256 + 128, hi[j]);
                        }
                }
                __threadfence();
                __syncwarp();
                int old = 0;
                if (lane == 0) old = atomicAdd(p.sem + w.tail * 8 + 4 * h + q, 1);
                old = __shfl_sync(0xffffffffu, old, 0);
                __threadfence();
                if (old != w.parts - 1) nrow = 0;   // another part comes later: its warp finishes
            }
#pragma unroll 1
            for (int c = 16 * h; c < nrow; c += 16 * H) {
                uint32_t lo[16], hi[16];
                __syncwarp();
                if (w.parts == 1) {
                    tmem_ld16x2(tb + c, tb + 128 + c, lo, hi);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        lo[j] = c + j < nrow ? static_cast<uint32_t>(__ldcg(sums + (c + j) * 256)) : 0u;
                        hi[j] = two && c + j < nrow ? static_cast<uint32_t>(__ldcg(sums + (c + j) * 256 + 128)) : 0u;
                    }
                }
                const float* sap = my_sa + c / (16 * H) * 16;
                float y[SWIGLU ? 16 : 32];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(sap + j);
                    uint64_t a0 = scaled2(lo[j], lo[j + 1], s.x, f0), a1 = scaled2(lo[j + 2], lo[j + 3], s.y, f0);
                    const uint64_t b0 = scaled2(hi[j], hi[j + 1], s.x, f1), b1 = scaled2(hi[j + 2], hi[j + 3], s.y, f1);
                    if constexpr (SWIGLU) {
                        a0 = swiglu2(a0, b0, out);
                        a1 = swiglu2(a1, b1, out);
                    } else {
                        const float2 v0 = unpk(b0), v1 = unpk(b1);
                        y[16 + j] = v0.x; y[17 + j] = v0.y; y[18 + j] = v1.x; y[19 + j] = v1.y;
                    }
                    const float2 u0 = unpk(a0), u1 = unpk(a1);
                    y[j] = u0.x; y[j + 1] = u0.y; y[j + 2] = u1.x; y[j + 3] = u1.y;
                }
                OutT* o = out + (row0 + c) * p.N;
                const int n = nrow - c;
                if (ch0 < p.N) put_rows<16>(o + ch0, p.N, n, y);
                if constexpr (!SWIGLU)
                    if (ch1 < p.N) put_rows<16>(o + ch1, p.N, n, y + 16);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[acc]);
            aph ^= 1u;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(*reinterpret_cast<volatile int*>(&ctl->abort_flag), 0)) {   // a wait gave up
        if (threadIdx.x == 0) {
            drain_loads(ctl, ctl->loaded, p);
        } else if (threadIdx.x == 32) {
            tc_commit(&ctl->drain);
            drain_i8(&ctl->drain, 0, p);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (threadIdx.x >> 5 == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(ctl->tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

// First launch of a product: the status word is MOE_OK, and the arrival
// counters and sums of the tail tiles are zero, before the product passes its
// wait. The product's launch and prologue run beside it and the kernel
// before. It waits itself before it writes: a product still running on the
// same workspace has completed by then.
__global__ void __launch_bounds__(256) i8_begin_kernel(const KP p, int grid) {
    __shared__ Ctl<1> c;
    pdl_launch();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    if (p.part == nullptr) return;
    if (threadIdx.x < 32) list_tiles(&c, p, BM);
    __syncthreads();
    const Units u = units_of(c.cum[p.E], c.most, (p.K + BKB - 1) / BKB, grid);
    if (u.n <= u.tail) return;   // no tile has more than one part
    for (int t = blockIdx.x; t < u.tail; t += gridDim.x) {
        const Tile tile = tile_of(&c, p, u.whole * u.grid + t, BM);
        const int n = min(tile.rows - tile.m_blk * BM, BM) * 64;
        int4* part = reinterpret_cast<int4*>(p.part + static_cast<size_t>(t) * 256 * p.part_rows);
        for (int i = threadIdx.x; i < n; i += 256) part[i] = make_int4(0, 0, 0, 0);
        if (threadIdx.x < 8) p.sem[t * 8 + threadIdx.x] = 0;
    }
}

// ---- host side --------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// [rows, cols] bytes, boxes of 128 columns x box_rows rows, 128-byte swizzle, zeros outside
bool map_i8(CUtensorMap* m, const void* base, long long rows, int cols, int box_rows) {
    const auto enc = encoder();
    if (enc == nullptr) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows > 0 ? rows : 1)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    cuuint32_t box[2] = {BKB, static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A, B0, B1 and two more: pair A in boxes of 32 rows and the results; single B0 and B1 in boxes of 64
struct Maps {
    CUtensorMap a, b0, b1, x0, x1;
};// results [rows, N], boxes of 32 rows x 32 bytes in stage_at's order (32-byte swizzle)
bool map_out(CUtensorMap* m, void* base, long long rows, int N, int dtype) {
    const auto enc = encoder();
    if (enc == nullptr) return false;
    const bool bf = dtype == MOE_DTYPE_BF16;
    const cuuint64_t es = bf ? 2 : 4;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(rows > 0 ? rows : 1)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * es};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(32 / es), 32}, estr[2] = {1, 1};
    return enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <auto KERNEL>
cudaError_t launch_tc(size_t smem, int grid, int threads, const Maps& m, const KP& kp, cudaStream_t st) {
    static bool attr_set[64] = {};   // per kernel (template) and device; the size never changes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    return launch_dep(KERNEL, dim3(grid), dim3(threads), smem, st, m.a, m.b0, m.b1, m.x0, m.x1, kp);
}

template <bool SWIGLU, typename OutT>
cudaError_t launch_form(const I8Gemm& g, const KP& kp, const Maps& m, cudaStream_t st) {
    if (g.form == I8_PAIR)
        return launch_tc<i8_pair_kernel<SWIGLU, OutT>>(
                         P_STAGES * P_STAGE_BYTES + EPI * (P_STAGE_FLOATS + P_SCALE_FLOATS) * 4 + 1024 + sizeof(Ctl<P_STAGES>),
                         device_sm_count() & ~1, NUM_THREADS, m, kp, st);
    const int grid = std::min(device_sm_count(), kI8MaxGrid);
    constexpr size_t smem = S_STAGES * S_STAGE_BYTES + 1024 + sizeof(Ctl<S_STAGES>);
    // Few rows: four warps to an accumulator in place of eight, which a launch of one token pays for (49.6 -> 48.8 us and
    // 30.4 -> 29.7 us, 8 experts, 4096 <-> 14336); 129 rows to each of 68 experts of K = 64 take 49 us with four, 43 with eight.
    if (g.rows <= 64) return launch_tc<i8_single_kernel<SWIGLU, OutT, 1>>(smem + 8 * S_ROW_FLOATS * 4, grid, 320, m, kp, st);
    return launch_tc<i8_single_kernel<SWIGLU, OutT, 2>>(smem + 16 * S_ROW_FLOATS * 4, grid, 576, m, kp, st);
}

}  // namespace

cudaError_t launch_i8_tc(const I8Gemm& g, cudaStream_t st) {
    const bool swiglu = g.B1 != nullptr, pair = g.form == I8_PAIR;
    const long long brows = static_cast<long long>(g.E) * g.N;
    Maps m;
    const int box = pair ? 64 : 128;
    bool ok = map_i8(&m.a, g.A, g.rows, g.K, pair ? BM : 32) && map_i8(&m.b0, g.B0, brows, g.K, box);
    m.b1 = m.b0;
    if (swiglu) ok = ok && map_i8(&m.b1, g.B1, brows, g.K, box);
    if (pair) {
        ok = ok && map_i8(&m.x0, g.A, g.rows, g.K, 32);
        ok = ok && map_out(&m.x1, g.out, g.rows, g.N, g.out_dtype);
    } else if (g.N % 128 != 0 && g.N % 128 <= 64) {
        ok = ok && map_i8(&m.x0, g.B0, brows, g.K, 64) && map_i8(&m.x1, swiglu ? g.B1 : g.B0, brows, g.K, 64);
    } else {   // no box of 64 rows
        m.x0 = m.b0;
        m.x1 = m.b1;
    }
    if (!ok) return cudaErrorInvalidValue;
    KP kp = {};
    kp.indptr = g.indptr; kp.sa = g.sa; kp.sb0 = g.sb0; kp.sb1 = g.sb1; kp.out = g.out; kp.status = g.status;
    kp.timeout_ns = wait_limit_ns();
    kp.drain_ns = kDrainLimitNs;
    kp.E = g.E; kp.N = g.N; kp.K = g.K; kp.rows = g.rows;
    kp.nt = ceil_div(g.N, (swiglu ? 128 : 256) * (pair ? 2 : 1));
    const long long blk = static_cast<long long>(pair ? 256 : BM) * g.K;
    kp.band_m = static_cast<int>(std::max(8ll, kBandBytes / blk));
    if (!pair) { kp.part = g.part; kp.sem = g.sem; kp.part_rows = g.part_rows; }
    const int grid = std::min(device_sm_count(), kI8MaxGrid);
    if (grid < 2) return cudaErrorInvalidDevice;
    cudaError_t e = launch_dep(i8_begin_kernel, dim3(pair ? 1 : grid), dim3(256), 0, st, kp, grid);
    if (e != cudaSuccess) return e;
    if (g.out_dtype == MOE_DTYPE_BF16)
        return swiglu ? launch_form<true, __nv_bfloat16>(g, kp, m, st)
                      : launch_form<false, __nv_bfloat16>(g, kp, m, st);
    return swiglu ? launch_form<true, float>(g, kp, m, st) : launch_form<false, float>(g, kp, m, st);
}

}  // namespace moe
