// Products of the experts in 8-bit integers on the sm_100a tensor cores
// (tcgen05 kind::i8, 32-bit integer accumulators in TMEM, TMA-fed): for every
// group e and row r of it, with a scale for each token and channel,
//   PLAIN   out[r][n] = S(A, B0) sa_r sb0_{e,n},  S(A, B) = sum_c A[r][c] B_e[n][c]
//   SWIGLU  a = S(A, B0) sa sb0, b = S(A, B1) sa sb1, out = SiLU(a) b
// The integer sums are exact (K 128^2 < 2^31), so no order of K, tile or form
// of the kernel changes a bit of the result; the float factors are applied
// as (float(sum) * sa) * sb and the result is rounded once.
//
// Both forms here are persistent kernels of six warps: one loads by TMA into
// a ring of 128-byte K blocks (128-byte swizzle), one issues the MMAs, four
// read the accumulators back (tcgen05.ld), apply the scales and store, while
// the next tile runs into the other accumulator. The tile list is formed in
// each CTA's shared memory from the group offsets. Every wait is bounded
// (moe_set_wait_limit): on expiry the CTA records MOE_ERR_TIMEOUT, lets what
// it started land, frees its tensor memory and returns.
//  * pair: clusters of two CTAs share 256 x 256 tiles (M = 256, cta_group::2):
//    each loads 128 rows of A and half of the weight rows, which halves the
//    shared-memory traffic of the weights; groups of many rows.
//  * single: one CTA a tile of 256 weight rows and up to 128 rows of A, for
//    groups of few rows: the weights bound it.
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
constexpr int NUM_THREADS = 192;
constexpr int P_STAGES = 6, P_STAGE_BYTES = A_BYTES + BH_BYTES;
constexpr int S_STAGES = 4, S_STAGE_BYTES = A_BYTES + 2 * BH_BYTES;
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
    int *part, *sem;   // single form: parts of the tail tiles [slots][part_rows][256] and arrivals [tail][4]
    int part_rows;
};

template <int STAGES>
struct Ctl {
    uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    int cum[MOE_MAX_E + 1];   // tiles before group g
    int row0[MOE_MAX_E], nrow[MOE_MAX_E];
};

// Tiles of every group in front of it, by one warp: cum[0..E], row0, nrow. A
// group whose offsets do not fit in the rows is left out.
template <int STAGES>
__device__ __forceinline__ void list_tiles(Ctl<STAGES>* c, const KP& p, int tile_m) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.E; g0 += 32) {
        const int g = g0 + lane;
        int v = 0;
        if (g < p.E) {
            const int lo = p.indptr[g], hi = p.indptr[g + 1];
            const bool ok = lo >= 0 && hi >= lo && hi <= p.rows;
            const int n = ok ? hi - lo : 0;
            bad |= !ok;
            c->row0[g] = lo;
            c->nrow[g] = n;
            v = (n + tile_m - 1) / tile_m * p.nt;
        }
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (g < p.E) c->cum[g] = base + incl - v;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) c->cum[p.E] = base;
    if (kDebugChecks && __any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) {
        pdl_wait();
        debug_record_bounds(p.status);
    }
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
    t.rows = c->nrow[lo];
    t.row0 = c->row0[lo];
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
    t.m_blk = m0 + id % h;
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
            pdl_wait();   // the status word has been reset by then
            atomicExch(p.status, MOE_ERR_TIMEOUT);
            return false;
        }
    }
}
// On the abort path: copies and MMAs in flight land before the CTA leaves.
__device__ __forceinline__ void drain_i8(uint64_t* bar, uint32_t parity, const KP& p) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > static_cast<uint64_t>(p.drain_ns)) {
            pdl_wait();
            atomicExch(p.status, MOE_ERR_TIMEOUT);
            return;
        }
}

// SiLU with the exponential of the output's precision
__device__ __forceinline__ float silu(float a, float*) { return a / (1.f + expf(-a)); }
__device__ __forceinline__ float silu(float a, __nv_bfloat16*) { return __fdividef(a, 1.f + __expf(-a)); }

__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// One accumulator row of this thread: columns [c0, c0 + n) of the gate (or
// plain) accumulator at tb and, SWIGLU, of the up accumulator at tb + up;
// output columns from col0. N is a multiple of 16, so 16 columns at a time.
template <bool SWIGLU, typename OutT>
__device__ __forceinline__ void store_cols(const KP& p, uint32_t tb, uint32_t up, int n, int col0, int g, bool valid,
                                           size_t orow, float sa) {
    OutT* out = static_cast<OutT*>(p.out) + orow * p.N;
    const float* s0 = p.sb0 + static_cast<size_t>(g) * p.N;
    const float* s1 = SWIGLU ? p.sb1 + static_cast<size_t>(g) * p.N : nullptr;
#pragma unroll 1
    for (int c = 0; c < n; c += 32) {
        uint32_t a[32], b[SWIGLU ? 32 : 1];
        tmem_ld32(tb + c, a);
        if constexpr (SWIGLU) tmem_ld32(tb + up + c, b);
#pragma unroll
        for (int q = 0; q < 32; q += 16) {
            const int col = col0 + c + q;
            if (!valid || col >= p.N) continue;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(s0 + col + i));
                v[i] = static_cast<float>(static_cast<int>(a[q + i])) * sa * f.x;
                v[i + 1] = static_cast<float>(static_cast<int>(a[q + i + 1])) * sa * f.y;
                v[i + 2] = static_cast<float>(static_cast<int>(a[q + i + 2])) * sa * f.z;
                v[i + 3] = static_cast<float>(static_cast<int>(a[q + i + 3])) * sa * f.w;
                if constexpr (SWIGLU) {
                    const float4 h = __ldg(reinterpret_cast<const float4*>(s1 + col + i));
                    v[i] = silu(v[i], out) * (static_cast<float>(static_cast<int>(b[q + i])) * sa * h.x);
                    v[i + 1] = silu(v[i + 1], out) * (static_cast<float>(static_cast<int>(b[q + i + 1])) * sa * h.y);
                    v[i + 2] = silu(v[i + 2], out) * (static_cast<float>(static_cast<int>(b[q + i + 2])) * sa * h.z);
                    v[i + 3] = silu(v[i + 3], out) * (static_cast<float>(static_cast<int>(b[q + i + 3])) * sa * h.w);
                }
            }
            store16(out + col, v);
        }
    }
}

// ---- pair form ----------------------------------------------------------------
// Accumulator columns: SWIGLU [128 gate | 128 up] (rank 0's weight rows come
// from B0, rank 1's from B1), PLAIN 256 output columns. The tiles that do not
// fill a whole wave run as two half-width items each when that still fits in
// one wave (64 columns of each half), so the last wave is half as long.
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
__device__ __forceinline__ int item_tile(const Work& w, int v, int& half) {
    if (v < w.full) { half = -1; return v; }
    half = (v - w.full) & 1;
    return w.full + ((v - w.full) >> 1);
}

template <bool SWIGLU, typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
i8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
               const __grid_constant__ CUtensorMap tmB1, const KP p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using C = Ctl<P_STAGES>;
    C* ctl = reinterpret_cast<C*>(smem + P_STAGES * P_STAGE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const uint32_t peer_abort = mapa_shared(smem_u32(&ctl->abort_flag), rank ^ 1u);
    const int cluster = static_cast<int>(blockIdx.x >> 1), nclusters = static_cast<int>(gridDim.x >> 1);
    constexpr int TM = 256;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&ctl->tfull[a], 1);
            mbar_init(&ctl->tempty[a], 8);
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
    if (warp == 2) list_tiles(ctl, p, TM);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Work work = work_of(ctl->cum[p.E], nclusters);
    const int num_kb = (p.K + BKB - 1) / BKB;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_ph = 0;
            bool aborted = false;
            const CUtensorMap* mb = SWIGLU && rank ? &tmB1 : &tmB0;
            auto full_of = [&](int st) { return mapa_shared(smem_u32(&ctl->full[st]), 0u); };
            for (int u = cluster; u < work.items && !aborted; u += nclusters) {
                int hf;
                const Tile t = tile_of(ctl, p, item_tile(work, u, hf), TM);
                const int arow = t.row0 + t.m_blk * TM + rank * BM;
                const int brow = t.g * p.N + (SWIGLU ? t.n_blk * 128 : t.n_blk * 256 + rank * 128);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!wait_i8(&ctl->empty[s], ph ^ 1u, ctl, p, peer_abort)) { aborted = true; break; }
                    const uint32_t sa = smem_u32(smem + s * P_STAGE_BYTES);
                    if (leader) {
                        mbar_arrive_expect_tx(&ctl->full[s], 2 * P_STAGE_BYTES);
                        armed |= 1u << s;
                        armed_ph = (armed_ph & ~(1u << s)) | (ph << s);
                    }
                    tma_load_2d_pair(sa, &tmA, full_of(s), kb * BKB, arow);
                    tma_load_2d_pair(sa + A_BYTES, mb, full_of(s), kb * BKB, brow);
                    if (++s == P_STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (aborted) {
                if (leader) {
                    for (int st = 0; st < P_STAGES; ++st)
                        if ((armed >> st) & 1u) drain_i8(&ctl->full[st], (armed_ph >> st) & 1u, p);
                } else {
                    // its own copies complete on the leader's barriers: a fixed time for them to land
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 50000ull) {}
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool aborted = false, issued = false;
            for (int u = cluster; u < work.items && !aborted; u += nclusters) {
                int hf;
                item_tile(work, u, hf);
                const uint32_t id = hf < 0 ? idesc_i8(TM, 256) : idesc_i8(TM, 128);
                const uint32_t boff = hf > 0 ? 64u * BKB : 0u;
                if (!wait_i8(&ctl->tempty[acc], aph ^ 1u, ctl, p, peer_abort)) { aborted = true; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * ACC_COLS);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!wait_i8(&ctl->full[s], ph, ctl, p, peer_abort)) { aborted = true; break; }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + s * P_STAGE_BYTES);
                    const uint64_t ad = sw128_desc(sa), bd = sw128_desc(sa + A_BYTES + boff);
#pragma unroll
                    for (int kk = 0; kk < BKB / 32; ++kk)
                        mma_i8_pair(d, ad + 2u * kk, bd + 2u * kk, id, (kb | kk) != 0 ? 1u : 0u);
                    issued = true;
                    tc_commit_pair_mc(&ctl->empty[s], 0x3);
                    if (++s == P_STAGES) { s = 0; ph ^= 1u; }
                }
                if (aborted) break;
                tc_commit_pair_mc(&ctl->tfull[acc], 0x3);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            if (aborted && issued) {
                tc_commit_pair(&ctl->drain);
                drain_i8(&ctl->drain, 0, p);
            }
        }
    } else {
        const int q = warp & 3;
        const int r = rank * BM + q * 32 + lane;
        const uint32_t tempty0[2] = {mapa_shared(smem_u32(&ctl->tempty[0]), 0u),
                                     mapa_shared(smem_u32(&ctl->tempty[1]), 0u)};
        int acc = 0;
        uint32_t aph = 0;
        for (int u = cluster; u < work.items; u += nclusters) {
            int hf;
            const Tile t = tile_of(ctl, p, item_tile(work, u, hf), TM);
            const int grow = t.m_blk * TM + r;
            const bool valid = grow < t.rows;
            const size_t orow = static_cast<size_t>(t.row0) + static_cast<size_t>(grow);
            const float sa = valid ? p.sa[orow] : 0.f;
            if (!wait_i8(&ctl->tfull[acc], aph, ctl, p, peer_abort)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * ACC_COLS);
            if (hf < 0) {
                if (SWIGLU) store_cols<true, OutT>(p, tb, 128, 128, t.n_blk * 128, t.g, valid, orow, sa);
                else store_cols<false, OutT>(p, tb, 0, 256, t.n_blk * 256, t.g, valid, orow, sa);
            } else if (SWIGLU) {
                store_cols<true, OutT>(p, tb, 64, 64, t.n_blk * 128 + 64 * hf, t.g, valid, orow, sa);
            } else {
                store_cols<false, OutT>(p, tb, 0, 64, t.n_blk * 256 + 64 * hf, t.g, valid, orow, sa);
                store_cols<false, OutT>(p, tb + 64, 0, 64, t.n_blk * 256 + 128 + 64 * hf, t.g, valid, orow, sa);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(&ctl->tempty[acc]);
                else mbar_arrive_remote(tempty0[acc]);
            }
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

// ---- single form ----------------------------------------------------------------
// The weights are the M operand: a tile is 256 weight rows (two MMAs of M =
// 128: SWIGLU 128 channels of B0 and the same of B1, PLAIN 256 channels of
// B0) against up to 128 rows of A as N = 16, 32, .. 128, so a group of few
// rows costs few tensor cycles and few bytes beside its weights, and a
// thread of the epilogue owns a channel: its two scales are loaded once and
// every store of a warp is 32 consecutive channels of one row.
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
constexpr int kMinShare = 4;   // K blocks: shorter shares cost more in joining than they save
__device__ __forceinline__ Units units_of(int tiles, int nkb, int grid) {
    Units u;
    u.grid = grid;
    u.nkb = nkb;
    u.whole = tiles / grid;
    u.tail = tiles - u.whole * grid;
    const int shares = static_cast<int>((static_cast<long long>(u.tail) * nkb + kMinShare - 1) / kMinShare);
    u.n = max(min(grid, max(shares, u.tail)), 1);
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

// sixteen consecutive columns of this thread's TMEM lane, at two places
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
__device__ __forceinline__ void red_add(int* p, uint32_t v) {
    asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <bool SWIGLU, typename OutT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
i8_single_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const KP p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using C = Ctl<S_STAGES>;
    C* ctl = reinterpret_cast<C*>(smem + S_STAGES * S_STAGE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = static_cast<int>(blockIdx.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S_STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&ctl->tfull[a], 1);
            mbar_init(&ctl->tempty[a], 4);
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
    // what this call's first launch writes (the status word and the arrival
    // counters) is touched only after the wait at the epilogue's start or by
    // a wait that gave up; all else was complete before that launch began
    if (warp == 2) list_tiles(ctl, p, BM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Units un = units_of(ctl->cum[p.E], (p.K + BKB - 1) / BKB, static_cast<int>(gridDim.x));

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_ph = 0;
            bool aborted = false;
            Unit w;
            for (int i = 0; !aborted && unit_at(un, b, i, w); ++i) {
                const Tile t = tile_of(ctl, p, w.tile, BM);
                const int arow = t.row0 + t.m_blk * BM;
                const int boxes = (min(t.rows - t.m_blk * BM, BM) + 31) / 32;
                const int brow = t.g * p.N + (SWIGLU ? t.n_blk * 128 : t.n_blk * 256);
                const int brow1 = SWIGLU ? brow : brow + 128;
                const CUtensorMap* mb1 = SWIGLU ? &tmB1 : &tmB0;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wait_i8(&ctl->empty[s], ph ^ 1u, ctl, p)) { aborted = true; break; }
                    const uint32_t sa = smem_u32(smem + s * S_STAGE_BYTES);
                    mbar_arrive_expect_tx(&ctl->full[s], 2 * BH_BYTES + boxes * 32 * BKB);
                    armed |= 1u << s;
                    armed_ph = (armed_ph & ~(1u << s)) | (ph << s);
                    tma_load_2d(sa + A_BYTES, &tmB0, &ctl->full[s], kb * BKB, brow);
                    tma_load_2d(sa + A_BYTES + BH_BYTES, mb1, &ctl->full[s], kb * BKB, brow1);
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(sa + q * 32 * BKB, &tmA, &ctl->full[s], kb * BKB, arow + 32 * q);
                    if (++s == S_STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (aborted)
                for (int st = 0; st < S_STAGES; ++st)
                    if ((armed >> st) & 1u) drain_i8(&ctl->full[st], (armed_ph >> st) & 1u, p);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool aborted = false, issued = false;
            Unit w;
            for (int i = 0; !aborted && unit_at(un, b, i, w); ++i) {
                const Tile t = tile_of(ctl, p, w.tile, BM);
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
                        mma_i8(d + 128u, w1 + 2u * kk, xd + 2u * kk, id, accum);
                    }
                    issued = true;
                    tc_commit(&ctl->empty[s]);
                    if (++s == S_STAGES) { s = 0; ph ^= 1u; }
                }
                if (aborted) break;
                tc_commit(&ctl->tfull[acc]);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            if (aborted && issued) {
                tc_commit(&ctl->drain);
                drain_i8(&ctl->drain, 0, p);
            }
        }
    } else {
        const int q = warp & 3, r = q * 32 + lane;   // this thread's channel of each half
        int acc = 0;
        uint32_t aph = 0;
        pdl_wait();
        OutT* out = static_cast<OutT*>(p.out);
        Unit w;
        for (int i = 0; unit_at(un, b, i, w); ++i) {
            const Tile t = tile_of(ctl, p, w.tile, BM);
            int nrow = min(t.rows - t.m_blk * BM, BM);
            const size_t row0 = static_cast<size_t>(t.row0) + static_cast<size_t>(t.m_blk) * BM;
            const int ch0 = (SWIGLU ? t.n_blk * 128 : t.n_blk * 256) + r, ch1 = SWIGLU ? ch0 : ch0 + 128;
            const size_t sc = static_cast<size_t>(t.g) * p.N;
            const float f0 = ch0 < p.N ? p.sb0[sc + ch0] : 0.f;
            const float f1 = ch1 < p.N ? (SWIGLU ? p.sb1 : p.sb0)[sc + ch1] : 0.f;
            float sa_l[4];   // row scales: lane l holds rows l, 32 + l, 64 + l, 96 + l
#pragma unroll
            for (int j = 0; j < 4; ++j) sa_l[j] = 32 * j + lane < nrow ? p.sa[row0 + 32 * j + lane] : 0.f;
            if (!wait_i8(&ctl->tfull[acc], aph, ctl, p)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * ACC_COLS);
            int* sums = p.part + static_cast<size_t>(w.tail) * 256 * p.part_rows + r;   // [row][256 channels]
            if (w.parts > 1) {
#pragma unroll 1
                for (int c = 0; c < nrow; c += 16) {
                    uint32_t lo[16], hi[16];
                    tmem_ld16x2(tb + c, tb + 128 + c, lo, hi);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < nrow) {
                            red_add(sums + (c + j) * 256, lo[j]);
                            red_add(sums + (c + j) * 256 + 128, hi[j]);
                        }
                }
                __threadfence();
                __syncwarp();
                int old = 0;
                if (lane == 0) old = atomicAdd(p.sem + w.tail * 4 + q, 1);
                old = __shfl_sync(0xffffffffu, old, 0);
                __threadfence();
                if (old != w.parts - 1) nrow = 0;   // another part comes later: its warp finishes
            }
            {
#pragma unroll 1
                for (int c = 0; c < nrow; c += 16) {
                    uint32_t lo[16], hi[16];
                    if (w.parts == 1) {
                        tmem_ld16x2(tb + c, tb + 128 + c, lo, hi);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            lo[j] = c + j < nrow ? static_cast<uint32_t>(__ldcg(sums + (c + j) * 256)) : 0u;
                            hi[j] = c + j < nrow ? static_cast<uint32_t>(__ldcg(sums + (c + j) * 256 + 128)) : 0u;
                        }
                    }
                    const float sa_c = c < 32 ? sa_l[0] : c < 64 ? sa_l[1] : c < 96 ? sa_l[2] : sa_l[3];
                    OutT* o = out + (row0 + c) * p.N;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float sa = __shfl_sync(0xffffffffu, sa_c, (c & 16) + j);
                        const bool in = c + j < nrow;
                        const float y0 = static_cast<float>(static_cast<int>(lo[j])) * sa * f0;
                        const float y1 = static_cast<float>(static_cast<int>(hi[j])) * sa * f1;
                        if (SWIGLU) {
                            if (in && ch0 < p.N) put(o + static_cast<size_t>(j) * p.N + ch0, silu(y0, out) * y1);
                        } else {
                            if (in && ch0 < p.N) put(o + static_cast<size_t>(j) * p.N + ch0, y0);
                            if (in && ch1 < p.N) put(o + static_cast<size_t>(j) * p.N + ch1, y1);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[acc]);
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

// First launch of a product: the status word is MOE_OK, and the arrival
// counters and accumulators of the tail tiles are zero, before any CTA of the
// product touches them. The product starts beside it (it needs nothing of
// this until its own wait).
__global__ void __launch_bounds__(256) i8_begin_kernel(const KP p, int grid) {
    __shared__ Ctl<1> c;
    pdl_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;
    if (p.part == nullptr) return;
    if (threadIdx.x < 32) list_tiles(&c, p, BM);
    __syncthreads();
    const Units u = units_of(c.cum[p.E], (p.K + BKB - 1) / BKB, grid);
    if (u.n <= u.tail) return;   // no tile has more than one part
    for (int t = blockIdx.x; t < u.tail; t += gridDim.x) {
        const Tile tile = tile_of(&c, p, u.whole * u.grid + t, BM);
        const int n = min(tile.rows - tile.m_blk * BM, BM) * 64;
        int4* part = reinterpret_cast<int4*>(p.part + static_cast<size_t>(t) * 256 * p.part_rows);
        for (int i = threadIdx.x; i < n; i += 256) part[i] = make_int4(0, 0, 0, 0);
        if (threadIdx.x < 4) p.sem[t * 4 + threadIdx.x] = 0;
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

template <typename Kernel>
cudaError_t launch_tc(Kernel kernel, size_t smem, int grid, const CUtensorMap& a, const CUtensorMap& b0,
                      const CUtensorMap& b1, const KP& kp, cudaStream_t st) {
    // the attribute belongs to the current device's context: set at every launch (a host-side call of about 1 us)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_k(kernel, dim3(grid), dim3(NUM_THREADS), smem, st, a, b0, b1, kp);
}

template <bool SWIGLU, typename OutT>
cudaError_t launch_form(const I8Gemm& g, const KP& kp, const CUtensorMap& a, const CUtensorMap& b0,
                        const CUtensorMap& b1, cudaStream_t st) {
    if (g.form == I8_PAIR)
        return launch_tc(i8_pair_kernel<SWIGLU, OutT>, P_STAGES * P_STAGE_BYTES + 1024 + sizeof(Ctl<P_STAGES>),
                         device_sm_count() & ~1, a, b0, b1, kp, st);
    return launch_tc(i8_single_kernel<SWIGLU, OutT>, S_STAGES * S_STAGE_BYTES + 1024 + sizeof(Ctl<S_STAGES>),
                     std::min(device_sm_count(), kI8MaxGrid), a, b0, b1, kp, st);
}

}  // namespace

cudaError_t launch_i8_tc(const I8Gemm& g, cudaStream_t st) {
    const bool swiglu = g.B1 != nullptr, pair = g.form == I8_PAIR;
    const long long brows = static_cast<long long>(g.E) * g.N;
    CUtensorMap a, b0, b1;
    if (!map_i8(&a, g.A, g.rows, g.K, pair ? BM : 32) || !map_i8(&b0, g.B0, brows, g.K, 128)) return cudaErrorInvalidValue;
    b1 = b0;
    if (swiglu && !map_i8(&b1, g.B1, brows, g.K, 128)) return cudaErrorInvalidValue;
    KP kp = {};
    kp.indptr = g.indptr; kp.sa = g.sa; kp.sb0 = g.sb0; kp.sb1 = g.sb1; kp.out = g.out; kp.status = g.status;
    kp.timeout_ns = wait_limit_ns();
    kp.drain_ns = kDrainLimitNs;
    kp.E = g.E; kp.N = g.N; kp.K = g.K; kp.rows = g.rows;
    kp.nt = ceil_div(g.N, swiglu ? 128 : 256);
    const long long blk = static_cast<long long>(pair ? 256 : BM) * g.K;
    kp.band_m = static_cast<int>(std::max(8ll, kBandBytes / blk));
    if (!pair) { kp.part = g.part; kp.sem = g.sem; kp.part_rows = g.part_rows; }
    const int grid = std::min(device_sm_count(), kI8MaxGrid);
    if (grid < 2) return cudaErrorInvalidDevice;
    cudaError_t e = launch_k(i8_begin_kernel, dim3(pair ? 1 : grid), dim3(256), 0, st, kp, grid);
    if (e != cudaSuccess) return e;
    struct Dependent {   // the product is launched as a programmatic dependent of it
        Dependent() { g_pdl = true; }
        ~Dependent() { g_pdl = false; }
    } dependent;
    if (g.out_dtype == MOE_DTYPE_BF16)
        return swiglu ? launch_form<true, __nv_bfloat16>(g, kp, a, b0, b1, st)
                      : launch_form<false, __nv_bfloat16>(g, kp, a, b0, b1, st);
    return swiglu ? launch_form<true, float>(g, kp, a, b0, b1, st) : launch_form<false, float>(g, kp, a, b0, b1, st);
}

}  // namespace moe
