// linear_bwd_tc.cu - the whole backward of a linear layer up to 128 wide on the input side in one
// pass over the batch, on tcgen05 tensor cores.
//
//   p = x W^T + b,  D = dy act'(p),  dx = D W,  dW = D^T x,  db = sum of D over the rows
//
// What bounds it: memory. A row of x, dy and dx is 2 (2 k + n) bytes; done as three products with
// D in memory it is read and written 2.3 times over (147456 x 128 -> 128 with sigmoid: 79 us). Here a
// CTA takes tiles of 128 rows, and from one copy of x and dy in shared memory makes all of it:
//   * W (up to 256 rows of it) stays in shared memory for the whole call, left in the one
//     layout that serves both as the right operand of p (K-major) and of dx (MN-major);
//   * per tile and 128 columns of n: p in tensor memory; sixteen worker warps turn dy into D
//     in place (the tile it arrived in); D is then the K-major left operand of dx and the
//     MN-major left operand of dW, x the MN-major right operand of dW, all as they lie;
//   * dx leaves tensor memory once per tile; dW stays there as a running sum over all the CTA's
//     tiles (128 or 256 columns) and is written once, in fp32, for linear_reduce_kernel to add up
//     the CTAs' parts in order; db likewise, summed from D before its rounding.
// n over 256 (kPair): two CTAs of a cluster take the same rows and 256 columns of n each, and send
// each other half of their parts of dx through distributed shared memory.
// kHeld8: x comes as E4M3 codes and E8M0 scales; the workers turn each tile into bf16 as it
// arrives, so the 8-bit form is all that is read.
//
// The workers read p in the 16 x 256-bit fragment form, so ldmatrix and stmatrix meet it in the
// swizzled tile without conflicts, and a lane's part of db is eight columns: it adds its rows in
// registers, tile after tile, and the lanes are joined once, at the end.
//
// D enters the products in bf16, their operand type: dx and dW are off by 0.0024 of their norm, against 0.0017 of their
// own rounding alone.
//
// Measured, call after call on the same inputs (and one call on inputs cold in L2): 147456 x 128 -> 128 with sigmoid
// 31 us (38), of which the sums over the CTAs are 4 and the start, where every CTA waits for its first tiles at once,
// 5; with relu, whose norms (linear_act.cuh) are the workers' too, 38 (44); -> 512 with silu 109 us (118), x in 8
// bits 123 (132): there the workers wait, on tensor memory and for their pair's part of dx.
//
// Roles: warp 0 TMA, warp 1 MMA issue, warps 2-17 workers. Every wait is bounded; see the barrier
// list below. Order within a tile, so that no role waits on itself: the MMA warp issues p of
// the next unit before it waits for D of this one (kHeld8: not across tiles, where x is still read),
// and dW of a unit before dx, which may wait for the drain of the tile before; the workers drain
// that after the tile's first unit.
#include <cuda_fp8.h>

#include "kernels.h"
#include "linear_act.cuh"

namespace trimul {
namespace lb {
constexpr int TILE = 128 * 128 * 2;       // 128 rows x 128 columns of bf16: two blocks of 64 columns
constexpr int HALF = TILE / 2;
constexpr int WORKERS = 16;
constexpr int THREADS = (2 + WORKERS) * 32;
constexpr int CODES = 128 * 128;          // a tile's codes
constexpr int OUT = 32 * 64;              // a worker's block of dx: 32 rows x 32 columns
constexpr int BAR_BYTES = 384;
// Four 32 KB tiles for W's slab and x: what W leaves is x's (with three tiles of x the next p need not
// wait for a load behind the last dW: 40 -> 37.5 us at 147456 x 128 -> 128). kHeld8: one tile of
// x in bf16, and the rest of x's share as 16 KB tiles of codes. Two tiles of dy, and 32 KB of dx blocks.
__host__ __device__ constexpr int xbufs(int chunks) { return 4 - chunks; }
__host__ __device__ constexpr int cbufs(int chunks) { return 2 * (3 - chunks); }
constexpr int XNORM = 2 * 128 * 2;        // relu: norms of two tiles' rows of x, bf16
constexpr size_t SMEM = 1024 + 7 * (size_t)TILE + 1024 + BAR_BYTES + XNORM;
static_assert(SMEM <= 232448, "shared memory budget");
constexpr int TMEM_COLS = 512, DX_COL = 384;
}  // namespace lb

namespace {

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ float2 two(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

// 16 bytes into a CTA of the cluster, counted on a barrier there when they land: the sender need not
// wait for its stores (a fence for plain remote ones took 5500 cycles a tile).
__device__ __forceinline__ void st_async_v4(uint32_t cluster_addr, uint32_t cluster_bar, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(cluster_addr),
        "r"(cluster_bar), "r"(a), "r"(b), "r"(c), "r"(d)
        : "memory");
}

// Four bf16 at column 4 l of row r of a 128 x 128 tile.
__device__ __forceinline__ uint2 tile_quad(const uint8_t *tile, int r, int l) {
    return *reinterpret_cast<const uint2 *>(tile + (l >> 4) * lb::HALF + r * 128 + ((((l & 15) >> 1) ^ (r & 7)) << 4) + (l & 1) * 8);
}

// A worker's 32 x 32 block of D in place of dy, at the lane's row address `tile` (8-column chunk c0 and
// on, row & 7 = x7); dsum gets the column sums over the lane's four rows. p as in make_d.
template <int ACT, bool kShare>
__device__ __forceinline__ void write_d(const float2 (&p)[16], uint32_t keep, uint32_t tile, int c0, int x7, float2 (&dsum)[4]) {
#pragma unroll
    for (int rh = 0; rh < 2; ++rh)
#pragma unroll
        for (int jp = 0; jp < 2; ++jp) {
            uint32_t dy[4];  // (row, row + 8) of column block 2 jp, then of 2 jp + 1
            const uint32_t at = tile + rh * 2048 + (uint32_t)(((c0 + 2 * jp) ^ x7) << 4);
            ldmatrix4(dy, at);
            float2 d[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) d[x] = two(dy[x]);
            if (ACT == LIN_RELU) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t b = keep >> (2 * (rh * 8 + 4 * jp + x));
                    d[x] = make_float2(b & 1u ? d[x].x : 0.f, b & 2u ? d[x].y : 0.f);
                }
            } else if (ACT != LIN_NONE) {
#pragma unroll
                for (int x = 0; x < 4; x += 2) {
                    float2 y[2] = {p[rh * 8 + 4 * jp + x], p[rh * 8 + 4 * jp + x + 1]};
                    const float2 e[2] = {d[x], d[x + 1]};
                    act_grad4<ACT, kShare>(y, e);
                    d[x] = y[0];
                    d[x + 1] = y[1];
                }
            }
            dsum[2 * jp] = __fadd2_rn(dsum[2 * jp], __fadd2_rn(d[0], d[1]));
            dsum[2 * jp + 1] = __fadd2_rn(dsum[2 * jp + 1], __fadd2_rn(d[2], d[3]));
            if (ACT != LIN_NONE) {
                uint32_t o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) o[x] = pack_bf16x2(d[x].x, d[x].y);
                stmatrix4(at, o);
            }
        }
}

}  // namespace

template <int CHUNKS, bool kPair, bool kHeld8, int ACT>
__global__ void __launch_bounds__(lb::THREADS, 1)
    linear_bwd_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmDy, const __grid_constant__ CUtensorMap tmDx,
                      const LinearBwdArgs args) {
    using namespace lb;
    constexpr int PRE = CHUNKS == 1 ? 2 : 1;     // accumulators of p
    constexpr int PRE_COL = 128 * CHUNKS;
    constexpr int XB = kHeld8 ? cbufs(CHUNKS) : xbufs(CHUNKS);  // tiles of x (codes) in flight
    static_assert(XB <= 4, "barriers");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *wbuf = smem;                               // [CHUNKS] 128 rows of W
    uint8_t *xbuf = wbuf + CHUNKS * TILE;               // [XB]; kHeld8: one tile
    uint8_t *codes = xbuf + TILE;                       // kHeld8: [XB]
    uint8_t *dbuf = xbuf + xbufs(CHUNKS) * TILE;        // [2] dy, then D
    uint8_t *obuf = dbuf + 2 * TILE;                    // [WORKERS] 2 KB; kPair: [8] 4 KB
    float *fbuf = reinterpret_cast<float *>(obuf + WORKERS * OUT);  // bias [256]
    uint32_t *rbuf = reinterpret_cast<uint32_t *>(fbuf);  // relu: the bias's bf16 below the norm of W's row, bf16 too
    uint64_t *bars = reinterpret_cast<uint64_t *>(fbuf + 256);
    __nv_bfloat16 *xnorm = reinterpret_cast<__nv_bfloat16 *>(reinterpret_cast<uint8_t *>(bars) + BAR_BYTES);  // [2][128]
    uint64_t *wfull = bars;            // W landed
    uint64_t *xfull = bars + 1;        // [XB] x (kHeld8: codes) landed
    uint64_t *xfree = bars + 5;        // [XB] products reading x are done (kHeld8: codes read, WORKERS arrivals)
    uint64_t *xready = bars + 9;       // kHeld8: x turned into bf16 (WORKERS arrivals)
    uint64_t *xdone = bars + 10;       // kHeld8: products reading x are done
    uint64_t *dfull = bars + 11;       // [2] dy landed
    uint64_t *dready = bars + 13;      // [2] D written (WORKERS arrivals)
    uint64_t *dfree = bars + 15;       // [2] products reading D are done
    uint64_t *pfull = bars + 17;       // [2] p complete
    uint64_t *pfree = bars + 19;       // [2] p read (WORKERS arrivals)
    uint64_t *dxfull = bars + 21;      // dx of a tile complete
    uint64_t *dxfree = bars + 22;      // dx read (WORKERS arrivals)
    uint64_t *drain = bars + 23;       // every product is done
    uint64_t *rfull = bars + 24;       // kPair: [8] the peer's part of a block of dx is here
    uint64_t *sfree = bars + 32;       // kPair: [8] the peer has room for the next part
    volatile uint32_t *sent = reinterpret_cast<volatile uint32_t *>(bars + 40);  // kPair: [8] parts the peer has sent
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 44);
    uint64_t *nready = bars + 45;      // relu: the norms of a tile's rows are written (WORKERS arrivals)
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KernelCtl &ctl = args.ctl;
    // kPair: the two CTAs of a cluster take the same rows, each 256 columns of n from n_first.
    const uint32_t rank = kPair ? cluster_rank() : 0u;
    const int team = kPair ? (int)blockIdx.x >> 1 : (int)blockIdx.x, teams = kPair ? (int)gridDim.x >> 1 : (int)gridDim.x;
    const int n_first = 256 * (int)rank, n_mine = min(args.n - n_first, 128 * CHUNKS);
    const int my_tiles = (args.row_tiles - team + teams - 1) / teams;
    const int units = my_tiles * CHUNKS;
    constexpr bool has_p = ACT != LIN_NONE;
    auto row0 = [&](int t) { return (team + t * teams) * 128; };

    if (threadIdx.x == 0) {
        mbar_init(wfull, 1);
        mbar_init(xready, WORKERS);
        mbar_init(xdone, 1);
        for (int i = 0; i < XB; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xfree[i], kHeld8 ? WORKERS : 1);
        }
        mbar_init(dxfull, 1);
        mbar_init(dxfree, WORKERS);
        mbar_init(drain, 1);
        mbar_init(nready, WORKERS);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dready[i], WORKERS);
            mbar_init(&dfree[i], 1);
            mbar_init(&pfull[i], 1);
            mbar_init(&pfree[i], WORKERS);
        }
        if (kPair)
            for (int i = 0; i < 8; ++i) {
                sent[i] = 0;
                mbar_init(&rfull[i], 1);
                mbar_init(&sfree[i], 1);
            }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmDy);
        if (args.has_dx) tma_prefetch_desc(&tmDx);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < 128 * CHUNKS; i += THREADS) {
        const uint32_t b = (args.bias && i < n_mine) ? reinterpret_cast<const uint16_t *>(args.bias)[n_first + i] : 0u;
        rbuf[i] = ACT == LIN_RELU ? b : b << 16;
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (args.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *ctl.status = DeviceStatus{0, 0, 0, 0};

    // Workers keep these across their branch: db of their columns.
    float2 dbs[CHUNKS][4];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) dbs[c][j] = make_float2(0.f, 0.f);
    const int ew = warp - 2, q = warp & 3, h = ew >> 2;  // worker: rows 32 q .., columns 32 h .. of a tile
    const uint32_t lanebase = tmem + ((uint32_t)(q * 32) << 16);
    bool ok = true;
    int my_parts = 0;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA ----------------
            int xs = 0, ds = 0;  // tiles of x and units of dy asked for
            mbar_arrive_expect_tx(wfull, CHUNKS * TILE);
            for (int c = 0; c < CHUNKS; ++c)
                for (int kb = 0; kb < 2; ++kb) tma_load_3d(wbuf + c * TILE + kb * HALF, &tmW, wfull, kb * 64, n_first + c * 128, 0);
            for (int u = 0; ok && u < units; ++u) {
                const int t = u / CHUNKS, c = u - t * CHUNKS;
                if (c == 0) {
                    const int xb = t % XB;
                    if (t >= XB && !(ok = wait_bounded(&xfree[xb], (uint32_t)(t / XB - 1) & 1u, abort_flag, ctl, SITE_LBW | 1, t))) break;
                    if (kHeld8) {
                        mbar_arrive_expect_tx(&xfull[xb], CODES);
                        tma_load_3d(codes + xb * CODES, &tmX, &xfull[xb], 0, row0(t), 0);
                    } else {
                        mbar_arrive_expect_tx(&xfull[xb], TILE);
                        for (int kb = 0; kb < 2; ++kb)
                            tma_load_3d(xbuf + xb * TILE + kb * HALF, &tmX, &xfull[xb], kb * 64, row0(t), 0);
                    }
                    ++xs;
                }
                const int db = u & 1;
                if (u >= 2 && !(ok = wait_bounded(&dfree[db], (uint32_t)((u >> 1) - 1) & 1u, abort_flag, ctl, SITE_LBW | 2, u))) break;
                mbar_arrive_expect_tx(&dfull[db], TILE);
                for (int nb = 0; nb < 2; ++nb)
                    tma_load_3d(dbuf + db * TILE + nb * HALF, &tmDy, &dfull[db], n_first + c * 128 + nb * 64, row0(t), 0);
                ++ds;
            }
            // No copy may be in flight when the CTA leaves.
            wait_drain(wfull, 0, ctl.timeout_ns);
            for (int x = max(0, xs - XB); x < xs; ++x) wait_drain(&xfull[x % XB], (uint32_t)(x / XB) & 1u, ctl.timeout_ns);
            for (int d = max(0, ds - 2); d < ds; ++d) wait_drain(&dfull[d & 1], (uint32_t)(d >> 1) & 1u, ctl.timeout_ns);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issue ----------------
            const uint32_t i_p = idesc_bf16(128, 128, 0, 0), i_dx = idesc_bf16(128, 128, 0, 1), i_dw = idesc_bf16(128, 128, 1, 1);
            const uint32_t w0 = smem_u32(wbuf), x0 = smem_u32(xbuf), d0 = smem_u32(dbuf);
            ok = wait_bounded(wfull, 0, abort_flag, ctl, SITE_LBW | 3, 0);
            auto xtile = [&](int t) { return x0 + (kHeld8 ? 0u : (uint32_t)((t % XB) * TILE)); };
            auto wait_x = [&](int t) {
                if (kHeld8) return wait_bounded(xready, (uint32_t)t & 1u, abort_flag, ctl, SITE_LBW | 4, t);
                return wait_bounded(&xfull[t % XB], (uint32_t)(t / XB) & 1u, abort_flag, ctl, SITE_LBW | 4, t);
            };
            // p of unit u, once x is there and the accumulator has been read.
            auto issue_p = [&](int u) {
                const int t = u / CHUNKS, c = u - t * CHUNKS, a = u % PRE;
                if (c == 0 && !wait_x(t)) return false;
                if (u >= PRE && !wait_bounded(&pfree[a], (uint32_t)(u / PRE - 1) & 1u, abort_flag, ctl, SITE_LBW | 5, u)) return false;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_bf16(tmem + PRE_COL + 128 * a, sdesc_sw128(xtile(t) + (j >> 2) * HALF + (j & 3) * 32, 16, 1024),
                             sdesc_sw128(w0 + c * TILE + (j >> 2) * HALF + (j & 3) * 32, 16, 1024), i_p, j ? 1u : 0u);
                mma_commit(&pfull[a]);
                return true;
            };
            if (ok && has_p && units > 0) ok = issue_p(0);
            for (int u = 0; ok && u < units; ++u) {
                const int t = u / CHUNKS, c = u - t * CHUNKS, db = u & 1;
                const bool wait_for_x = kHeld8 && c == CHUNKS - 1;  // the next p needs x's tile, which dW here still reads
                if (has_p && u + 1 < units && !wait_for_x && !(ok = issue_p(u + 1))) break;
                if (!has_p && c == 0 && !(ok = wait_x(t))) break;
                if (!(ok = wait_bounded(&dready[db], (uint32_t)(u >> 1) & 1u, abort_flag, ctl, SITE_LBW | 6, u))) break;
                tc_fence_after();
                const uint32_t dt = d0 + db * TILE;
                if (args.has_dw) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mma_bf16(tmem + 128 * c, sdesc_sw128(dt + j * 2048, HALF, 1024), sdesc_sw128(xtile(t) + j * 2048, HALF, 1024),
                                 i_dw, (t | j) ? 1u : 0u);
                }
                if (c == CHUNKS - 1) mma_commit(kHeld8 ? xdone : &xfree[t % XB]);  // the last product that reads x
                if (args.has_dx) {
                    if (c == 0 && t > 0) {
                        if (!(ok = wait_bounded(dxfree, (uint32_t)(t - 1) & 1u, abort_flag, ctl, SITE_LBW | 7, t))) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mma_bf16(tmem + DX_COL, sdesc_sw128(dt + (j >> 2) * HALF + (j & 3) * 32, 16, 1024),
                                 sdesc_sw128(w0 + c * TILE + j * 2048, HALF, 1024), i_dx, (c | j) ? 1u : 0u);
                }
                mma_commit(&dfree[db]);
                if (c == CHUNKS - 1) mma_commit(dxfull);
                if (has_p && u + 1 < units && wait_for_x && !(ok = issue_p(u + 1))) break;
            }
            mma_commit(drain);
            wait_drain(drain, 0, ctl.timeout_ns);
        }
    } else {
        // ---------------- workers ----------------
        const uint32_t la_off = (uint32_t)((32 * q + (lane & 7) + ((lane >> 3) & 1) * 8) * 128);  // row of an ldmatrix address
        const int la_c = lane >> 4, x7 = lane & 7;
        // kPair: dx is the sum of both CTAs' products. Columns 0-63 are finished by rank 0, 64-127 by rank 1: a
        // worker of the other half sends its 32 x 32 block, in the order its lanes hold it, to the worker with
        // the same rows and columns of the peer, which adds its own.
        const bool home = !kPair || (h >> 1) == (int)rank;
        const int pslot = 2 * q + (h & 1);
        uint8_t *ob = kPair ? obuf + pslot * 4096 : obuf + ew * OUT;
        bool owes_room = false;  // the block's buffer is still to be given back to the sender
        int parts = 0;           // parts of dx sent, or waited for
        auto give_room = [&]() {
            if (kPair && owes_room) {
                if (lane == 0) {
                    tma_store_wait_read<0>();
                    mbar_arrive_remote(map_to_rank(&sfree[pslot], rank ^ 1u));
                }
                owes_room = false;
            }
        };
        // kHeld8: thread (row, 32-column block) of the conversion
        const int crow = ew * 8 + (lane >> 2), cblk = lane & 3, kblk = args.k >> 5;

        auto scale_of = [&](int t) -> uint32_t {
            const long long r = (long long)row0(t) + crow;
            return (kHeld8 && t < my_tiles && r < args.rows && cblk < kblk) ? (uint32_t)__ldg(args.scales + r * kblk + cblk) : 0u;
        };
        uint32_t scale_next = kHeld8 ? scale_of(0) : 0u;
        // relu: the norms that bound p's rounding, rounded up to bf16: W's once, x's for each tile, eight rows a warp. A
        // tile's go to the buffer of the tile before the last, which every warp has left when all have written the
        // last one's. kHeld8: with the conversion, whose threads have the values in hand, and whose barrier covers them.
        auto norms = [&](const uint8_t *tile) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint2 v = tile_quad(tile, 8 * ew + i, lane);
                s[i] = add_squares(add_squares(0.f, v.x), v.y);
            }
            return sums_of_8(s, lane);
        };
        auto write_w_norms = [&]() {
            if (!warp_wait(wfull, 0, abort_flag, ctl, SITE_LBW | 14, 0)) return false;
#pragma unroll 1
            for (int cc = 0; cc < CHUNKS; ++cc) {
                const __nv_bfloat16 v = __float2bfloat16_ru(norm_of(norms(wbuf + cc * TILE)));
                if ((lane & 3) == 0) reinterpret_cast<__nv_bfloat16 *>(rbuf + cc * 128 + 8 * ew + (lane >> 2))[1] = v;
            }
            return true;
        };
        auto write_x_norm = [&](int t, float squares) {  // of row 8 ew + lane / 4
            if ((lane & 3) == 0) xnorm[(t & 1) * 128 + 8 * ew + (lane >> 2)] = __float2bfloat16_ru(norm_of(squares));
        };
        auto write_norms = [&](int t) {
            if (t == 0 && !write_w_norms()) return false;
            if (!warp_wait(&xfull[t % XB], (uint32_t)(t / XB) & 1u, abort_flag, ctl, SITE_LBW | 14, t)) return false;
            write_x_norm(t, norms(xbuf + (t % XB) * TILE));
            __syncwarp();
            if (lane == 0) mbar_arrive(nready);
            return true;
        };

        auto convert = [&](int t) {
            if (ACT == LIN_RELU && t == 0 && !write_w_norms()) return false;
            if (!warp_wait(&xfull[t % XB], (uint32_t)(t / XB) & 1u, abort_flag, ctl, SITE_LBW | 8, t)) return false;
            if (t > 0 && !warp_wait(xdone, (uint32_t)(t - 1) & 1u, abort_flag, ctl, SITE_LBW | 9, t)) return false;
            const uint32_t s = scale_next;
            scale_next = scale_of(t + 1);
            const float size = e8m0_value(s);
            const uint8_t *src = codes + (t % XB) * CODES + crow * 128;
            uint8_t *dst = xbuf + (cblk >> 1) * HALF + crow * 128;
            float squares = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + (((2 * cblk + i) ^ (crow & 7)) << 4));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const __half2_raw hv = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hv));
                    o[j] = pack_bf16x2(f.x * size, f.y * size);
                    if (ACT == LIN_RELU) squares = add_squares(squares, o[j]);
                }
                const int ch = 4 * (cblk & 1) + 2 * i;
                *reinterpret_cast<uint4 *>(dst + ((ch ^ (crow & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(dst + (((ch + 1) ^ (crow & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            if (ACT == LIN_RELU) {
                squares += __shfl_xor_sync(0xffffffffu, squares, 1);
                write_x_norm(t, squares + __shfl_xor_sync(0xffffffffu, squares, 2));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&xfree[t % XB]);
                mbar_arrive(xready);
            }
            return true;
        };

        // D of unit u in place of dy; db of its columns.
        auto make_d = [&](int u) {
            const int t = u / CHUNKS, c = u - t * CHUNKS, a = u % PRE, db = u & 1;
            give_room();
            float2 p[16];  // [16-row half][8-column block][row, row + 8]
            if (has_p) {
                if (!warp_wait(&pfull[a], (uint32_t)(u / PRE) & 1u, abort_flag, ctl, SITE_LBW | 10, u)) return false;
                tc_fence_after();
                uint32_t v[2][16];
#pragma unroll
                for (int rh = 0; rh < 2; ++rh)
                    tmem_ld16x256_x4(lanebase + ((uint32_t)(16 * rh) << 16) + (uint32_t)(PRE_COL + 128 * a + 32 * h), v[rh]);
                tmem_ld_wait_regs(v[0]);
                tmem_ld_wait_regs(v[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfree[a]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = c * 128 + 32 * h + 8 * j + 2 * (lane & 3);
                    const float2 bv = ACT == LIN_RELU ? make_float2(__uint_as_float(rbuf[col] << 16), __uint_as_float(rbuf[col + 1] << 16))
                                                      : *reinterpret_cast<const float2 *>(fbuf + col);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float2 &y = p[(x >> 1) * 8 + 2 * j + (x & 1)];
                        const uint32_t *r = &v[x >> 1][4 * j + 2 * (x & 1)];
                        y = __fadd2_rn(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])), bv);
                    }
                }
            }
            if (!warp_wait(&dfull[db], (uint32_t)(u >> 1) & 1u, abort_flag, ctl, SITE_LBW | 11, u)) return false;
            const uint32_t tile = smem_u32(dbuf + db * TILE + (h >> 1) * HALF) + la_off;
            float2 dsum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            uint32_t keep = 0xFFFFFFFFu;  // relu: bit 2 i + e of value p[i].x or .y
            if (ACT == LIN_RELU) {
                // Where p is under the bound of its rounding (linear_act.cuh) its sign is taken again in 64 bits.
                uint32_t check = 0;
                keep = 0;
                if (c == 0 && !warp_wait(kHeld8 ? xready : nready, (uint32_t)t & 1u, abort_flag, ctl, SITE_LBW | 14, u)) return false;
                float bound[4];  // of rows 16 (x >> 1) + 8 (x & 1) + lane / 4
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    bound[x] = sign_bound(args.k) * __bfloat162float(xnorm[(t & 1) * 128 + 32 * q + 8 * x + (lane >> 2)]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t *w = rbuf + c * 128 + 32 * h + 8 * j + 2 * (lane & 3);
                    const float w0 = __uint_as_float(w[0] & 0xFFFF0000u), w1 = __uint_as_float(w[1] & 0xFFFF0000u);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int i = (x >> 1) * 8 + 2 * j + (x & 1);
                        keep |= ((p[i].x > 0.f ? 1u : 0u) | (p[i].y > 0.f ? 2u : 0u)) << (2 * i);
                        check |= ((fabsf(p[i].x) < bound[x] * w0 ? 1u : 0u) | (fabsf(p[i].y) < bound[x] * w1 ? 2u : 0u)) << (2 * i);
                    }
                }
                for (unsigned who = __ballot_sync(0xffffffffu, check != 0); who; who &= who - 1) {
                    const int src = __ffs(who) - 1;
                    for (uint32_t left = __shfl_sync(0xffffffffu, check, src); left; left &= left - 1) {
                        const int bit = __ffs(left) - 1, i = bit >> 1;
                        const int r = 32 * q + 16 * (i >> 3) + 8 * (i & 1) + (src >> 2);
                        const int col = 32 * h + 8 * ((i >> 1) & 3) + 2 * (src & 3) + (bit & 1);
                        const uint2 xv = tile_quad(xbuf + (kHeld8 ? 0 : (t % XB) * TILE), r, lane), wv = tile_quad(wbuf + c * TILE, col, lane);
                        const float2 xa = two(xv.x), xb = two(xv.y), wa = two(wv.x), wb = two(wv.y);
                        double sum = (double)xa.x * wa.x + (double)xa.y * wa.y + (double)xb.x * wb.x + (double)xb.y * wb.y;
#pragma unroll
                        for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                        if (lane == src) keep = (keep & ~(1u << bit)) | (sum + (double)__uint_as_float(rbuf[c * 128 + col] << 16) > 0.0 ? 1u << bit : 0u);
                    }
                }
            }
            // One test for all of the warp's values: the four blocks below then overlap, and their matrix loads
            // and stores, which the whole warp does together, stand on one side of the branch.
            const bool share = !has_p || ACT == LIN_RELU || __all_sync(0xffffffffu, can_share(p));
            if (!share) {
                // Places outside the matrices are products with zeros, NaN where one met an infinity (and a NaN is never
                // shared): p is 0 there, so that with dy = 0 (TMA's fill) D is 0 too. (relu's D is 0 where p is not over 0.)
                const int cols_left = n_mine - (c * 128 + 32 * h), rows_left = (int)args.rows - (row0(t) + 32 * q);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (8 * ((i >> 1) & 3) >= cols_left || 16 * (i >> 3) + 8 * (i & 1) + (lane >> 2) >= rows_left)
                        p[i] = make_float2(0.f, 0.f);
                write_d<ACT, false>(p, keep, tile, 4 * (h & 1) + la_c, x7, dsum);
            } else write_d<ACT, true>(p, keep, tile, 4 * (h & 1) + la_c, x7, dsum);
#pragma unroll
            for (int cc = 0; cc < CHUNKS; ++cc)
                if (cc == c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dbs[cc][j] = __fadd2_rn(dbs[cc][j], dsum[j]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dready[db]);
            return true;
        };

        // dx of tile t: this worker's 32 rows x 32 columns.
        auto drain_dx = [&](int t) {
            if (!warp_wait(dxfull, (uint32_t)t & 1u, abort_flag, ctl, SITE_LBW | 12, t)) return false;
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32(lanebase + (uint32_t)(DX_COL + 32 * h), v);
            tmem_ld_wait_regs(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dxfree);
            const int col = 32 * h;
            if (kPair && !home) {
                if (t > 0 && !warp_wait_cluster(&sfree[pslot], (uint32_t)(t - 1) & 1u, abort_flag, ctl, SITE_LBW | 15, t)) return false;
                const uint32_t dst = map_to_rank(ob, rank ^ 1u) + lane * 16;
                const uint32_t bar = map_to_rank(&rfull[pslot], rank ^ 1u);
#pragma unroll
                for (int j = 0; j < 8; ++j) st_async_v4(dst + j * 512, bar, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                ++parts;
                return true;
            }
            if (kPair) {
                if (lane == 0) mbar_arrive_expect_tx(&rfull[pslot], 4096);
                ++parts;
                if (!warp_wait_cluster(&rfull[pslot], (uint32_t)t & 1u, abort_flag, ctl, SITE_LBW | 15, t)) return false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(ob + j * 512 + lane * 16);
                    v[4 * j] = __float_as_uint(__uint_as_float(v[4 * j]) + f.x);
                    v[4 * j + 1] = __float_as_uint(__uint_as_float(v[4 * j + 1]) + f.y);
                    v[4 * j + 2] = __float_as_uint(__uint_as_float(v[4 * j + 2]) + f.z);
                    v[4 * j + 3] = __float_as_uint(__uint_as_float(v[4 * j + 3]) + f.w);
                }
                __syncwarp();  // the block has been read: it now stages the result
                owes_room = true;
            }
            if (lane == 0) tma_store_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    o[x] = pack_bf16x2(__uint_as_float(v[8 * j + 2 * x]), __uint_as_float(v[8 * j + 2 * x + 1]));
                *reinterpret_cast<uint4 *>(ob + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && col < args.k && row0(t) + 32 * q < args.rows) {
                tma_store_3d(&tmDx, ob, col, row0(t) + 32 * q, 0);
                tma_store_commit();
            }
            return true;
        };

        const bool has_dx = args.has_dx != 0;
        if (ACT == LIN_RELU && !kHeld8 && my_tiles > 0) ok = write_norms(0);
        for (int t = 0; ok && t < my_tiles; ++t) {
            if (kHeld8) {
                // x first: p of the tile is then computed while dx of the tile before is drained.
                if (!(ok = convert(t))) break;
                if (has_dx && t > 0 && !(ok = drain_dx(t - 1))) break;
            }
            for (int c = 0; c < CHUNKS; ++c) {
                if (!(ok = make_d(t * CHUNKS + c))) break;
                if (!kHeld8 && c == 0 && has_dx && t > 0 && !(ok = drain_dx(t - 1))) break;
            }
            // The next tile's norms, so that its D need not wait for them.
            if (ACT == LIN_RELU && !kHeld8 && ok && t + 1 < my_tiles) ok = write_norms(t + 1);
        }
        if (ok && has_dx && my_tiles > 0) ok = drain_dx(my_tiles - 1);
        if (lane == 0) tma_store_wait_all<0>();
        if (kPair) {
            // How many parts were sent, so that after a timeout the receiver can let the last one land.
            if (!home && lane == 0) st_remote_u32(map_to_rank((const void *)&sent[pslot], rank ^ 1u), (uint32_t)parts);
            my_parts = parts;
        }
        // dW, once every product is done: lane = row of the 128, 32 columns of k.
        if (ok) ok = warp_wait(drain, 0, abort_flag, ctl, SITE_LBW | 13, 0);
        if (ok && args.has_dw) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                __syncwarp();
                uint32_t v[32];
                tmem_ld32(lanebase + (uint32_t)(128 * c + 32 * h), v);
                tmem_ld_wait_regs(v);
                const int rc = c * 128 + 32 * q + lane, r = n_first + rc;
                if (rc >= n_mine) continue;
                if (args.dw_out) {
                    __nv_bfloat16 *dst = args.dw_out + (size_t)r * args.k + 32 * h;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (32 * h + 8 * j < args.k) {
                            uint32_t o[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                o[x] = pack_bf16x2(__uint_as_float(v[8 * j + 2 * x]), __uint_as_float(v[8 * j + 2 * x + 1]));
                            *reinterpret_cast<uint4 *>(dst + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                } else {
                    float *dst = args.partial + ((size_t)team * args.n + r) * args.k + 32 * h;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (32 * h + 4 * j < args.k)
                            *reinterpret_cast<uint4 *>(dst + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // The sums over the teams. Here, not at the start: 147456 x 128 -> 128 with relu (without its norms) took 36.0 us
    // without the overlap, 35.4 so, and 37.1 with the sums' blocks waiting all the while.
    if (args.partial) next_kernel_may_start();
    if (kPair) {
        cluster_sync();  // the counts of parts sent are here
        if (warp >= 2 && (h >> 1) == (int)rank && lane == 0) {
            // At most one part can be under way: the sender waits for room. A complete pass has taken all.
            const int slot = 2 * q + (h & 1), n_sent = (int)sent[slot];
            if (n_sent > my_parts) mbar_arrive_expect_tx(&rfull[slot], 4096);
            if (n_sent > 0) wait_drain(&rfull[slot], (uint32_t)(n_sent - 1) & 1u, ctl.timeout_ns);
        }
        __syncthreads();
        cluster_sync();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
    if (!args.has_db) return;
    // db: each worker's lanes that share columns (lane % 4) are joined, then the four row quarters. The
    // tiles' memory is free by now.
    float *part = reinterpret_cast<float *>(dbuf);  // [4][128 CHUNKS]
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 s = dbs[c][j];
#pragma unroll
                for (int w = 4; w <= 16; w <<= 1) {
                    s.x += __shfl_xor_sync(0xffffffffu, s.x, w);
                    s.y += __shfl_xor_sync(0xffffffffu, s.y, w);
                }
                if (lane < 4) *reinterpret_cast<float2 *>(part + q * 128 * CHUNKS + c * 128 + 32 * h + 8 * j + 2 * lane) = s;
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_mine; i += THREADS) {
        const float s = (part[i] + part[128 * CHUNKS + i]) + (part[256 * CHUNKS + i] + part[384 * CHUNKS + i]);
        if (args.db_out) args.db_out[n_first + i] = __float2bfloat16_rn(s);
        else args.sums[(size_t)team * args.n + n_first + i] = s;
    }
}

namespace {
template <int CHUNKS, bool kPair, bool kHeld8, int ACT>
cudaError_t allow() {
    return cudaFuncSetAttribute(linear_bwd_kernel<CHUNKS, kPair, kHeld8, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lb::SMEM);
}
template <int CHUNKS, bool kPair, bool kHeld8>
cudaError_t allow_acts() {
    cudaError_t e;
    if ((e = allow<CHUNKS, kPair, kHeld8, LIN_NONE>()) || (e = allow<CHUNKS, kPair, kHeld8, LIN_RELU>()) ||
        (e = allow<CHUNKS, kPair, kHeld8, LIN_SIGMOID>()))
        return e;
    return allow<CHUNKS, kPair, kHeld8, LIN_SILU>();
}
template <int CHUNKS, bool kPair, bool kHeld8, int ACT>
cudaError_t go(const LinearBwdMaps &m, const LinearBwdArgs &a, int teams, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kPair ? 2 * teams : teams));
    cfg.blockDim = dim3(lb::THREADS);
    cfg.dynamicSmemBytes = lb::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = kPair ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linear_bwd_kernel<CHUNKS, kPair, kHeld8, ACT>, m.x, m.w, m.dy, m.dx, a);
}
template <int CHUNKS, bool kPair, bool kHeld8>
cudaError_t go_act(const LinearBwdMaps &m, const LinearBwdArgs &a, int teams, cudaStream_t s) {
    if (a.act == LIN_NONE) return go<CHUNKS, kPair, kHeld8, LIN_NONE>(m, a, teams, s);
    if (a.act == LIN_RELU) return go<CHUNKS, kPair, kHeld8, LIN_RELU>(m, a, teams, s);
    if (a.act == LIN_SIGMOID) return go<CHUNKS, kPair, kHeld8, LIN_SIGMOID>(m, a, teams, s);
    return go<CHUNKS, kPair, kHeld8, LIN_SILU>(m, a, teams, s);
}
}  // namespace

cudaError_t linear_bwd_setup() {
    cudaError_t e;
    if ((e = allow_acts<1, false, false>()) || (e = allow_acts<1, false, true>()) || (e = allow_acts<2, false, false>()) ||
        (e = allow_acts<2, false, true>()) || (e = allow_acts<2, true, false>()))
        return e;
    return allow_acts<2, true, true>();
}

cudaError_t launch_linear_bwd(const LinearBwdMaps &m, const LinearBwdArgs &a, bool held8, int teams, cudaStream_t s) {
    if (a.n > 256) return held8 ? go_act<2, true, true>(m, a, teams, s) : go_act<2, true, false>(m, a, teams, s);
    if (a.n > 128) return held8 ? go_act<2, false, true>(m, a, teams, s) : go_act<2, false, false>(m, a, teams, s);
    return held8 ? go_act<1, false, true>(m, a, teams, s) : go_act<1, false, false>(m, a, teams, s);
}

}  // namespace trimul
