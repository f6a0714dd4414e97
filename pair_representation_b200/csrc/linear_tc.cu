// linear_tc.cu - a linear layer with its epilogue, and the three products of its
// backward, on tcgen05 tensor cores.
//
//   LIN_FWD   Y = act(A B^T + bias) + E           (E: the residual, optional)
//   LIN_GRAD  Y = E * act'(A B^T + bias)          (E: dL/dy; column sums of Y before
//                                                  rounding give dL/dbias)
//   LIN_WG    Y_s = A_s B_s^T in fp32             (split s of the contraction; with an
//                                                  optional column of ones: row sums of A)
//
// A(m, k) and B(n, k) are bf16, each K-major ([rows][k]) or MN-major ([k][rows]): the
// forward reads x and W K-major, dx = D W reads W MN-major, dW = D^T x reads both
// MN-major with the rows of the batch as the contracted index.
//
// LIN_GRAD rounds Y to bf16, the products' operand type: dx and dW are then off by 0.0024 of their norm, against 0.0017
// of their own rounding alone (2^-8 at most for each).
//
// What bounds it: at the widths of a pair or atom representation (128 to 512 channels)
// a row moves 2 (k + n) bytes for 2 k n operations, under the card's ratio of about 260
// operations per byte, so the batch's rows are streamed once and everything else stays
// on chip. A CTA owns one column tile (BN wide) and walks down the row tiles: with
// kResident its slab of B (at most 64 KB) is loaded once and stays in shared memory;
// only A tiles travel, through a ring. Wider contractions stream A and B together, over
// tiles of 256 rows (HIGH = 2) where there are rows enough.
// The accumulator is double-buffered in tensor memory (2 x BN columns) and drained by
// sixteen warps, each storing its own 32 x 32 blocks by TMA, so the drain of one tile
// overlaps the loads and MMAs of the next. E blocks arrive by TMA in the very buffer
// the result leaves from, one block ahead.
//
// Measured, call after call on the same inputs (and one call on inputs cold in L2): 147456 x 512 -> 128 with a
// residual 38 us, 6.0 TB/s (48); 589824 x 128 -> 512 133 us, 5.7 TB/s (137), with silu 160 (170) at 1965 MHz and
// 190 at the 1650 MHz that the power cap leaves in long runs: the drain warps then issue at 54 % of their slots and
// wait on exponentials and shared memory.
// Sixteen warps on blocks of 32 columns (eight on 64 columns: 188 us).
//
// Every wait is bounded; on a timeout the CTA lets its copies land and returns.
#include "kernels.h"
#include "linear_act.cuh"

namespace trimul {
namespace lin {
constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BM * BK * 2;        // 16 KB
constexpr int EPI_WARPS = 16;               // four per tensor-memory lane quarter
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr int WBUF = 4096;                  // a drain warp's: two blocks of 32 rows x 32 bf16, or one of fp32
constexpr int OUT_BYTES = EPI_WARPS * WBUF;
constexpr int BIAS_BYTES = EPI_WARPS * 64 * 4;  // each drain warp's own copy of its columns' bias
constexpr int ONES_BYTES = 16 * BK * 2;     // 16 rows of ones (LIN_WG), or (LIN_GRAD) the norms of 256 rows of W and 2 x 128 of x
constexpr int BAR_BYTES = 512;
constexpr int RES_BYTES = 65536;            // resident slab of B
constexpr int TMEM_COLS = 512;
constexpr int ONES_COL = 256;               // LIN_WG (BN = 128): accumulators of the ones column

__host__ __device__ constexpr int stages(int bn, bool res, int high = 1) { return res ? 5 : bn == 256 || high == 2 ? 3 : 4; }
__host__ __device__ constexpr int stage_bytes(int bn, bool res, int high = 1) {
    return high * A_BYTES + (res ? 0 : bn * BK * 2);
}
__host__ __device__ constexpr size_t smem(int bn, bool res, int high = 1) {
    return 1024 + (size_t)stages(bn, res, high) * stage_bytes(bn, res, high) + (res ? RES_BYTES : 0) + OUT_BYTES + BIAS_BYTES +
           ONES_BYTES + BAR_BYTES;
}
static_assert(smem(256, false) <= 232448 && smem(256, true) <= 232448 && smem(128, false) <= 232448 &&
                  smem(128, false, 2) <= 232448,
              "shared memory");

// The tiles of one CTA, in the order every role of the CTA visits them.
template <int MODE>
struct Tiles {
    const LinearArgs &a;
    int ct, rt, kb0, kb1, split;  // column tile, row tile, K blocks, split of the contraction
    long long u;
    __device__ explicit Tiles(const LinearArgs &args) : a(args), ct(0), rt(-1), kb0(0), kb1(args.kblocks), split(0), u(-1) {}
    __device__ bool next() {
        if (MODE == LIN_WG) {
            u = u < 0 ? (long long)blockIdx.x : u + gridDim.x;
            const int per = a.row_tiles * a.col_tiles;
            if (u >= (long long)per * a.splits) return false;
            split = (int)(u / per);
            const int r = (int)(u - (long long)split * per);
            rt = r / a.col_tiles;
            ct = r - rt * a.col_tiles;
            kb0 = split * a.kb_per_split;
            kb1 = min(a.kblocks, kb0 + a.kb_per_split);
            return true;
        }
        if (rt < 0) {
            ct = (int)blockIdx.x % a.col_tiles;
            rt = (int)blockIdx.x / a.col_tiles;
        } else {
            rt += a.groups;
        }
        return rt < a.row_tiles;
    }
};
}  // namespace lin

namespace {

// 32 columns of one accumulator row (bias added): activation, residual (or the gradient), packed
// to bf16 into the row's 64 swizzled bytes. In LIN_GRAD p receives the unrounded values.
template <int MODE, int ACT, bool kShare, bool kE>
__device__ __forceinline__ void finish_columns(float2 (&p)[16], uint8_t *row, int swz) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(row + ((c ^ swz) << 4));
        uint4 ev = make_uint4(0u, 0u, 0u, 0u);
        if (kE) ev = *at;
        const uint32_t ew[4] = {ev.x, ev.y, ev.z, ev.w};
        uint32_t o[4];
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            float2 e[2], y[2] = {p[4 * c + t], p[4 * c + t + 1]};
#pragma unroll
            for (int u = 0; u < 2; ++u)
                e[u] = make_float2(__uint_as_float(ew[t + u] << 16), __uint_as_float(ew[t + u] & 0xFFFF0000u));
            if (MODE == LIN_GRAD) act_grad4<ACT, kShare>(y, e);
            else act_fwd4<ACT, kShare>(y);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (MODE == LIN_FWD && kE) y[u] = __fadd2_rn(y[u], e[u]);
                if (MODE == LIN_GRAD) p[4 * c + t + u] = y[u];
                o[t + u] = pack_bf16x2(y[u].x, y[u].y);
            }
        }
        *at = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int MODE, int ACT, bool kE>
__device__ __forceinline__ void finish_row(float2 (&p)[16], uint8_t *row, int swz) {
    if (ACT == LIN_NONE || ACT == LIN_RELU || can_share(p)) finish_columns<MODE, ACT, true, kE>(p, row, swz);
    else finish_columns<MODE, ACT, false, kE>(p, row, swz);
}

template <int MODE, bool kE>
__device__ __forceinline__ void finish(int act, float2 (&p)[16], uint8_t *row, int swz) {
    if (act == LIN_NONE) finish_row<MODE, LIN_NONE, kE>(p, row, swz);
    else if (MODE == LIN_FWD && act == LIN_RELU) finish_row<MODE, LIN_RELU, kE>(p, row, swz);
    else if (act == LIN_SIGMOID) finish_row<MODE, LIN_SIGMOID, kE>(p, row, swz);
    else finish_row<MODE, LIN_SILU, kE>(p, row, swz);
}

// Norms of eight rows of a matrix [rows][K] from row `first`, 0 past the last: lane l returns that of row
// first + (l >> 2).
__device__ __forceinline__ float norms_of_8(const __nv_bfloat16 *m, int first, int rows, int K, int lane) {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 8 * lane; k < K; k += 256) {  // K is a multiple of 8
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = first + i < rows ? *reinterpret_cast<const uint4 *>(m + (size_t)(first + i) * K + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = add_squares(add_squares(add_squares(add_squares(s[i], v[i].x), v[i].y), v[i].z), v[i].w);
    }
    return norm_of(sums_of_8(s, lane));
}

// The products of two bf16 pairs, exact in fp32, in 64 bits.
__device__ __forceinline__ double pair_product(uint32_t x, uint32_t w) {
    return (double)(__uint_as_float(x << 16) * __uint_as_float(w << 16)) +
           (double)(__uint_as_float(x & 0xFFFF0000u) * __uint_as_float(w & 0xFFFF0000u));
}

// relu's gradient of one accumulator row: keep E where p > 0. Where p is under the bound of its rounding
// (linear_act.cuh; `bound` has the row's norm of x in it, wnorm those of W), the warp takes the row's product
// again, one place at a time.
__device__ __forceinline__ void finish_row_relu_grad(float2 (&v)[16], const float *bias, uint8_t *row, int swz,
                                                     const LinearArgs &a, int r, int col0, int lane, float bound,
                                                     const float *wnorm) {
    uint32_t keep = 0, check = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float p = j & 1 ? v[j >> 1].y : v[j >> 1].x;
        keep |= (uint32_t)(p > 0.f) << j;
        check |= (uint32_t)(fabsf(p) < bound * wnorm[j]) << j;
    }
    for (unsigned who = __ballot_sync(0xffffffffu, check != 0); who; who &= who - 1) {
        const int src = __ffs(who) - 1;
        const __nv_bfloat16 *xr = a.x + (size_t)(r - lane + src) * a.K;
        for (uint32_t left = __shfl_sync(0xffffffffu, check, src); left; left &= left - 1) {
            const int j = __ffs(left) - 1;
            const __nv_bfloat16 *wr = a.w + (size_t)(col0 + j) * a.K;
            double sum = 0.0;
#pragma unroll 4
            for (int k = 8 * lane; k < a.K; k += 256) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xr + k), w = *reinterpret_cast<const uint4 *>(wr + k);
                sum += (pair_product(x.x, w.x) + pair_product(x.y, w.y)) + (pair_product(x.z, w.z) + pair_product(x.w, w.w));
            }
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            if (lane == src) keep = (keep & ~(1u << j)) | (uint32_t)(sum + (double)bias[j] > 0.0) << j;
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(row + ((c ^ swz) << 4));
        const uint4 e = *at;
        uint32_t o[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t two = keep >> (8 * c + 2 * t);
            o[t] &= (two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u);
            v[4 * c + t] = make_float2(__uint_as_float(o[t] << 16), __uint_as_float(o[t] & 0xFFFF0000u));
        }
        *at = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Sums of 32 columns over the warp's 32 lanes: lane l returns column l's sum. Each step halves
// the columns a lane holds (lanes with the bit set keep the upper half): 31 shuffles in all,
// and the order of the additions is fixed.
__device__ __forceinline__ float column_sum32(const float2 *v, int lane) {
    float s[16];
    const bool hi = (lane & 16) != 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float lo = i & 1 ? v[i >> 1].y : v[i >> 1].x, up = i & 1 ? v[(i >> 1) + 8].y : v[(i >> 1) + 8].x;
        const float keep = hi ? up : lo, give = hi ? lo : up;
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? s[i + w] : s[i], give = up ? s[i] : s[i + w];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    return s[0];
}

}  // namespace

template <int BN, bool kResident, int MODE, int HIGH>
__global__ void __launch_bounds__(lin::THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmY,
                     const LinearArgs args) {
    using namespace lin;
    static_assert(HIGH == 1 || (BN <= 128 && MODE == LIN_FWD), "a drain warp's chunks are then of the same columns");
    constexpr int STAGES = stages(BN, kResident, HIGH), STAGE_BYTES = stage_bytes(BN, kResident, HIGH);
    constexpr int B_BYTES = BN * BK * 2;
    constexpr int CHUNK = 32;                                      // accumulator columns per stored block
    constexpr int WIDE = BN / CHUNK;                               // of a row of the tile
    constexpr int CHUNKS = HIGH * WIDE, MINE = (CHUNKS + 3) / 4;  // of a tile, and of them a drain warp's (at most)
    constexpr int COLS = (WIDE + 3) / 4;                           // a drain warp's chunks of a row
    constexpr int BLOCK = MODE == LIN_WG ? 4096 : 2048, BUFS = WBUF / BLOCK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem;
    uint8_t *bres = ring + STAGES * STAGE_BYTES;
    uint8_t *outbuf = bres + (kResident ? RES_BYTES : 0);
    uint8_t *ones = outbuf + OUT_BYTES;
    float *biasbuf = reinterpret_cast<float *>(ones + ONES_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(biasbuf) + BIAS_BYTES);
    uint64_t *full = bars;                  // [STAGES] operands landed
    uint64_t *empty = bars + STAGES;        // [STAGES] MMAs reading the stage are done
    uint64_t *bfull = bars + 2 * STAGES;    // the resident slab landed
    uint64_t *tfull = bfull + 1;            // [2] accumulator complete
    uint64_t *tempty = tfull + 2;           // [2] accumulator drained (EPI_WARPS arrivals)
    uint64_t *efull = tempty + 2;           // [EPI_WARPS][2] E block landed
    uint64_t *drain = efull + 2 * EPI_WARPS;
    uint64_t *nready = drain + 1;           // relu's LIN_GRAD: norms of a tile's rows written (EPI_WARPS arrivals)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(nready + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KernelCtl &ctl = args.ctl;
    const bool with_ones = MODE == LIN_WG && (args.sums != nullptr || args.db_out != nullptr);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(bfull, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], EPI_WARPS);
        }
        for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(&efull[i], 1);
        mbar_init(drain, 1);
        mbar_init(nready, EPI_WARPS);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmY);
        if (MODE != LIN_WG && args.has_e) tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    if (with_ones) {
        for (int i = threadIdx.x; i < ONES_BYTES / 4; i += THREADS) reinterpret_cast<uint32_t *>(ones)[i] = 0x3F803F80u;
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto load_b = [&](uint8_t *dst, uint64_t *bar, int k0, int n0) {
        if (!args.b_mn) {
            tma_load_3d(dst, &tmB, bar, k0, n0, 0);
        } else {
#pragma unroll
            for (int h = 0; h < BN / 64; ++h) tma_load_3d(dst + h * (BK * 128), &tmB, bar, n0 + 64 * h, k0, 0);
        }
    };
    if (kResident && threadIdx.x == 0) {  // W: no kernel of the call writes it
        const int n0 = ((int)blockIdx.x % args.col_tiles) * BN;
        mbar_arrive_expect_tx(bfull, (uint32_t)(args.kblocks * B_BYTES));
        for (int kb = 0; kb < args.kblocks; ++kb) load_b(bres + kb * B_BYTES, bfull, kb * BK, n0);
    }
    if (args.more) next_kernel_may_start();
    wait_for_kernel_before();
    if (args.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *ctl.status = DeviceStatus{0, 0, 0, 0};

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            uint32_t issued = 0;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            Tiles<MODE> t(args);
            while (ok && t.next()) {
                const int m0 = t.rt * (HIGH * BM), n0 = t.ct * BN;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!wait_bounded(&empty[stage], phase ^ 1u, abort_flag, ctl, SITE_LIN | 2, t.rt)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = ring + stage * STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
                    const int k0 = kb * BK;
                    if (!args.a_mn) {
#pragma unroll
                        for (int r = 0; r < HIGH; ++r) tma_load_3d(sa + r * A_BYTES, &tmA, &full[stage], k0, m0 + r * BM, 0);
                    } else {
                        tma_load_3d(sa, &tmA, &full[stage], m0, k0, 0);
                        tma_load_3d(sa + BK * 128, &tmA, &full[stage], m0 + 64, k0, 0);
                    }
                    if (!kResident) load_b(sa + HIGH * A_BYTES, &full[stage], k0, n0);
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // No copy may be in flight when the CTA leaves.
            for (int s = 0; s < STAGES; ++s) {
                const uint32_t n = issued / STAGES + ((uint32_t)s < issued % STAGES ? 1u : 0u);
                if (n > 0) wait_drain(&full[s], (n - 1) & 1u, ctl.timeout_ns);
            }
            if (kResident) wait_drain(bfull, 0, ctl.timeout_ns);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            const uint32_t idesc = idesc_bf16(BM, BN, args.a_mn, args.b_mn);
            const uint32_t idesc_ones = idesc_bf16(BM, 16, args.a_mn, 0);
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            bool ok = !kResident || wait_bounded(bfull, 0, abort_flag, ctl, SITE_LIN | 3, 0);
            Tiles<MODE> t(args);
            while (ok && t.next()) {
                const int acc = lt & 1;
                if (!wait_bounded(&tempty[acc], ((uint32_t)(lt >> 1) & 1u) ^ 1u, abort_flag, ctl, SITE_LIN | 4, t.rt)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * HIGH * BN);
                const bool sum_rows = with_ones && t.ct == 0;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!wait_bounded(&full[stage], phase, abort_flag, ctl, SITE_LIN | 5, t.rt)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + stage * STAGE_BYTES);
                    const uint32_t sb = kResident ? smem_u32(bres + kb * B_BYTES) : sa + HIGH * A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        const uint64_t ad = args.a_mn ? sdesc_sw128(sa + kk * 2048, BK * 128, 1024)
                                                      : sdesc_sw128(sa + kk * 32, 16, 1024);
                        const uint64_t bd = args.b_mn ? sdesc_sw128(sb + kk * 2048, BK * 128, 1024)
                                                      : sdesc_sw128(sb + kk * 32, 16, 1024);
                        const uint32_t more = (kb != t.kb0 || kk != 0) ? 1u : 0u;
                        mma_bf16(d, ad, bd, idesc, more);
                        if (HIGH == 2)
                            mma_bf16(d + BN, sdesc_sw128(sa + A_BYTES + kk * 32, 16, 1024), bd, idesc, more);
                        if (sum_rows)
                            mma_bf16(tmem + ONES_COL + 16 * acc, ad, sdesc_sw128(smem_u32(ones) + kk * 32, 16, 1024),
                                     idesc_ones, more);
                    }
                    mma_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit(&tfull[acc]);
                ++lt;
            }
            mma_commit(drain);
            wait_drain(drain, 0, ctl.timeout_ns);
        }
    } else {
        // ---------------- drain warps 2..17 ----------------
        // Warp (q, h): accumulator rows 32 q .. 32 q + 31, chunks h and h + 4 of each tile (HIGH = 2: the
        // second of them the same columns of the lower 128 rows). Block n of this warp (counted over all its tiles) goes through buffer n % BUFS.
        const int ew = warp - 2, q = warp & 3, h = ew >> 2;
        uint8_t *wbuf = outbuf + ew * WBUF;
        uint64_t *ebar = efull + 2 * ew;
        float *mybias = biasbuf + ew * 64;
        const uint32_t lanebase = tmem + ((uint32_t)(q * 32) << 16);
        const bool has_e = MODE != LIN_WG && args.has_e;
        float colsum[COLS];
        int nst = 0, nload = 0, lt = 0;

        // Iterator over this warp's blocks, for the E loads that run one block ahead.
        Tiles<MODE> ahead(args);
        int ahead_c = CHUNKS;
        bool ahead_ok = has_e;
        auto load_next_e = [&]() {
            if (!ahead_ok) return;
            for (;;) {
                ahead_c += 4;
                if (ahead_c >= CHUNKS) {
                    if (!ahead.next()) {
                        ahead_ok = false;
                        return;
                    }
                    ahead_c = h;
                    if (ahead_c >= CHUNKS) continue;
                }
                const int col = ahead.ct * BN + ahead_c % WIDE * CHUNK, row = (ahead.rt * HIGH + ahead_c / WIDE) * BM + 32 * q;
                if (col < args.N && row < args.M) {
                    if (lane == 0) {
                        tma_store_wait_read<0>();  // the block that last left from this buffer has been read
                        mbar_arrive_expect_tx(&ebar[nload & 1], BLOCK);
                        tma_load_3d(wbuf + (nload & 1) * BLOCK, &tmE, &ebar[nload & 1], col, row, 0);
                    }
                    ++nload;
                    return;
                }
            }
        };
        load_next_e();
        if (MODE != LIN_WG) {
            const int n0 = ((int)blockIdx.x % args.col_tiles) * BN;
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                const int col = n0 + (HIGH == 2 ? h % WIDE : h + 4 * i) * 32 + lane;
                mybias[32 * i + lane] = (args.bias && col < args.N) ? __bfloat162float(args.bias[col]) : 0.f;
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < COLS; ++i) colsum[i] = 0.f;
        // relu's gradient: the norms that bound p's rounding, of W's rows of this column tile and of each tile's rows of
        // x, eight rows a warp, read again through L2 while the products run. A tile's go to the buffer of the tile before
        // the last, which every warp has left when all have written the last one's.
        const bool relu_grad = MODE == LIN_GRAD && args.act == LIN_RELU;
        float *wnorm = reinterpret_cast<float *>(ones), *xnorm = wnorm + 256;
        if (relu_grad) {
            const int n0 = ((int)blockIdx.x % args.col_tiles) * BN;
            for (int j = 8 * ew; j < BN; j += 8 * EPI_WARPS) {
                const float norm = norms_of_8(args.w, n0 + j, args.N, args.K, lane);
                if ((lane & 3) == 0) wnorm[j + (lane >> 2)] = norm;
            }
        }
        bool ok = true;
        Tiles<MODE> t(args);
        while (ok && t.next()) {
            const int acc = lt & 1;
            if (relu_grad) {
                const float norm = norms_of_8(args.x, t.rt * BM + 8 * ew, args.M, args.K, lane);
                if ((lane & 3) == 0) xnorm[acc * BM + 8 * ew + (lane >> 2)] = norm;
                __syncwarp();
                if (lane == 0) mbar_arrive(nready);
            }
            if (!warp_wait(&tfull[acc], (uint32_t)(lt >> 1) & 1u, abort_flag, ctl, SITE_LIN | 6, t.rt)) break;
            tc_fence_after();
            if (relu_grad && !warp_wait(nready, (uint32_t)lt & 1u, abort_flag, ctl, SITE_LIN | 8, t.rt)) break;
            const int top = t.rt * (HIGH * BM) + 32 * q;
#pragma unroll
            for (int ci = 0; ci < MINE; ++ci) {
                const int ch = h + 4 * ci, wide = HIGH == 2 ? ch % WIDE : ch, col = t.ct * BN + wide * CHUNK;
                const int row0 = top + (HIGH == 2 ? ch / WIDE * BM : 0), mine = HIGH == 2 ? 0 : ci;
                if (ch >= CHUNKS || row0 >= args.M || col >= args.N) continue;
                uint8_t *ob = wbuf + (nst % BUFS) * BLOCK;
                const uint32_t taddr = lanebase + (uint32_t)(acc * HIGH * BN + ch * CHUNK);
                uint32_t v[32];
                tmem_ld32(taddr, v);
                if (has_e) {
                    load_next_e();
                    if (!(ok = warp_wait(&ebar[nst & 1], (uint32_t)(nst >> 1) & 1u, abort_flag, ctl, SITE_LIN | 7, t.rt)))
                        break;
                } else if (lane == 0) {
                    tma_store_wait_read<BUFS - 1>();
                }
                __syncwarp();
                tmem_ld_wait_regs(v);
                if constexpr (MODE == LIN_WG) {
                    if (args.out_bf16) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                o[x] = pack_bf16x2(__uint_as_float(v[8 * c + 2 * x]), __uint_as_float(v[8 * c + 2 * x + 1]));
                            *reinterpret_cast<uint4 *>(ob + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4 *>(ob + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                                make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                    }
                } else {
                    const float *bias = mybias + 32 * mine;
                    float2 p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        p[j] = __fadd2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])),
                                          *reinterpret_cast<const float2 *>(bias + 2 * j));
                    // Rows past the last are zeros times W, NaN where it holds an infinity: kept out of the column sums.
                    if (MODE == LIN_GRAD && row0 + lane >= args.M) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) p[j] = make_float2(0.f, 0.f);
                    }
                    uint8_t *row = ob + lane * 64;
                    const int swz = (lane >> 1) & 3;
                    if (MODE == LIN_GRAD && args.act == LIN_RELU)
                        finish_row_relu_grad(p, bias, row, swz, args, row0 + lane, col, lane,
                                             sign_bound(args.K) * xnorm[acc * BM + 32 * q + lane], wnorm + ch * CHUNK);
                    else if (MODE == LIN_GRAD || has_e)
                        finish<MODE, true>(args.act, p, row, swz);
                    else
                        finish<MODE, false>(args.act, p, row, swz);
                    if (MODE == LIN_GRAD && args.sums != nullptr) colsum[mine] += column_sum32(p, lane);
                }
                ++nst;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmY, ob, col, row0, MODE == LIN_WG ? t.split : 0);
                    tma_store_commit();
                }
            }
            if (!ok) break;
            if (with_ones && t.ct == 0 && h == 0) {
                uint32_t v[16];
                tmem_ld16(lanebase + (uint32_t)(ONES_COL + 16 * acc), v);
                tmem_ld_wait_regs(v);
                const int row = top + lane;
                if (row < args.M) {
                    if (args.db_out) args.db_out[row] = __float2bfloat16_rn(__uint_as_float(v[0]));
                    else args.sums[(size_t)t.split * args.M + row] = __uint_as_float(v[0]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
            ++lt;
        }
        if (MODE == LIN_GRAD && args.sums != nullptr) {
            float *dst = args.sums + (size_t)(((int)blockIdx.x / args.col_tiles) * 4 + q) * args.N;
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                const int ch = h + 4 * i, col = ((int)blockIdx.x % args.col_tiles) * BN + ch * 32 + lane;
                if (ch < WIDE && col < args.N) dst[col] = colsum[i];
            }
        }
        // E blocks still in flight (only after a timeout: a complete pass consumed them all).
        for (int n = nst; n < nload; ++n) wait_drain(&ebar[n & 1], (uint32_t)(n >> 1) & 1u, ctl.timeout_ns);
        if (lane == 0) tma_store_wait_all<0>();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
    if (MODE == LIN_GRAD && args.db_out != nullptr) {
        // The only CTA of its columns: the four quarters' sums (written before the barrier above) give db.
        const int n0 = ((int)blockIdx.x % args.col_tiles) * BN;
        for (int i = threadIdx.x; i < BN && n0 + i < args.N; i += THREADS) {
            const float *sum = args.sums + n0 + i;
            args.db_out[n0 + i] = __float2bfloat16_rn((sum[0] + sum[args.N]) + (sum[2 * (size_t)args.N] + sum[3 * (size_t)args.N]));
        }
    }
}

// ---------------------------------------------------------------------------
// Sums of the split products and of the column-sum partials, rounded once to bf16.
// dw[i] = sum_s partial[s][i]; db[j] = sum_s sums[s][j]. A warp takes 32 places and at most
// ten partials of them at a time, all in flight at once: up to ten partials need one warp, up to
// 148 a block's sixteen, whose sums are joined in shared memory in order: the result does not
// depend on the launch. Bound by the latency of reading the partials where there are many, by
// their bytes where there are few.
// ---------------------------------------------------------------------------
namespace {

constexpr int kReduceWarps = 16, kReduceLoads = 10;

__device__ __forceinline__ void add4(float4 &s, const float4 &v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
}

__global__ void __launch_bounds__(kReduceWarps * 32) linear_reduce_kernel(const LinearReduceArgs a) {
    __shared__ float4 part[kReduceWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool weight = (int)blockIdx.x < a.weight_blocks;
    // `join` warps share their places, each with every join-th partial.
    const int join = weight ? a.join : kReduceWarps, first = warp & (join - 1);
    const long long i = ((long long)blockIdx.x * (kReduceWarps / join) + warp / join) * 32 + lane;  // four values of dw
    const long long quads = a.count >> 2;  // n k is a multiple of 64
    const int j = ((int)blockIdx.x - a.weight_blocks) * 32 + lane;
    wait_for_kernel_before();
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 s = zero, v[kReduceLoads];
    if (weight) {
        const float4 *p = reinterpret_cast<const float4 *>(a.partial) + i;
        for (int k0 = first; k0 < a.splits; k0 += join * kReduceLoads) {
#pragma unroll
            for (int u = 0; u < kReduceLoads; ++u) {
                const int k = k0 + u * join;
                v[u] = i < quads && k < a.splits ? __ldcs(p + (size_t)k * quads) : zero;
            }
#pragma unroll
            for (int u = 0; u < kReduceLoads; ++u) add4(s, v[u]);
        }
    } else {
        for (int k0 = first; k0 < a.sum_rows; k0 += join * kReduceLoads) {
#pragma unroll
            for (int u = 0; u < kReduceLoads; ++u) {
                const int k = k0 + u * join;
                v[u].x = j < a.n && k < a.sum_rows ? a.sums[(size_t)k * a.n + j] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kReduceLoads; ++u) s.x += v[u].x;
        }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (first != 0) return;
    for (int k = 1; k < join; ++k) add4(s, part[warp + k][lane]);
    if (weight) {
        if (i < quads) reinterpret_cast<uint2 *>(a.dw)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    } else {
        if (j < a.n) a.db[j] = __float2bfloat16_rn(s.x);
    }
}

}  // namespace

namespace {
// A launch whose kernel may start while the one before it in the stream still runs (`after`).
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    Launch(int grid, int threads, size_t smem, bool after, cudaStream_t s) {
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = after ? 1 : 0;
    }
};
}  // namespace

cudaError_t launch_linear_reduce(LinearReduceArgs a, bool after, cudaStream_t s) {
    a.join = 1;
    while (a.join < kReduceWarps && a.join * kReduceLoads < a.splits) a.join *= 2;
    const long long places = 32 * (kReduceWarps / a.join);  // of a block, four values each
    a.weight_blocks = a.dw ? (int)((a.count / 4 + places - 1) / places) : 0;
    const int grid = a.weight_blocks + (a.db ? (a.n + 31) / 32 : 0);
    if (grid == 0) return cudaSuccess;
    const Launch l(grid, kReduceWarps * 32, 0, after, s);
    return cudaLaunchKernelEx(&l.cfg, linear_reduce_kernel, a);
}

bool linear_resident(int bn, int kblocks) { return (long long)kblocks * bn * lin::BK * 2 <= lin::RES_BYTES; }

namespace {
template <int BN, bool RES, int MODE, int HIGH = 1>
cudaError_t allow() {
    return cudaFuncSetAttribute(linear_tc_kernel<BN, RES, MODE, HIGH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lin::smem(BN, RES, HIGH));
}
template <int BN, bool RES, int MODE, int HIGH = 1>
cudaError_t go(const LinearMaps &m, const LinearArgs &a, int grid, bool after, cudaStream_t s) {
    const Launch l(grid, lin::THREADS, lin::smem(BN, RES, HIGH), after, s);
    return cudaLaunchKernelEx(&l.cfg, linear_tc_kernel<BN, RES, MODE, HIGH>, m.a, m.b, m.e, m.y, a);
}
template <int MODE>
cudaError_t pick(const LinearMaps &m, const LinearArgs &a, int bn, int grid, bool after, cudaStream_t s) {
    const bool res = linear_resident(bn, a.kblocks);
    if (MODE == LIN_FWD && a.high == 2)
        return bn == 64 ? go<64, false, LIN_FWD, 2>(m, a, grid, after, s) : go<128, false, LIN_FWD, 2>(m, a, grid, after, s);
    if (bn == 64) return res ? go<64, true, MODE>(m, a, grid, after, s) : go<64, false, MODE>(m, a, grid, after, s);
    if (bn == 128) return res ? go<128, true, MODE>(m, a, grid, after, s) : go<128, false, MODE>(m, a, grid, after, s);
    return res ? go<256, true, MODE>(m, a, grid, after, s) : go<256, false, MODE>(m, a, grid, after, s);
}
}  // namespace

cudaError_t linear_tc_setup() {
    cudaError_t e;
    if ((e = allow<64, true, LIN_FWD>()) || (e = allow<64, false, LIN_FWD>()) || (e = allow<128, true, LIN_FWD>()) ||
        (e = allow<128, false, LIN_FWD>()) || (e = allow<256, true, LIN_FWD>()) || (e = allow<256, false, LIN_FWD>()) ||
        (e = allow<64, true, LIN_GRAD>()) || (e = allow<64, false, LIN_GRAD>()) || (e = allow<128, true, LIN_GRAD>()) ||
        (e = allow<128, false, LIN_GRAD>()) || (e = allow<256, true, LIN_GRAD>()) ||
        (e = allow<256, false, LIN_GRAD>()) || (e = allow<64, false, LIN_FWD, 2>()) || (e = allow<128, false, LIN_FWD, 2>()))
        return e;
    return allow<128, false, LIN_WG>();
}

cudaError_t launch_linear_tc(const LinearMaps &m, const LinearArgs &a, int mode, int bn, int grid, bool after, cudaStream_t s) {
    if (mode == LIN_WG) return go<128, false, LIN_WG>(m, a, grid, after, s);
    return mode == LIN_GRAD ? pick<LIN_GRAD>(m, a, bn, grid, after, s) : pick<LIN_FWD>(m, a, bn, grid, after, s);
}

}  // namespace trimul
