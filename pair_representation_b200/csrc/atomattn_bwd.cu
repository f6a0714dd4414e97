// atomattn_bwd.cu - gradients of sequence-local atom attention (include/atomattn.h).
//
// For one batch element and head, window w (queries 32w .., key slots 32w - 48 ..):
//   P = softmax over the valid slots of q k^T / sqrt(32) + bias     (recomputed)
//   dP = dO v^T,  delta_i = sum_s P_is dP_is,  dS = P (dP - delta)
//   dq = dS k / sqrt(32),  dk += dS^T q / sqrt(32),  dv += P^T dO,  dbias = dS
//
// A key atom takes part in four consecutive windows. Keys are taken in groups of 32
// (group g: atoms 32g - 48 .. 32g - 17); window w holds groups w .. w + 3. A block of
// four warps walks down consecutive windows of one (batch, head); group g belongs to warp
// g mod 4 and stays with it through its four windows, so that q, k, v, dO and bias are
// each read once. dk and dv of the four groups are sums in tensor memory, group g in lanes
// 32 (g mod 4) ..: per window two tcgen05 products (128 keys x 32 channels x 32 queries,
// P^T and dS^T as MN-major operands) add to all of them, and the warp whose group has seen
// its last window reads its lanes, writes the 32 atoms' dk and dv, and clears them. No
// partial sum leaves the chip and nothing is added atomically. A block owns a run of
// groups; it first recomputes the three windows before its run, which the block before
// owns, for their share of dk and dv.
//
// What bounds it: memory, 448 B per atom and head, and 512 B of bias and its gradient,
// against 41 k operations; and next to it the 4096 exponentials and gradients of each
// window. Scores and dP run on the warp-level tensor instruction (m16n8k16): a warp
// holds 32 queries x its 32 keys in registers, so a query's statistics take two shuffles
// and one exchange of (maximum, sum of exponentials, sum of p dP) among the four warps.
// (A tcgen05 tile of 128 query rows would spend most of S outside the windows, and bring
// it back through tensor memory.) P goes to a tile of its own, dS to the bias's: both are
// the tcgen05 products' left operands as they lie; dq (m16n8k16) and the copy to dbias read
// dS there too. Keeping dk and dv in registers instead took 64 of them per lane: two blocks
// an SM fitted then, four do now (8 x 18432 atoms, 4 heads: 309 -> 168 us).
//
// Measured, the same size, call after call on the same inputs (and one call on inputs cold in L2): 144 us with bias,
// 3.9 TB/s (154), 152 (161) with 5 % of the atoms masked as well. DRAM is busy 45 %; the shared-memory
// pipe 61 %, the issue slots 45 %. A window's phases depend on each other, and four warps a scheduler
// do not cover that.
//
// Copies: TMA, kStages windows in flight (64-byte rows with the 64-byte swizzle; the bias as
// four tiles of 32 slots, one per warp). Every wait is bounded.
#include "kernels.h"

namespace trimul {
namespace ab {
constexpr int QW = 32, KOFF = 48;
constexpr int kStages = 2;
constexpr int kBlocks = 4;                 // blocks per SM
constexpr int RING = kStages + 3;          // key groups held: the window's four and those in flight
constexpr int TILE = 32 * 64;              // 32 rows of 32 bf16
constexpr int BIAS = 4 * TILE;             // [warp] 32 queries x the 32 slots of the warp's group
constexpr int THREADS = 128;
constexpr int OFF_BIAS = 0;                          // [kStages] bias, then dS
constexpr int OFF_P = OFF_BIAS + kStages * BIAS;     // P
constexpr int OFF_Q = OFF_P + BIAS;                  // [kStages] q
constexpr int OFF_DO = OFF_Q + kStages * TILE;       // [kStages] dO
constexpr int OFF_K = OFF_DO + kStages * TILE;       // [RING] k
constexpr int OFF_V = OFF_K + RING * TILE;           // [RING] v
constexpr int OFF_RED = OFF_V + RING * TILE;         // [4][32] float4: each warp's max, sum, sum p dP per query
constexpr int OFF_ROW = OFF_RED + 4 * 32 * 16;       // [4][32] float2: a warp's factor and -delta per query
constexpr int OFF_BAR = OFF_ROW + 4 * 32 * 8;
constexpr size_t SMEM = 512 + OFF_BAR + 64;
constexpr int DK_COL = 0, DV_COL = 32, TMEM_COLS = 64;
static_assert(kBlocks * (SMEM + 1024) <= 233472, "shared memory of an SM");
}  // namespace ab

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d = a b, d += a b: 16 x 8 (fp32) from 16 x 16 and 16 x 8 (bf16). d[0] holds row lane / 4, d[1] row
// lane / 4 + 8, columns 2 (lane % 4) and the next.
__device__ __forceinline__ void mma_first(float2 (&d)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0].x), "=f"(d[0].y), "=f"(d[1].x), "=f"(d[1].y)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_next(float2 (&d)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2_hw(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte offset of 16-byte chunk c (0..3) of row r in a tile of 64-byte rows (64-byte swizzle). The
// swizzle is an exclusive or, so a lane keeps the offset of its own row and chunk 0 or 1: chunk
// c + 2 is that offset ^ 32, and 16 rows more add 1024.
__device__ __forceinline__ uint32_t at64(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// Zeros in the warp's 32 lanes x 32 columns of tensor memory.
__device__ __forceinline__ void tmem_zero32(uint32_t taddr) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(taddr),
        "r"(0)
        : "memory");
}

// The sum, or the maximum, over the four lanes that hold one row of an accumulator.
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// s[32 queries][32 keys] = x[queries][32] y[keys][32]^T, tiles of 64-byte rows given as the lane's
// addresses (rows as left and as right operand); s[16-row tile][8-key tile].
__device__ __forceinline__ void product_32x32(float2 (&s)[2][4][2], uint32_t xa, uint32_t yb) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        uint32_t a0[4], a1[4], b01[4], b23[4];
        ldsm4(a0, xa ^ (32 * kk));
        ldsm4(a1, (xa ^ (32 * kk)) + 1024);
        ldsm4(b01, yb ^ (32 * kk));
        ldsm4(b23, (yb ^ (32 * kk)) + 1024);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            const uint32_t(&a)[4] = mt ? a1 : a0;
            if (kk == 0) {
                mma_first(s[mt][0], a, b01[0], b01[1]);
                mma_first(s[mt][1], a, b01[2], b01[3]);
                mma_first(s[mt][2], a, b23[0], b23[1]);
                mma_first(s[mt][3], a, b23[2], b23[3]);
            } else {
                mma_next(s[mt][0], a, b01[0], b01[1]);
                mma_next(s[mt][1], a, b01[2], b01[3]);
                mma_next(s[mt][2], a, b23[0], b23[1]);
                mma_next(s[mt][3], a, b23[2], b23[3]);
            }
        }
    }
}

}  // namespace

__global__ void __launch_bounds__(ab::THREADS, ab::kBlocks)
    atomattn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDo,
                        const __grid_constant__ CUtensorMap tmBias, const __grid_constant__ CUtensorMap tmDbias,
                        const __grid_constant__ CUtensorMap tmDq, const __grid_constant__ CUtensorMap tmDk,
                        const __grid_constant__ CUtensorMap tmDv, const AttnBwdArgs args) {
    using namespace ab;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((512u - (smem_u32(smem_raw) & 511u)) & 511u);
    const uint32_t sbase = smem_u32(smem);
    float4 *red = reinterpret_cast<float4 *>(smem + OFF_RED);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + OFF_BAR);  // [kStages] window landed
    uint64_t *summed = full + kStages;                               // the window's dk and dv products are done
    uint64_t *drain = summed + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int quad = lane & 3, grp = lane >> 2;
    const KernelCtl &ctl = args.ctl;
    const int h = (int)(blockIdx.x % args.heads);
    const int rest = (int)(blockIdx.x / args.heads);
    const int chain = rest % args.chains, b = rest / args.chains;
    const int n = args.n, nw = args.n_windows;
    // Groups (and windows' dq, dbias) this block owns: [s0, s1); it computes windows [first, wend).
    const int s0 = chain * args.per_chain, s1 = min(nw + 2, s0 + args.per_chain);
    const int first = max(0, s0 - 3), wend = min(nw, s1);
    const bool has_bias = args.has_bias != 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        mbar_init(summed, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (args.clear_status && blockIdx.x == 0 && threadIdx.x == 0) *ctl.status = DeviceStatus{0, 0, 0, 0};

    // Loads of window s: its q, dO and bias into stage (s - first) % kStages, and the key group
    // s + 3 (for the block's first window all four groups) into ring slot (group - first) % RING.
    auto issue = [&](int s) {
        const int i = s - first, st = i % kStages;
        const int g0 = i == 0 ? s : s + 3;
        mbar_arrive_expect_tx(&full[st], (uint32_t)(2 * TILE + (s + 4 - g0) * 2 * TILE + (has_bias ? BIAS : 0)));
        tma_load_3d(smem + OFF_Q + st * TILE, &tmQ, &full[st], h * 32, s * QW, b);
        tma_load_3d(smem + OFF_DO + st * TILE, &tmDo, &full[st], h * 32, s * QW, b);
        for (int g = g0; g < s + 4; ++g) {
            const int slot = (g - first) % RING;
            tma_load_3d(smem + OFF_K + slot * TILE, &tmK, &full[st], h * 32, g * 32 - KOFF, b);
            tma_load_3d(smem + OFF_V + slot * TILE, &tmV, &full[st], h * 32, g * 32 - KOFF, b);
        }
        if (has_bias)
            for (int x = 0; x < 4; ++x)
                tma_load_5d(smem + OFF_BIAS + st * BIAS + x * TILE, &tmBias, &full[st], ((x - s) & 3) * 32, 0, h, s, b);
    };
    int issued = 0;  // thread 0: windows whose loads have been issued
    if (threadIdx.x == 0)
        for (; issued < kStages && first + issued < wend; ++issued) issue(first + issued);

    uint32_t vmask = 0;  // valid keys of this warp's group, bit = atom - first atom of the group
    const float scale = args.scale, log2e = 1.4426950408889634f;
    const size_t row_elems = (size_t)args.heads * 32;
    // ldmatrix / stmatrix lane addresses within a tile: rows as a left operand's, as a right operand's.
    const uint32_t a64 = at64((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t b64 = at64((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
    const int s_r = (lane & 7) + ((lane >> 3) & 1) * 8;
    const uint32_t s32 = (uint32_t)(s_r * 32 + (((lane >> 4) ^ ((s_r >> 2) & 1)) << 4));
    const int q0 = (warp & 1) * 16, c0 = (warp >> 1) * 2;  // dq: this warp's 16 queries, and 16 channels from 8 c0
    const uint32_t mytmem = tmem + ((uint32_t)(warp * 32) << 16);
    auto ring_at = [&](int base, int j) { return base + j < RING ? base + j : base + j - RING; };

    // dk and dv of group g, whose windows are all summed, from this warp's lanes (lane = atom); with
    // `clear` the lanes are set to 0 for the warp's next group.
    auto write_group = [&](int g, bool clear, uint8_t *dv_tile) {
        if (g >= s0 && g < s1) {  // warp-uniform; else another block's
            const int row = g * 32 - KOFF, atom = row + lane;
            const bool valid = (vmask >> lane) & 1u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t v[32];
                tmem_ld32(mytmem + (x ? DV_COL : DK_COL), v);
                tmem_ld_wait_regs(v);
                if (clear) tmem_zero32(mytmem + (x ? DV_COL : DK_COL));
                const float f = x ? 1.f : scale;
                // Through P's tile, which is free from the window's sums to the next window's P: a lane's 64 bytes
                // straight to memory are 32 rows an instruction, and such stores were a quarter of the passes
                // through L1's data pipe (157 -> 148 us without them). (A block that starts before the first
                // atom: there is one for each sequence.)
                uint8_t *tile = (x ? dv_tile : smem + OFF_P + warp * TILE) + lane * 64;
                __nv_bfloat16 *dst = (x ? args.dv : args.dk) + ((size_t)b * n + atom) * row_elems + h * 32;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        o[t] = valid ? pack_bf16x2(__uint_as_float(v[8 * c + 2 * t]) * f,
                                                   __uint_as_float(v[8 * c + 2 * t + 1]) * f)
                                     : 0u;
                    if (row >= 0)
                        *reinterpret_cast<uint4 *>(tile + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    else if (atom >= 0 && atom < n)
                        reinterpret_cast<uint4 *>(dst)[c] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (row >= 0 && row < n) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmDk, smem + OFF_P + warp * TILE, h * 32, row, b);
                    tma_store_3d(&tmDv, dv_tile, h * 32, row, b);
                    tma_store_commit();
                }
            }
        } else if (clear) {
            tmem_zero32(mytmem + DK_COL);
            tmem_zero32(mytmem + DV_COL);
        }
    };
    // Whether this lane's key of group g is valid, as the mask's bits (0: not). Asked a window ahead.
    auto key_bits = [&](int g) -> uint16_t {
        const int atom = g * 32 - KOFF + lane;
        if (atom < 0 || atom >= n) return 0;
        return args.mask ? __ldg(reinterpret_cast<const uint16_t *>(args.mask) + (size_t)b * n + atom) : (uint16_t)0x3F80u;
    };
    uint16_t key = key_bits(first + ((warp - first) & 3));

    bool ok = true;
    int st = 0, base = 0;  // stage of window s, ring slot of group s
    uint32_t phase = 0;
    for (int s = first; s < wend; ++s) {
        const int i = s - first, pos = (warp - s) & 3;  // the place of this warp's group in the window
        const int slot = ring_at(base, pos);
        const uint32_t qa = sbase + OFF_Q + st * TILE + a64, oa = sbase + OFF_DO + st * TILE + a64;
        const uint32_t bt = sbase + OFF_BIAS + st * BIAS, mine = bt + warp * TILE + a64, pt = sbase + OFF_P + warp * TILE + a64;
        // [16-query tile][8-key tile][row, row + 8]: scores, then p; dP, then dS.
        float2 sc[2][4][2], dp[2][4][2];
        // The sums of the window before: its operands' tiles are free, and its oldest group is complete.
        ok = i == 0 || warp_wait(summed, (uint32_t)(i - 1) & 1u, abort_flag, ctl, SITE_ATB | 2, s);
        ok = ok && warp_wait(&full[st], phase, abort_flag, ctl, SITE_ATB | 1, s);
        if (ok) {
            if (pos == 3 || i == 0) {  // a new group
                if (i > 0) {
                    tc_fence_after();
                    // No other warp writes a group now: dv takes the next warp's part of the tile.
                    write_group(s - 1, true, smem + OFF_P + ((warp + 1) & 3) * TILE);
                } else {
                    tmem_zero32(mytmem + DK_COL);
                    tmem_zero32(mytmem + DV_COL);
                }
                // Which of its keys are valid. Masked ones are zeroed, so that what is stored there (anything,
                // infinities and NaN included) meets a zero weight as a zero.
                const bool valid = (key & 0x7FFFu) != 0;
                vmask = __ballot_sync(0xffffffffu, valid);
                if (!valid) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        *reinterpret_cast<uint4 *>(smem + OFF_K + slot * TILE + lane * 64 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(smem + OFF_V + slot * TILE + lane * 64 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();  // the slot is TMA's again later
                }
                __syncwarp();
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
            }
            product_32x32(sc, qa, sbase + OFF_K + slot * TILE + b64);
            product_32x32(dp, oa, sbase + OFF_V + slot * TILE + b64);
            // Logits; -inf where the key is not valid or the query is past the sequence.
            const float2 sc2 = make_float2(scale, scale);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    uint32_t bw[4] = {0u, 0u, 0u, 0u};  // (row, row + 8) of key tile 2 np, then of 2 np + 1
                    if (has_bias) ldsm4(bw, (mine ^ (32 * np)) + 1024 * mt);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float2 &l = sc[mt][2 * np + (x >> 1)][x & 1];
                        l = __ffma2_rn(l, sc2, make_float2(__uint_as_float(bw[x] << 16), __uint_as_float(bw[x] & 0xFFFF0000u)));
                    }
                }
            if (vmask != 0xFFFFFFFFu) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const uint32_t two = vmask >> (8 * nt + 2 * quad);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        // dP too: where every key is masked, dO may hold anything, and P = 0 would not hide it.
                        float2 &l = sc[x >> 1][nt][x & 1], &d = dp[x >> 1][nt][x & 1];
                        if (!(two & 1u)) l.x = -INFINITY, d.x = 0.f;
                        if (!(two & 2u)) l.y = -INFINITY, d.y = 0.f;
                    }
                }
            }
            const int left = n - s * QW;  // queries of this window
            if (left < QW) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (8 * x + grp >= left)
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) sc[x >> 1][nt][x & 1] = make_float2(-INFINITY, -INFINITY);
            }
            // Over this warp's keys, for each of the lane's four queries (8 x + grp): the maximum, the
            // sum of p = exp(l - maximum) and the sum of p dP.
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int mt = x >> 1, r = x & 1;
                float mx = fmaxf(sc[mt][0][r].x, sc[mt][0][r].y);
#pragma unroll
                for (int nt = 1; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(sc[mt][nt][r].x, sc[mt][nt][r].y));
                mx = quad_max(mx);
                const float m = mx == -INFINITY ? 0.f : mx;
                const float2 nm = make_float2(-m, -m), l2 = make_float2(log2e, log2e);
                float2 sum = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    // The difference before the factor: logits next to the type's lowest value stay finite.
                    const float2 t = __fmul2_rn(__fadd2_rn(sc[mt][nt][r], nm), l2);
                    const float2 p = make_float2(ex2_hw(t.x), ex2_hw(t.y));
                    sc[mt][nt][r] = p;
                    sum = __fadd2_rn(sum, p);
                    dot = __ffma2_rn(p, dp[mt][nt][r], dot);
                }
                const float tsum = quad_sum(sum.x + sum.y), tdot = quad_sum(dot.x + dot.y);
                if (quad == x) red[warp * 32 + 8 * x + grp] = make_float4(mx, tsum, tdot, 0.f);
            }
        }
        // This warp's copies out of shared memory (the window before's dq, its group's dk and dv) have read it.
        if (lane == 0) tma_store_wait_read<0>();
        // Every warp's part is there; and every warp is done with the window before.
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (pos == 0) key = key_bits(s + 4);  // the warp's next group
        float2 *rowv = reinterpret_cast<float2 *>(smem + OFF_ROW) + warp * 32;
        uint32_t empty;  // queries without weight, the same in every warp: past the last, or with no logit over -inf
        {
            float4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = red[32 * x + lane];
            const float m = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x));
            float total = 0.f, dots = 0.f, own = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float f = v[x].x == -INFINITY ? 0.f : ex2_hw((v[x].x - m) * log2e);
                total = fmaf(f, v[x].y, total);
                dots = fmaf(f, v[x].z, dots);
                if (x == warp) own = f;
            }
            const float inv = total == 0.f ? 0.f : 1.f / total;  // a query without a valid key: P = 0
            rowv[lane] = make_float2(own * inv, -dots * inv);
            empty = __ballot_sync(0xffffffffu, total == 0.f);
            // Their q and dO may hold anything, and 0 times it would not hide it in dk and dv. (Every warp is done with
            // its scores: the products below are the tiles' last readers.)
            if ((empty >> lane) & 1u) {
                *reinterpret_cast<uint4 *>(smem + OFF_Q + st * TILE + lane * 64 + 16 * warp) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4 *>(smem + OFF_DO + st * TILE + lane * 64 + 16 * warp) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        __syncwarp();
        // P and dS, each rounded once to bf16, the type of the products' other operands (the gradients are then off by
        // 0.0024 of their norm, against 0.0017 of their own rounding alone).
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t pb[4][2], ds[4][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 fd = rowv[16 * mt + 8 * r + grp];
                const float2 f2 = make_float2(fd.x, fd.x), nd = make_float2(fd.y, fd.y);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const float2 p = __fmul2_rn(sc[mt][nt][r], f2);
                    const float2 d = __fmul2_rn(p, __fadd2_rn(dp[mt][nt][r], nd));
                    pb[nt][r] = pack_bf16x2(p.x, p.y);
                    ds[nt][r] = pack_bf16x2(d.x, d.y);
                }
            }
            if (empty != 0u || vmask != 0xFFFFFFFFu) {
                // dS is 0 there, also where the query's sums are not numbers (P is written as 0, or to a masked
                // key's row of dv, which is not kept).
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const uint32_t two = vmask >> (8 * nt + 2 * quad);
                    const uint32_t kept = ((two & 1u) ? 0xFFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int r = 0; r < 2; ++r) ds[nt][r] &= (empty >> (16 * mt + 8 * r + grp)) & 1u ? 0u : kept;
                }
            }
            stsm4(pt + 1024 * mt, pb[0][0], pb[0][1], pb[1][0], pb[1][1]);
            stsm4((pt ^ 32) + 1024 * mt, pb[2][0], pb[2][1], pb[3][0], pb[3][1]);
            stsm4(mine + 1024 * mt, ds[0][0], ds[0][1], ds[1][0], ds[1][1]);
            stsm4((mine ^ 32) + 1024 * mt, ds[2][0], ds[2][1], ds[3][0], ds[3][1]);
        }
        fence_proxy_async_smem();
        __syncthreads();  // P and dS of all 128 slots are in their tiles
        if (threadIdx.x == 0 && i > 0 && first + issued < wend) {
            // The stage of window s - 1 and the ring slot of group s - 1 have been free since the barrier before
            // this one. Issued here, where no warp waits for this one, a window still passes before the data is
            // needed.
            issue(first + issued);
            ++issued;
        }
        if (threadIdx.x == 32) {
            // dv += P^T dO, dk += dS^T q: 128 keys (group g mod 4 in lanes 32 (g mod 4) ..) x 32 channels,
            // K = 32 queries in two steps; tiles of 32 keys are 2 KB apart.
            tc_fence_after();
            const uint32_t idesc = idesc_bf16(128, 32, 1, 1);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const uint32_t q_at = sbase + OFF_Q + st * TILE + 1024 * kk, o_at = sbase + OFF_DO + st * TILE + 1024 * kk;
                mma_bf16(tmem + DV_COL, sdesc_sw64(sbase + OFF_P + 1024 * kk, TILE, 512), sdesc_sw64(o_at, TILE, 512), idesc, 1u);
                mma_bf16(tmem + DK_COL, sdesc_sw64(bt + 1024 * kk, TILE, 512), sdesc_sw64(q_at, TILE, 512), idesc, 1u);
            }
            mma_commit(summed);
        }
        if (s >= s0) {
            if (args.has_dbias && threadIdx.x == 0) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    tma_store_5d(&tmDbias, smem + OFF_BIAS + st * BIAS + x * TILE, ((x - s) & 3) * 32, 0, h, s, b);
                tma_store_commit();
            }
            __syncwarp();
            float2 dq[2][2];
            const uint32_t da = bt + a64 + q0 * 64, ka = sbase + OFF_K + (a64 ^ (c0 << 4));
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // tile x = kk / 2 holds the group of warp x
                uint32_t a[4], bk[4];
                ldsm4(a, (da ^ (32 * (kk & 1))) + (kk >> 1) * TILE);
                ldsm4_t(bk, ka + ring_at(base, ((kk >> 1) - s) & 3) * TILE + (kk & 1) * 1024);
                if (kk == 0) {
                    mma_first(dq[0], a, bk[0], bk[1]);
                    mma_first(dq[1], a, bk[2], bk[3]);
                } else {
                    mma_next(dq[0], a, bk[0], bk[1]);
                    mma_next(dq[1], a, bk[2], bk[3]);
                }
            }
            // Out through the slot of v of the group that has just seen its last scores: 512 bytes a warp, rows of 32
            // bytes with the 32-byte swizzle.
            uint32_t o[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    o[x][r] = (empty >> (q0 + 8 * r + grp)) & 1u ? 0u : pack_bf16x2(dq[x][r].x * scale, dq[x][r].y * scale);
            uint8_t *out = smem + OFF_V + base * TILE + warp * 512;
            stsm4(smem_u32(out) + s32, o[0][0], o[0][1], o[1][0], o[1][1]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && s * QW + q0 < n) {
                tma_store_3d(&tmDq, out, h * 32 + c0 * 8, s * QW + q0, b);
                tma_store_commit();
            }
        }
        if (++st == kStages) {
            st = 0;
            phase ^= 1u;
        }
        base = ring_at(base, 1);
    }
    // The groups of the last window: those this block owns have no window after it.
    if (ok) {
        const int last = wend - 1;
        if (warp_wait(summed, (uint32_t)(last - first) & 1u, abort_flag, ctl, SITE_ATB | 3, last)) {
            tc_fence_after();
            // Here up to three warps do: dv takes the warp's part of the bias tile that no window needs any more.
            write_group(last + ((warp - last) & 3), false, smem + OFF_BIAS + st * BIAS + warp * TILE);
        }
    } else if (threadIdx.x == 32) {
        mma_commit(drain);  // no product may still be running when the block leaves
        wait_drain(drain, 0, ctl.timeout_ns);
    }
    // No copy may be in flight when the block leaves (loads: only after a timeout).
    if (threadIdx.x == 0)
        for (int x = max(0, issued - kStages); x < issued; ++x)
            wait_drain(&full[x % kStages], (uint32_t)(x / kStages) & 1u, ctl.timeout_ns);
    if (lane == 0) tma_store_wait_all<0>();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

cudaError_t atomattn_bwd_setup() {
    return cudaFuncSetAttribute(atomattn_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ab::SMEM);
}

cudaError_t launch_atomattn_bwd(const AttnBwdMaps &m, AttnBwdArgs a, int sms, cudaStream_t s) {
    // The shortest runs that still fit one wave of kBlocks blocks an SM: a block's work is its run and
    // three windows more, so long sequences get long runs and short ones little depth.
    const long long pairs = (long long)a.batch * a.heads, wave = (long long)ab::kBlocks * sms;
    const int steps = a.n_windows + 2;
    long long chains = wave / pairs;
    if (chains < 1) chains = 1;
    if (chains > steps) chains = steps;
    a.per_chain = (int)((steps + chains - 1) / chains);
    a.chains = (steps + a.per_chain - 1) / a.per_chain;
    atomattn_bwd_kernel<<<(unsigned)(pairs * a.chains), ab::THREADS, ab::SMEM, s>>>(m.q, m.k, m.v, m.dout, m.bias, m.dbias, m.dq,
                                                                                     m.dk, m.dv, a);
    return cudaGetLastError();
}

}  // namespace trimul
