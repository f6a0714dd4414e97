// atomattn_bwd.cu - gradients of sequence-local atom attention (include/atomattn.h).
//
// For one batch element and head, window w (queries 32w .., key slots 32w - 48 ..):
//   P = softmax over the valid slots of q k^T / sqrt(32) + bias     (recomputed)
//   dP = dO v^T,  delta_i = sum_s P_is dP_is,  dS = P (dP - delta)
//   dq = dS k / sqrt(32),  dk += dS^T q / sqrt(32),  dv += P^T dO,  dbias = dS
//
// A key atom takes part in four consecutive windows. Keys are taken in groups of 32
// (group g: atoms 32g - 48 .. 32g - 17); window w holds groups w .. w + 3. A block of
// four warps walks down consecutive windows of one (batch, head): warp g mod 4 keeps
// the fp32 sums dk and dv of group g in registers through the group's four windows and
// then writes them once, so no sum leaves the chip unfinished, nothing is added
// atomically, and q, k, v, dO and bias are each read once. A block owns a run of
// groups; it first recomputes the three windows before its run, which the block
// before owns, for their share of dk and dv.
//
// What bounds it: memory, 448 B per atom and head, and 512 B of bias and its gradient,
// against 41 k operations. The five products run on the warp-level tensor instruction
// (m16n8k16): at 32 x 128 x 32 per window a tcgen05 tile of 128 query rows would spend
// seven eighths of each product outside the windows, and its accumulators would
// have to leave tensor memory for the softmax and return through shared memory in two
// layouts. The scores are held transposed, keys as rows: P^T and dS^T are then, as they
// lie in registers, the left operands of dv and dk; only dS is turned, by a
// transposing store into the bias's own tile, from which dq's product and the copy to
// dbias both read.
//
// Softmax across the four warps: each takes its own keys' maximum, sum of exponentials
// and sum of p dP, and one exchange through shared memory joins the three.
//
// Copies: TMA, kStages windows in flight (64-byte rows with the 64-byte swizzle, bias
// rows with the 128-byte one). Every wait is bounded.
#include "kernels.h"

namespace trimul {
namespace ab {
constexpr int QW = 32, KOFF = 48;
constexpr int kStages = 3;
constexpr int RING = kStages + 3;          // key groups held: the window's four and those in flight
constexpr int TILE = 32 * 64;              // 32 atoms of one head
constexpr int BIAS_HALF = 32 * 128;        // 32 rows x 64 slots
constexpr int BIAS = 2 * BIAS_HALF;
constexpr int THREADS = 128;
constexpr int OFF_BIAS = 0;                          // [kStages][2][32][64] bias, then dS
constexpr int OFF_Q = OFF_BIAS + kStages * BIAS;     // [kStages] q
constexpr int OFF_DO = OFF_Q + kStages * TILE;       // [kStages] dO
constexpr int OFF_K = OFF_DO + kStages * TILE;       // [RING] k
constexpr int OFF_V = OFF_K + RING * TILE;           // [RING] v
constexpr int OFF_RED = OFF_V + RING * TILE;         // [2][32][4] float4: each warp's max, sum, sum p dP
constexpr int OFF_ROW = OFF_RED + 2 * 32 * 4 * 16;   // [4][32] float2: a warp's factor and delta per query
constexpr int OFF_BAR = OFF_ROW + 4 * 32 * 8;
constexpr size_t SMEM = 1024 + OFF_BAR + 64;
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
// d += a b: 16 x 8 (fp32) from 16 x 16 and 16 x 8 (bf16).
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2_hw(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte chunk c (0..3) of row r in a tile of 64-byte rows (64-byte swizzle).
__device__ __forceinline__ uint32_t at64(uint32_t tile, int r, int c) {
    return tile + (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
// 16-byte chunk c (0..15, 8 slots each) of row r in a bias tile (two halves of 128-byte rows).
__device__ __forceinline__ uint32_t at128(uint32_t tile, int r, int c) {
    return tile + (uint32_t)((c >> 3) * ab::BIAS_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// A reduction over the eight lanes that share lane % 4, of eight values each: lane group
// r = lane / 4 returns the result of value index r with its bits reversed (see value_of).
template <typename Op>
__device__ __forceinline__ float reduce_scatter8(const float (&x)[8], int lane, Op op) {
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float y[4], z[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = b4 ? x[i + 4] : x[i], give = b4 ? x[i] : x[i + 4];
        y[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 16));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = b3 ? y[i + 2] : y[i], give = b3 ? y[i] : y[i + 2];
        z[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 8));
    }
    const float keep = b2 ? z[1] : z[0], give = b2 ? z[0] : z[1];
    return op(keep, __shfl_xor_sync(0xffffffffu, give, 4));
}

}  // namespace

__global__ void __launch_bounds__(ab::THREADS, 3)
    atomattn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDo,
                        const __grid_constant__ CUtensorMap tmBias, const __grid_constant__ CUtensorMap tmDbias,
                        const AttnBwdArgs args) {
    using namespace ab;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    float4 *red = reinterpret_cast<float4 *>(smem + OFF_RED);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + OFF_BAR);  // [kStages]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(full + kStages);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane & 3, grp = lane >> 2;
    const KernelCtl &ctl = args.ctl;
    const int h = (int)(blockIdx.x % args.heads);
    const int rest = (int)(blockIdx.x / args.heads);
    const int chain = rest % args.chains, b = rest / args.chains;
    const int n = args.n, nw = args.n_windows;
    // Groups (and windows' dq, dbias) this block owns: [s0, s1); its first window is s0 - 3.
    const int s0 = chain * args.per_chain, s1 = min(nw + 2, s0 + args.per_chain);
    const int first = max(0, s0 - 3), wend = min(nw, s1);
    const bool has_bias = args.has_bias != 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) *ctl.status = DeviceStatus{0, 0, 0, 0};

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
        if (has_bias) {
            tma_load_5d(smem + OFF_BIAS + st * BIAS, &tmBias, &full[st], 0, 0, h, s, b);
            tma_load_5d(smem + OFF_BIAS + st * BIAS + BIAS_HALF, &tmBias, &full[st], 64, 0, h, s, b);
        }
    };
    int issued = 0;  // thread 0: windows whose loads have been issued
    if (threadIdx.x == 0)
        for (; issued < kStages && first + issued < wend; ++issued) issue(first + issued);

    float dk[2][4][4], dv[2][4][4];  // [16-key tile][8-channel tile] sums of this warp's group
#pragma unroll
    for (int i = 0; i < 32; ++i) (&dk[0][0][0])[i] = (&dv[0][0][0])[i] = 0.f;
    uint32_t vmask = 0;  // valid keys of this warp's group, bit = atom - first atom of the group
    const float scale = args.scale, log2e = 1.4426950408889634f;
    const size_t row_elems = (size_t)args.heads * 32;
    // ldmatrix / stmatrix lane coordinates: row and chunk of the matrix a lane addresses.
    const int la_r = (lane & 7) + ((lane >> 3) & 1) * 8, la_c = lane >> 4;  // 16 rows, 2 chunks
    const int lb_r = (lane & 7) + (lane >> 4) * 8, lb_c = (lane >> 3) & 1;

    bool ok = true;
    int seen = -1;  // the group whose keys this warp has looked at
    for (int s = first; s < s1; ++s) {
        const int i = s - first;
        const int pos = (warp - s) & 3, g = s + pos;  // this warp's group and its place in the window
        if (s < wend) {
            const int st = i % kStages, slot = (g - first) % RING;
            const uint32_t kt = sbase + OFF_K + slot * TILE, vt = sbase + OFF_V + slot * TILE;
            const uint32_t qt = sbase + OFF_Q + st * TILE, dot_ = sbase + OFF_DO + st * TILE;
            const uint32_t bt = sbase + OFF_BIAS + st * BIAS;
            float sc[2][4][4], dp[2][4][4];  // [16-key tile][8-query tile]: scores, then P; dP, then dS
            ok = warp_wait(&full[st], (uint32_t)(i / kStages) & 1u, abort_flag, ctl, SITE_ATB | 1, s);
            if (ok) {
                if (g != seen) {
                    // New keys: which are valid. Masked ones are zeroed, so that what is stored there
                    // (anything, infinities and NaN included) meets a zero weight as a zero.
                    const int atom = g * 32 - KOFF + lane;
                    bool valid = atom >= 0 && atom < n;
                    if (valid && args.mask) valid = (__ldg(reinterpret_cast<const uint16_t *>(args.mask) + (size_t)b * n + atom) & 0x7FFFu) != 0;
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
                    seen = g;
                }
                // Scores and dP, transposed: 32 keys x 32 queries.
#pragma unroll
                for (int x = 0; x < 32; ++x) (&sc[0][0][0])[x] = (&dp[0][0][0])[x] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t a0[4], a1[4], b01[4], b23[4];
                    ldsm4(a0, at64(kt, la_r, kk * 2 + la_c));
                    ldsm4(a1, at64(kt, 16 + la_r, kk * 2 + la_c));
                    ldsm4(b01, at64(qt, lb_r, kk * 2 + lb_c));
                    ldsm4(b23, at64(qt, 16 + lb_r, kk * 2 + lb_c));
                    mma16816(sc[0][0], a0, b01[0], b01[1]);
                    mma16816(sc[0][1], a0, b01[2], b01[3]);
                    mma16816(sc[0][2], a0, b23[0], b23[1]);
                    mma16816(sc[0][3], a0, b23[2], b23[3]);
                    mma16816(sc[1][0], a1, b01[0], b01[1]);
                    mma16816(sc[1][1], a1, b01[2], b01[3]);
                    mma16816(sc[1][2], a1, b23[0], b23[1]);
                    mma16816(sc[1][3], a1, b23[2], b23[3]);
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t a0[4], a1[4], b01[4], b23[4];
                    ldsm4(a0, at64(vt, la_r, kk * 2 + la_c));
                    ldsm4(a1, at64(vt, 16 + la_r, kk * 2 + la_c));
                    ldsm4(b01, at64(dot_, lb_r, kk * 2 + lb_c));
                    ldsm4(b23, at64(dot_, 16 + lb_r, kk * 2 + lb_c));
                    mma16816(dp[0][0], a0, b01[0], b01[1]);
                    mma16816(dp[0][1], a0, b01[2], b01[3]);
                    mma16816(dp[0][2], a0, b23[0], b23[1]);
                    mma16816(dp[0][3], a0, b23[2], b23[3]);
                    mma16816(dp[1][0], a1, b01[0], b01[1]);
                    mma16816(dp[1][1], a1, b01[2], b01[3]);
                    mma16816(dp[1][2], a1, b23[0], b23[1]);
                    mma16816(dp[1][3], a1, b23[2], b23[3]);
                }
                // Logits; -inf where the key is not valid or the query is past the sequence.
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    uint32_t bw[4] = {0u, 0u, 0u, 0u};  // key blocks of 8: (16-key tile 0, 0), (0, +8), (1, 0), (1, +8)
                    if (has_bias) ldsm4_t(bw, at128(bt, nt * 8 + (lane & 7), pos * 4 + (lane >> 3)));
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint32_t w = bw[2 * mt + r];
                            sc[mt][nt][2 * r] = fmaf(sc[mt][nt][2 * r], scale, __uint_as_float(w << 16));
                            sc[mt][nt][2 * r + 1] = fmaf(sc[mt][nt][2 * r + 1], scale, __uint_as_float(w & 0xFFFF0000u));
                        }
                }
                if (vmask != 0xFFFFFFFFu) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (!((vmask >> (16 * mt + 8 * r + grp)) & 1u))
#pragma unroll
                                for (int nt = 0; nt < 4; ++nt) sc[mt][nt][2 * r] = sc[mt][nt][2 * r + 1] = -INFINITY;
                }
                const int left = n - s * QW;  // queries of this window
                if (left < QW) {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (nt * 8 + 2 * quad + e >= left)
#pragma unroll
                                for (int mt = 0; mt < 2; ++mt) sc[mt][nt][e] = sc[mt][nt][2 + e] = -INFINITY;
                }
                // This warp's maximum per query (column nt * 8 + 2 quad + e; index 2 nt + e), to all lanes.
                float mx[8], sum[8], dot[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int nt = c >> 1, e = c & 1;
                    mx[c] = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 4));
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 8));
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 16));
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int nt = c >> 1, e = c & 1;
                    const float m = mx[c] == -INFINITY ? 0.f : mx[c];
                    sum[c] = 0.f;
                    dot[c] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            // The difference before the factor: logits next to the type's lowest value stay finite.
                            const float p = ex2_hw((sc[mt][nt][2 * r + e] - m) * log2e);
                            sc[mt][nt][2 * r + e] = p;
                            sum[c] += p;
                            dot[c] = fmaf(p, dp[mt][nt][2 * r + e], dot[c]);
                        }
                }
                const auto add = [](float x, float y) { return x + y; };
                const float tsum = reduce_scatter8(sum, lane, add), tdot = reduce_scatter8(dot, lane, add);
                // Lane group grp holds column index c with bits (16, 8, 4) of the lane as its bits (4, 2, 1).
                const int c = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
                float tmax = mx[0];
#pragma unroll
                for (int x = 1; x < 8; ++x) tmax = c == x ? mx[x] : tmax;
                const int col = (c >> 1) * 8 + 2 * quad + (c & 1);
                red[((i & 1) * 32 + col) * 4 + warp] = make_float4(tmax, tsum, tdot, 0.f);
            }
            // Every warp's part is there; and every warp is done with the window before.
            ok = __syncthreads_and(ok);
            if (!ok) break;
            if (threadIdx.x == 0 && i > 0 && first + issued < wend) {
                // The stage of window s - 1 and the ring slot of group s - 1 are free once the copy of its dbias
                // has read the tile.
                tma_store_wait_read<0>();
                issue(first + issued);
                ++issued;
            }
            float2 *rowv = reinterpret_cast<float2 *>(smem + OFF_ROW) + warp * 32;
            {
                const float4 *r4 = red + ((i & 1) * 32 + lane) * 4;
                float4 v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = r4[x];
                const float m = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x));
                float total = 0.f, dots = 0.f, mine = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float f = v[x].x == -INFINITY ? 0.f : ex2_hw((v[x].x - m) * log2e);
                    total = fmaf(f, v[x].y, total);
                    dots = fmaf(f, v[x].z, dots);
                    if (x == warp) mine = f;
                }
                const float inv = total == 0.f ? 0.f : 1.f / total;  // a query without a valid key: P = 0
                rowv[lane] = make_float2(mine * inv, dots * inv);
            }
            __syncwarp();
            // P and dS.
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float4 fd = *reinterpret_cast<const float4 *>(&rowv[nt * 8 + 2 * quad]);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float p0 = sc[mt][nt][2 * r] * fd.x, p1 = sc[mt][nt][2 * r + 1] * fd.z;
                        sc[mt][nt][2 * r] = p0;
                        sc[mt][nt][2 * r + 1] = p1;
                        dp[mt][nt][2 * r] = p0 * (dp[mt][nt][2 * r] - fd.y);
                        dp[mt][nt][2 * r + 1] = p1 * (dp[mt][nt][2 * r + 1] - fd.w);
                    }
            }
            // bf16 operands: P and dS are rounded once, to the type of the products' other operands.
            uint32_t ds[2][4][2];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) ds[mt][nt][r] = pack_bf16x2(dp[mt][nt][2 * r], dp[mt][nt][2 * r + 1]);
                stmatrix_x4_trans(at128(bt, nt * 8 + (lane & 7), pos * 4 + (lane >> 3)), ds[0][nt][0], ds[0][nt][1],
                                  ds[1][nt][0], ds[1][nt][1]);
            }
            fence_proxy_async_smem();
            if (g >= s0 && g < s1) {
#pragma unroll
                for (int kq = 0; kq < 2; ++kq) {
                    uint32_t pa[2][4], sa[2][4];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        pa[mt][0] = pack_bf16x2(sc[mt][2 * kq][0], sc[mt][2 * kq][1]);
                        pa[mt][1] = pack_bf16x2(sc[mt][2 * kq][2], sc[mt][2 * kq][3]);
                        pa[mt][2] = pack_bf16x2(sc[mt][2 * kq + 1][0], sc[mt][2 * kq + 1][1]);
                        pa[mt][3] = pack_bf16x2(sc[mt][2 * kq + 1][2], sc[mt][2 * kq + 1][3]);
                        sa[mt][0] = ds[mt][2 * kq][0];
                        sa[mt][1] = ds[mt][2 * kq][1];
                        sa[mt][2] = ds[mt][2 * kq + 1][0];
                        sa[mt][3] = ds[mt][2 * kq + 1][1];
                    }
#pragma unroll
                    for (int nd = 0; nd < 2; ++nd) {
                        uint32_t bo[4], bq[4];
                        ldsm4_t(bo, at64(dot_, kq * 16 + la_r, nd * 2 + la_c));
                        ldsm4_t(bq, at64(qt, kq * 16 + la_r, nd * 2 + la_c));
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            mma16816(dv[mt][2 * nd], pa[mt], bo[0], bo[1]);
                            mma16816(dv[mt][2 * nd + 1], pa[mt], bo[2], bo[3]);
                            mma16816(dk[mt][2 * nd], sa[mt], bq[0], bq[1]);
                            mma16816(dk[mt][2 * nd + 1], sa[mt], bq[2], bq[3]);
                        }
                    }
                }
            }
            __syncthreads();  // dS of all 128 slots is in the tile
            if (s >= s0) {
                if (args.has_dbias && threadIdx.x == 0) {
                    tma_store_5d(&tmDbias, smem + OFF_BIAS + st * BIAS, 0, 0, h, s, b);
                    tma_store_5d(&tmDbias, smem + OFF_BIAS + st * BIAS + BIAS_HALF, 64, 0, h, s, b);
                    tma_store_commit();
                }
                // dq: warp (x, y) takes queries 16 x .. and channels 16 y ..
                const int q0 = (warp & 1) * 16, c0 = (warp >> 1) * 2;
                float dq[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    uint32_t a[4], bk[4];
                    const uint32_t kg = sbase + OFF_K + ((s + (kk >> 1) - first) % RING) * TILE;
                    ldsm4(a, at128(bt, q0 + la_r, kk * 2 + la_c));
                    ldsm4_t(bk, at64(kg, (kk & 1) * 16 + la_r, c0 + la_c));
                    mma16816(dq[0], a, bk[0], bk[1]);
                    mma16816(dq[1], a, bk[2], bk[3]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int atom = s * QW + q0 + 8 * r + grp;
                    if (atom < n) {
                        __nv_bfloat16 *dst = args.dq + ((size_t)b * n + atom) * row_elems + h * 32 + c0 * 8 + 2 * quad;
                        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(dq[0][2 * r] * scale, dq[0][2 * r + 1] * scale);
                        *reinterpret_cast<uint32_t *>(dst + 8) = pack_bf16x2(dq[1][2 * r] * scale, dq[1][2 * r + 1] * scale);
                    }
                }
            }
        }
        // Group s has seen its last window.
        if (pos == 0) {
            if (s >= s0) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int at = 16 * mt + 8 * r + grp, atom = g * 32 - KOFF + at;
                        if (atom >= 0 && atom < n) {
                            const bool valid = (vmask >> at) & 1u;
                            const size_t off = ((size_t)b * n + atom) * row_elems + h * 32 + 2 * quad;
#pragma unroll
                            for (int nt = 0; nt < 4; ++nt) {
                                *reinterpret_cast<uint32_t *>(args.dk + off + 8 * nt) =
                                    valid ? pack_bf16x2(dk[mt][nt][2 * r] * scale, dk[mt][nt][2 * r + 1] * scale) : 0u;
                                *reinterpret_cast<uint32_t *>(args.dv + off + 8 * nt) =
                                    valid ? pack_bf16x2(dv[mt][nt][2 * r], dv[mt][nt][2 * r + 1]) : 0u;
                            }
                        }
                    }
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) (&dk[0][0][0])[x] = (&dv[0][0][0])[x] = 0.f;
        }
    }
    if (threadIdx.x == 0) {
        // No copy may be in flight when the block leaves (loads: only after a timeout).
        for (int x = max(0, issued - kStages); x < issued; ++x)
            wait_drain(&full[x % kStages], (uint32_t)(x / kStages) & 1u, ctl.timeout_ns);
        tma_store_wait_all<0>();
    }
}

size_t atomattn_bwd_smem() { return ab::SMEM; }

cudaError_t atomattn_bwd_setup() {
    return cudaFuncSetAttribute(atomattn_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ab::SMEM);
}

cudaError_t launch_atomattn_bwd(const AttnBwdMaps &m, AttnBwdArgs a, int sms, cudaStream_t s) {
    // The shortest runs that still fit one wave of three blocks an SM: a block's work is its run and
    // three windows more, so long sequences get long runs and short ones little depth.
    const long long pairs = (long long)a.batch * a.heads, wave = 3ll * sms;
    const int steps = a.n_windows + 2;
    long long chains = wave / pairs;
    if (chains < 1) chains = 1;
    if (chains > steps) chains = steps;
    a.per_chain = (int)((steps + chains - 1) / chains);
    a.chains = (steps + a.per_chain - 1) / a.per_chain;
    atomattn_bwd_kernel<<<(unsigned)(pairs * a.chains), ab::THREADS, ab::SMEM, s>>>(m.q, m.k, m.v, m.dout, m.bias, m.dbias, a);
    return cudaGetLastError();
}

}  // namespace trimul
