// Gated feed-forward block for sm_100a, forward and backward.
//
//   G = X Wg^T,  U = X Wu^T,  H = act(G) * U        one kernel
//   Y = H Wd^T                                      one kernel (or a sparse layer)
//   backward:
//   dH = dY Wd,  dG = dH U act'(G),  dU = dH act(G) one kernel
//   dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X,  dWd = dY^T H
//                                                   one kernel for all four
//
// All of it is GEMM work, bound by the tensor cores but for few tokens, which
// have kernels of their own going forward (gated_few.cu, gated_some.cu).  One persistent kernel template serves the four launches:
// a CTA pair computes 256 x 256 of fp32 accumulator with cta_group::2 MMAs, each
// CTA holding 128 rows of A and 128 of B, with the accumulator double-buffered
// in tensor memory so that the epilogue of one tile overlaps the main loop of
// the next.  Warp 0 loads by TMA, warp 1 issues the MMAs, the others run the
// epilogue.  Where tiles are fewer than CTA pairs and long, they are cut along
// K; the parts are left in fp32 in the caller's workspace, and a small kernel
// adds them in order.
//
// Measured, TFLOP/s of the call (the measured cuBLAS rate is 1632 in a burst and
// 1354 under the power cap): forward at 32760 x 5120 -> 13824 1354-1590 by the
// power state, training step on 8192 tokens 1266-1530.  Tensor pipe active
// 92% (gate and up), 83% (down), 88% (dH) and 96% (gradients) at 4096 tokens.
// A stage's operands are 32 KB a CTA for 512 cycles of MMAs, so L2 has to deliver
// 64 bytes a cycle to every SM: rows that do not start on 128-byte lines (widths
// not a multiple of 64) stretch a stage to about 700 cycles.  With D below about 512
// the epilogue outlasts the main loop.
//
// Gate and up projections in one kernel: CTA 0's half of B is 128 rows of Wg,
// CTA 1's the same 128 rows of Wu.  The pair's MMA then leaves G in columns
// 0-127 and U in 128-255 of the same tensor-memory rows, so the thread that
// reads G[m, j] reads U[m, j] too: the activation and the product need no
// exchange, and X is read once for both.
//
// Operands come in the layout they are stored in: "K-major" rows (X, Wg) or
// "MN-major" where the reduction runs down the rows (dG^T X sums over tokens;
// dY Wd over Wd's rows).  No transposed copy is made: the tensor map's box is
// 64 contiguous elements by 64 rows either way, and the MMA's descriptors say
// which of the two is K.
//
// fp32 accumulation throughout.  H, dG and dU are rounded to bf16 once, as the
// next MMA takes bf16; H is made from the unrounded G and U.  G and U are no
// operand of anything, so what backward keeps of them is 24 bits: the upper 16
// of each, and the next eight of both in one more 16-bit array.  Kept as bf16
// they would add two roundings to dG and dU (error of the weights' gradients
// 1.85 times a bf16 rounding, 1.4 so).
#include "../../include/rtlynx.h"
#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"

#include <type_traits>

namespace rtlynx {
namespace {

constexpr uint32_t kTmemColumns = 512;
constexpr int kTile = 256;                      // rows of a tile, and accumulator columns unless narrow
constexpr int kHalf = 128;                      // one CTA's share of either operand
constexpr int kNarrow = 128;                    // accumulator columns of a narrow tile
constexpr int kOperandBytes = kHalf * 64 * 2;   // 128 x 64 values
constexpr int kStagingBytes = 6 * 2 * kOperandBytes;  // six stages of A and B; eight where B is half as wide
constexpr int kEpiWarps = 8;                    // two on each quadrant of tensor-memory lanes, half of the columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kPieceBytes = 32 * 32 * 2;        // 32 rows x 32 columns on their way out
constexpr int kSmemBytes = kStagingBytes + kEpiWarps * 2 * kPieceBytes + 1024 + 1024;
constexpr int kMaxProblems = 4;
constexpr int kMaxMaps = 16;
static_assert(kSmemBytes <= 232448, "shared memory budget");

enum Epilogue { kStore = 0, kGatedForward = 1, kGatedBackward = 2 };

// One product A B^T (+ A' B'^T) of a launch.  Map indices point into
// GatedArgs::maps; going forward CTA 0 reads B through map b0 (Wg) and CTA 1
// through the next one (Wu).
struct Problem {
    int m_pairs, n_tiles, group_n;
    int first_unit, split;      // units [first_unit, first_unit + tiles * split)
    int k0, k;                  // stages of the first operand pair, of both
    int a0, b0, a1, b1;
    int a_mn, b_mn;             // operand is MN-major
    int rows, cols;             // of the output
    int out[4];                 // maps of the outputs; forward: H, G, U, low (the last three may be -1); backward: dG, dU
    uint16_t* sum_out[2];       // split > 1: the outputs themselves, for the summing kernel
    int sum_pitch;              // values from one of their rows to the next
    const uint16_t* in[3];      // backward: G, U, low
    float* part;                // split > 1: fp32 partial tiles
};

struct GatedArgs {
    CUtensorMap maps[kMaxMaps];
    Problem p[kMaxProblems];
    int problems, units;
    int longs, extra;  // see Units
    int* err;
};

struct Unit {
    int problem, mp, nt, kb, ke;
    int index;  // among the problem's units
};

// Column tiles in groups of group_n, a group's tiles row pair by row pair.
__device__ __forceinline__ void tile_at(const Problem& p, int tile, int& mp, int& nt) {
    const int per_group = p.m_pairs * p.group_n;
    const int g = tile / per_group;
    const int width = min(p.group_n, p.n_tiles - g * p.group_n);
    const int in_group = tile - g * per_group;
    mp = in_group / width;
    nt = g * p.group_n + in_group - mp * width;
}

// The units of a CTA pair, one after another.  The first `longs` units (the
// longer kind where a launch has two) are dealt round; the pairs from `rest` on,
// which have one of them less, take `extra` of the others each instead, and what
// is left is dealt round.  Divisions are kept out of the way of the common case
// (nothing split, no long units): every role computes this between two tiles.
struct Units {
    int pair, pairs, rest, own, shift;

    __device__ __forceinline__ Units(const GatedArgs& args, int pair_, int pairs_) : pair(pair_), pairs(pairs_) {
        rest = own = 0;
        if (args.longs > 0) {
            rest = args.longs % pairs;
            own = args.longs / pairs + (pair < rest ? 1 : 0);
        }
        shift = args.longs + args.extra * (pairs - rest);  // first unit dealt round after the extra ones
    }

    __device__ __forceinline__ bool at(int i, const GatedArgs& args, Unit& w) const {
        int u;
        if (i < own) {
            u = pair + i * pairs;
        } else {
            const int j = i - own, extra = pair >= rest ? args.extra : 0;
            u = j < extra ? args.longs + j * (pairs - rest) + pair - rest : shift + (j - extra) * pairs + pair;
        }
        if (u >= args.units) return false;
        int n = 0;
        while (n + 1 < args.problems && u >= args.p[n + 1].first_unit) ++n;
        const Problem& p = args.p[n];
        w.problem = n;
        w.index = u - p.first_unit;
        int tile = w.index;
        w.kb = 0;
        w.ke = p.k;
        if (p.split > 1) {
            tile = w.index / p.split;
            const int part = w.index - tile * p.split;
            w.kb = part * p.k / p.split;
            w.ke = (part + 1) * p.k / p.split;
        }
        tile_at(p, tile, w.mp, w.nt);
        return true;
    }
};

__device__ __forceinline__ bool whole_warp_wait(uint64_t* bar, uint32_t parity, int* err) {
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, err) ? 1u : 0u;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

using KMajor = std::integral_constant<bool, false>;
using MnMajor = std::integral_constant<bool, true>;

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// 128 x 64 values into shared memory (64 x 64 of B of a narrow tile), 128B
// swizzle.  K-major: rows of 64 K values, as many as the map's box has.
// MN-major: boxes of 64 row values x 64 K.
template <bool MN, int ROWS = kHalf>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row) {
    if (MN) {
        tma_load_pair(dst, map, bar, row, k);
        if (ROWS > 64) tma_load_pair(dst + kOperandBytes / 2, map, bar, row + 64, k);
    } else {
        tma_load_pair(dst, map, bar, k, row);
    }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// 32 accumulator columns, rounded.
__device__ __forceinline__ void pack32(const uint32_t (&r)[32], uint4 (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[8 * q + j]);
        v[q] = pack8(f);
    }
}

// The upper 16 bits of eight values.
__device__ __forceinline__ uint4 high8(const uint32_t* r) {
    return make_uint4(__byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632), __byte_perm(r[4], r[5], 0x7632),
                      __byte_perm(r[6], r[7], 0x7632));
}

// The eight bits below those, of two arrays: the first's in the low byte.
__device__ __forceinline__ uint32_t low2(uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1) {
    return __byte_perm(__byte_perm(a0, b0, 0x0051), __byte_perm(a1, b1, 0x0051), 0x5410);
}
__device__ __forceinline__ uint4 low8(const uint32_t* a, const uint32_t* b) {
    return make_uint4(low2(a[0], b[0], a[1], b[1]), low2(a[2], b[2], a[3], b[3]), low2(a[4], b[4], a[5], b[5]),
                      low2(a[6], b[6], a[7], b[7]));
}

// Eight values of G and U from their upper bits and the shared lower ones (the
// last byte repeated below itself, so that what was cut off is not biased).
__device__ __forceinline__ void restore8(uint4 g, uint4 u, uint4 low, float* gf, float* uf) {
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w}, lw[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        gf[2 * i] = __uint_as_float(__byte_perm(gw[i], lw[i], 0x1044));
        uf[2 * i] = __uint_as_float(__byte_perm(uw[i], lw[i], 0x1055));
        gf[2 * i + 1] = __uint_as_float(__byte_perm(gw[i], lw[i], 0x3266));
        uf[2 * i + 1] = __uint_as_float(__byte_perm(uw[i], lw[i], 0x3277));
    }
}

// dH with G and U, to dG and dU in their place.
template <int ACT>
__device__ __forceinline__ void gated_slopes(float dh, float& g, float& u) {
    float value, slope;
    act_both<ACT>(g, value, slope);
    g = dh * u * slope;
    u = dh * value;
}

__device__ __forceinline__ uint4 swap_lanes(uint4 v, int mask) {
    return make_uint4(__shfl_xor_sync(0xFFFFFFFFu, v.x, mask), __shfl_xor_sync(0xFFFFFFFFu, v.y, mask),
                      __shfl_xor_sync(0xFFFFFFFFu, v.z, mask), __shfl_xor_sync(0xFFFFFFFFu, v.w, mask));
}

// 32 columns of the lane's own row (row0 + lane) of a [rows, cols] array, zeros
// outside it, in two steps.  Four lanes read 64 contiguous bytes of a row, eight
// rows at a time, and a 4 x 4 exchange among them gives each its row: 16 bytes
// from each of 32 rows at a time cost the load unit four times as much.
__device__ __forceinline__ void load_rows32(const uint16_t* base, int row0, int col, int rows, int cols, uint4 (&v)[4]) {
    const int lane = threadIdx.x & 31, u = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = row0 + (lane & ~3) + i, c = col + 8 * u;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < rows && c < cols) v[i] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(row) * cols + c);
    }
}

__device__ __forceinline__ void own_row32(uint4 (&v)[4]) {
    const int u = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint4 got = swap_lanes(u & 1 ? v[i] : v[i + 1], 1);
        if (u & 1)
            v[i] = got;
        else
            v[i + 1] = got;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 got = swap_lanes(u & 2 ? v[i] : v[i + 2], 2);
        if (u & 2)
            v[i] = got;
        else
            v[i + 2] = got;
    }
}

// TN: accumulator columns of a tile, half of them from either CTA's rows of B.
template <int EPI, int ACT, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    rtlynx_gated_gemm_kernel(const __grid_constant__ GatedArgs args) {
    constexpr int kColumns = TN / 2;  // rows of B a CTA holds
    constexpr int kStageBytes = kOperandBytes + kColumns * 64 * 2;
    constexpr int kStages = kStagingBytes / kStageBytes;
    static_assert(EPI != kStore || TN == kTile, "narrow tiles are for one-product launches with an epilogue of their own");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* pieces = smem + kStagingBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(pieces + kEpiWarps * 2 * kPieceBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;  // [2]
    uint64_t* acc_empty = acc_full + 2;    // [2], used in the leader only
    uint64_t* done_bar = acc_empty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    int* err = args.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(done_bar, 1);
        fence_mbar_init();
        for (int i = 0; i < args.problems; ++i) {
            prefetch_tmap(&args.maps[args.p[i].a0]);
            prefetch_tmap(&args.maps[args.p[i].b0 + (EPI == kGatedForward ? static_cast<int>(rank) : 0)]);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, kTmemColumns);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dependency_wait();
    launch_dependents();  // the next kernel's setup may overlap this one

    const Units units(args, pair, num_pairs);
    Unit w;
    if (warp == 0) {
        // The whole warp runs the loop and one elected lane issues, so that
        // addresses, coordinates and map pointers are uniform values: the two
        // to four loads of a stage have to be issued in the 256 cycles that
        // its MMAs take.
        const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
        const uint32_t smem0 = smem_u32(smem);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto fetch = [&](auto a_major, auto b_major, const CUtensorMap* ma, const CUtensorMap* mb, int k, int stages,
                         int row0, int col0) {
            constexpr bool A_MN = decltype(a_major)::value, B_MN = decltype(b_major)::value;
            for (int i = 0; i < stages; ++i, k += 64) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, err))) {
                    ok = false;
                    break;
                }
                const uint32_t dst = smem0 + static_cast<uint32_t>(stage * kStageBytes);
                const uint32_t bar = full0 + static_cast<uint32_t>(stage) * 8u;
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(&full[stage], 2u * kStageBytes);
                    load_operand<A_MN>(dst, ma, bar, k, row0);
                    load_operand<B_MN, kColumns>(dst + kOperandBytes, mb, bar, k, col0);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        };
        for (int i = 0; ok && units.at(i, args, w); ++i) {
            const Problem& p = args.p[w.problem];
            const int row0 = w.mp * kTile + static_cast<int>(rank) * kHalf;
            const int col0 = EPI == kGatedForward ? w.nt * kColumns : w.nt * TN + static_cast<int>(rank) * kColumns;
            // one run of stages for each operand pair
            for (int seg = 0; seg < 2 && ok; ++seg) {
                const int begin = seg ? max(w.kb, p.k0) : w.kb, end = seg ? w.ke : min(w.ke, p.k0);
                const CUtensorMap* ma = &args.maps[seg ? p.a1 : p.a0];
                const CUtensorMap* mb = &args.maps[(seg ? p.b1 : p.b0) + (EPI == kGatedForward ? static_cast<int>(rank) : 0)];
                const int k = (begin - (seg ? p.k0 : 0)) * 64;
                if (EPI == kGatedForward || (EPI == kStore && !p.b_mn)) {
                    fetch(KMajor(), KMajor(), ma, mb, k, end - begin, row0, col0);
                } else if (EPI == kGatedBackward || !p.a_mn) {
                    fetch(KMajor(), MnMajor(), ma, mb, k, end - begin, row0, col0);
                } else {
                    fetch(MnMajor(), MnMajor(), ma, mb, k, end - begin, row0, col0);
                }
            }
        }
        // every stage this CTA filled has been released, so no commit arrival
        // is still on its way to this CTA
        for (int i = 0; i < kStages && ok; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, err))) break;
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // The whole warp runs the loop and one elected lane issues (see
            // gemm.cu, where this form measured 2-4% faster than one lane).
            // Stage s adds s * kStageBytes / 16 to a descriptor's address
            // field.  Within a stage an MMA's 16 K values are 32 bytes of a
            // K-major row, or 16 rows of 128 bytes of an MN-major box.
            const uint32_t smem0 = smem_u32(smem);
            int stage = 0;
            uint32_t phase = 0;
            uint64_t off = 0;
            bool ok = true;
            // the stages of one unit, operand layouts fixed at compile time so
            // that descriptors, steps and the instruction word stay constants
            // and uniform values
            auto issue = [&](auto a_major, auto b_major, uint32_t d, int stages) {
                constexpr bool A_MN = decltype(a_major)::value, B_MN = decltype(b_major)::value;
                constexpr uint32_t idesc = make_idesc_bf16(kTile, TN, false) | (A_MN ? 1u << 15 : 0u) |
                                           (B_MN ? 1u << 16 : 0u);
                // MN-major: 64-value blocks 8 KB apart, groups of eight K rows 1 KB apart
                const uint64_t desc_a = make_sdesc(smem0, A_MN ? kOperandBytes / 2 : 16, 1024, kSw128);
                const uint64_t desc_b = make_sdesc(smem0 + kOperandBytes, B_MN ? kOperandBytes / 2 : 16, 1024, kSw128);
                constexpr uint64_t step_a = A_MN ? 128 : 2, step_b = B_MN ? 128 : 2;
                constexpr uint64_t kStageStep = kStageBytes >> 4;
                for (int i = 0; i < stages; ++i) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, err))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = desc_a + off, b = desc_b + off;
                    const uint32_t acc = i != 0;
                    if (elect_one()) {
                        mma_f16_pair(d, a, b, idesc, acc);
                        mma_f16_pair(d, a + step_a, b + step_b, idesc, 1u);
                        mma_f16_pair(d, a + 2 * step_a, b + 2 * step_b, idesc, 1u);
                        mma_f16_pair(d, a + 3 * step_a, b + 3 * step_b, idesc, 1u);
                    }
                    if (elect_one()) tc_commit_pair_mc(&empty[stage], 0x3);
                    off += kStageStep;
                    if (++stage == kStages) {
                        stage = 0;
                        off = 0;
                        phase ^= 1u;
                    }
                }
            };
            for (int local = 0; ok && units.at(local, args, w); ++local) {
                const Problem& p = args.p[w.problem];
                const int buf = local & 1;
                const uint32_t use = static_cast<uint32_t>(local >> 1);
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_empty[buf], (use & 1u) ^ 1u, err))) break;
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * TN);
                if (EPI == kGatedForward || (EPI == kStore && !p.b_mn)) {
                    issue(KMajor(), KMajor(), d, w.ke - w.kb);
                } else if (EPI == kGatedBackward || !p.a_mn) {
                    issue(KMajor(), MnMajor(), d, w.ke - w.kb);
                } else {
                    issue(MnMajor(), MnMajor(), d, w.ke - w.kb);
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair_mc(&acc_full[buf], 0x3);
            }
            // every MMA of the pair has finished before tensor memory is freed
            if (elect_one()) tc_commit_pair_mc(done_bar, 0x1);
            mbar_wait(done_bar, 0, nullptr);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;          // tensor-memory lane quadrant of this warp
        const int part = (warp - 2) >> 2;   // which share of the columns
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        // A lane has 32 columns of its own row: they go out as 32 x 32 pieces
        // through shared memory (64B swizzle) and TMA, which clips the ragged
        // edges.  (Training step on 64 tokens at 5120 -> 13824, whose weights'
        // gradients are all output: 319 us; 478 with 16 bytes to each of 32 rows
        // at a time straight from the lanes, 372 with rows exchanged through
        // shared memory and plain stores.)
        uint8_t* piece = pieces + (warp - 2) * 2 * kPieceBytes;
        int turn = 0;
        auto put = [&](int map, const uint4 (&v)[4], int col, int row) {
            uint8_t* dst = piece + turn * kPieceBytes;
            if (lane == 0) bulk_wait_group_read<1>();  // the store that last used dst has read it
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(dst + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = v[q];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&args.maps[map], dst, col, row);
                bulk_commit_group();
            }
            turn ^= 1;
        };
        for (int local = 0; units.at(local, args, w); ++local) {
            const Problem& p = args.p[w.problem];
            const int buf = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1);
            const int row_in_cta = quad * 32 + lane;
            const int row0 = w.mp * kTile + static_cast<int>(rank) * kHalf + quad * 32;  // of the warp
            const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * TN) + lane_addr;
            if (!whole_warp_wait(&acc_full[buf], use & 1u, err)) break;
            tc_fence_after();
            // called once the warp has read its share of the accumulator: the
            // MMAs of the tile after next may overwrite it
            bool held = true;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                held = false;
            };
            if constexpr (EPI == kGatedForward) {
                constexpr int kCols = kColumns / (kEpiWarps / 4);
                const int c0 = part * kCols;
#pragma unroll 1
                for (int c = c0; c < c0 + kCols; c += 32) {
                    const int col = w.nt * kColumns + c;
                    if (row0 >= p.rows || col >= p.cols) break;  // the same in the whole warp
                    uint32_t g[32], v[32];
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), g);
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(kColumns + c), v);
                    tmem_ld_wait();
                    if (c + 32 >= c0 + kCols) release();
                    uint4 packed[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float h[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            h[j] = act_value<ACT>(__uint_as_float(g[8 * q + j])) * __uint_as_float(v[8 * q + j]);
                        packed[q] = pack8(h);
                    }
                    put(p.out[0], packed, col, row0);
                    if (p.out[1] >= 0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) packed[q] = high8(g + 8 * q);
                        put(p.out[1], packed, col, row0);
#pragma unroll
                        for (int q = 0; q < 4; ++q) packed[q] = high8(v + 8 * q);
                        put(p.out[2], packed, col, row0);
#pragma unroll
                        for (int q = 0; q < 4; ++q) packed[q] = low8(g + 8 * q, v + 8 * q);
                        put(p.out[3], packed, col, row0);
                    }
                }
            } else if constexpr (EPI == kGatedBackward) {
                constexpr int kCols = TN / (kEpiWarps / 4);
                const int c0 = part * kCols;
#pragma unroll 1
                for (int c = c0; c < c0 + kCols; c += 32) {
                    uint32_t r[32];
                    uint4 gp[4], up[4], lp[4];
                    const int col0 = w.nt * TN + c;
                    if (row0 >= p.rows || col0 >= p.cols) break;  // the same in the whole warp
                    load_rows32(p.in[0], row0, col0, p.rows, p.cols, gp);
                    load_rows32(p.in[1], row0, col0, p.rows, p.cols, up);
                    load_rows32(p.in[2], row0, col0, p.rows, p.cols, lp);
                    own_row32(gp);
                    own_row32(up);
                    own_row32(lp);
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), r);
                    tmem_ld_wait();
                    if (c + 32 >= c0 + kCols) release();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float gf[8], uf[8];
                        restore8(gp[q], up[q], lp[q], gf, uf);
#pragma unroll
                        for (int j = 0; j < 8; ++j) gated_slopes<ACT>(__uint_as_float(r[8 * q + j]), gf[j], uf[j]);
                        gp[q] = pack8(gf);
                        up[q] = pack8(uf);
                    }
                    put(p.out[0], gp, col0, row0);
                    put(p.out[1], up, col0, row0);
                }
            } else if (p.split > 1) {
                // this CTA's half of the fp32 partial: [column / 4][row][4]
                float* dst = p.part + (static_cast<size_t>(w.index) * 2 + rank) * (kHalf * kTile);
                constexpr int kCols = kTile / (kEpiWarps / 4);
#pragma unroll 1
                for (int c = part * kCols; c < (part + 1) * kCols; c += 32) {
                    if (row0 >= p.rows || w.nt * kTile + c >= p.cols) break;  // never read; the same in the whole warp
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        reinterpret_cast<uint4*>(dst)[(c / 4 + q) * kHalf + row_in_cta] =
                            make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
                }
            } else {
                // all of the warp's share at once, so that the accumulator is
                // free before the first piece goes out
                constexpr int kCols = kTile / (kEpiWarps / 4);
                const int c0 = part * kCols;
                uint32_t r[kCols / 32][32];
#pragma unroll
                for (int i = 0; i < kCols / 32; ++i) tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c0 + 32 * i), r[i]);
                tmem_ld_wait();
                release();
#pragma unroll
                for (int i = 0; i < kCols / 32; ++i) {
                    const int col = w.nt * kTile + c0 + 32 * i;
                    if (row0 < p.rows && col < p.cols) {  // the same in the whole warp
                        uint4 packed[4];
                        pack32(r[i], packed);
                        put(p.out[0], packed, col, row0);
                    }
                }
            }
            if (held) release();
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    __syncwarp();  // reconverge the role warps before the cluster barrier
    // after an abort, copies still in flight get time to land before the
    // shared memory they target is released
    if (error_seen(err)) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemColumns);
    }
}

// Eight columns of one row of a split tile, its parts added in order.
__device__ __forceinline__ void sum_octet(const Problem& p, int tile, int rank, int row_in_cta, int octet, float (&sum)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    for (int s = 0; s < p.split; ++s) {
        const float4* src = reinterpret_cast<const float4*>(
            p.part + ((static_cast<size_t>(tile) * p.split + s) * 2 + rank) * (kHalf * kTile));
        const float4 a = src[(2 * octet) * kHalf + row_in_cta], b = src[(2 * octet + 1) * kHalf + row_in_cta];
        sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
        sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
    }
}

// Sums the partial tiles of the split problems, and takes dH on to dG and dU
// where it is that (EPI kGatedBackward): a thread owns eight columns of one row.
// Grid: (tile * 2 + rank) x 16 x problem, with 256 threads = 2 column octets x
// 128 rows.
template <int EPI, int ACT>
__global__ void __launch_bounds__(256) rtlynx_gated_sum_parts_kernel(const __grid_constant__ GatedArgs args) {
    grid_dependency_wait();
    launch_dependents();
    const Problem& p = args.p[blockIdx.z];
    const int tile = blockIdx.x >> 1, rank = blockIdx.x & 1;
    if (p.split <= 1 || tile >= p.m_pairs * p.n_tiles) return;
    const int row_in_cta = threadIdx.x & 127, octet = blockIdx.y * 2 + (threadIdx.x >> 7);
    int mp, nt;
    tile_at(p, tile, mp, nt);
    const int row = mp * kTile + rank * kHalf + row_in_cta;
    const int col = nt * kTile + 8 * octet;
    if (row >= p.rows || col >= p.cols) return;
    const size_t at = static_cast<size_t>(row) * p.cols + col;
    const size_t to = static_cast<size_t>(row) * p.sum_pitch + col;
    auto write = [&](int i, uint4 v) { *reinterpret_cast<uint4*>(p.sum_out[i] + to) = v; };
    float f[8];
    sum_octet(p, tile, rank, row_in_cta, octet, f);
    if constexpr (EPI == kStore) {
        write(0, pack8(f));
    } else {
        auto read = [&](int i) { return *reinterpret_cast<const uint4*>(p.in[i] + at); };
        float g[8], u[8];
        restore8(read(0), read(1), read(2), g, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) gated_slopes<ACT>(f[j], g[j], u[j]);
        write(0, pack8(g));
        write(1, pack8(u));
    }
}

// ---------------------------------------------------------------- host side
template <int EPI, int ACT, int TN>
int launch_tiles(const GatedArgs& args, int num_sms, cudaStream_t stream) {
    auto kernel = rtlynx_gated_gemm_kernel<EPI, ACT, TN>;
    static std::atomic<uint64_t> smem_set{0};
    const int e = allow_max_dynamic_smem(kernel, smem_set);
    if (e) return e;
    const int most = num_sms / 2;
    const int pairs = args.units < most ? args.units : most;
    return launch_dependent(kernel, dim3(2 * pairs), dim3(kThreads), kSmemBytes, stream, args);
}

// The tiled kernel; where anything was split, the plain one, whose units
// leave partial tiles, and the sums with the epilogue asked for.  (The gate and
// up projections are never split: launch_tiles.)
template <int EPI, int ACT, int TN = kTile>
int launch_gated(const GatedArgs& args, int num_sms, cudaStream_t stream) {
    static_assert(EPI != kGatedForward, "has no sums of its own");
    int tiles = 0;
    for (int i = 0; i < args.problems; ++i)
        if (args.p[i].split > 1 && args.p[i].m_pairs * args.p[i].n_tiles > tiles) tiles = args.p[i].m_pairs * args.p[i].n_tiles;
    if (tiles == 0) return launch_tiles<EPI, ACT, TN>(args, num_sms, stream);
    const int e = launch_tiles<kStore, 0, kTile>(args, num_sms, stream);
    if (e) return e;
    return launch_dependent(rtlynx_gated_sum_parts_kernel<EPI, ACT>, dim3(2 * tiles, 16, args.problems), dim3(256), 0,
                            stream, args);
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Column tiles swept together (group_n): about sqrt(2 pairs) = 12, so that one
// wave covers 6 rows x 12 columns of tiles and reads few bytes from HBM for
// its MMAs, whatever K.  Measured against the linear layer's rule (one column,
// or as many as 48 MiB of B hold, gemm.cu), TFLOP/s: 32760 x 5120, K = 27648:
// 1520 against 1380; 8192 x 13824, K = 5120: 1540 against 1510; 13824 x 5120,
// K = 8192: 1535 against 1292 at one column.
int raster_group(const Problem& p, int pairs) {
    int width = 1;
    while ((width + 1) * (width + 1) <= 2 * pairs) ++width;
    const int groups = (p.n_tiles + width - 1) / width;
    return (p.n_tiles + groups - 1) / groups;  // groups of equal width
}

struct Maps {
    GatedArgs& args;
    int count = 0;
    bool ok = true;
    // a bf16 matrix [rows, cols], its rows `pitch` values apart, read in boxes
    // of 64 contiguous values x box_rows
    int add_pitched(const void* base, int64_t rows, int64_t cols, int64_t pitch, bool mn, int box_rows = kHalf) {
        if (encode_tmap_uncached(&args.maps[count], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, pitch * 2, 64,
                                 mn ? 64 : box_rows, CU_TENSOR_MAP_SWIZZLE_128B))
            ok = false;
        return count++;
    }
    int add(const void* base, int64_t rows, int64_t cols, bool mn, int box_rows = kHalf) {
        return add_pitched(base, rows, cols, cols, mn, box_rows);
    }
    // a bf16 output, written in 32 x 32 pieces
    int out_pitched(void* base, int64_t rows, int64_t cols, int64_t pitch) {
        if (!base) return -1;
        if (encode_tmap_uncached(&args.maps[count], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, pitch * 2, 32, 32,
                                 CU_TENSOR_MAP_SWIZZLE_64B))
            ok = false;
        return count++;
    }
    int out(void* base, int64_t rows, int64_t cols) { return out_pitched(base, rows, cols, cols); }
};

int check_sizes(int64_t M, int64_t D, int64_t F, int act) {
    if (M <= 0 || D <= 0 || F <= 0 || D % 8 || F % 8) return RTLYNX_ERR_INVALID_ARG;
    if (act != RTLYNX_ACT_SILU && act != RTLYNX_ACT_GELU) return RTLYNX_ERR_INVALID_ARG;
    // tile counts and tensor-map coordinates fit 32 bits with room
    if (M > (int64_t(1) << 28) || D > (int64_t(1) << 22) || F > (int64_t(1) << 22)) return RTLYNX_ERR_UNSUPPORTED;
    if (M / kTile * (F / kHalf) > (int64_t(1) << 28) || M / kTile * (D / kHalf) > (int64_t(1) << 28))
        return RTLYNX_ERR_UNSUPPORTED;
    return RTLYNX_OK;
}

struct Range {
    const void* p;
    uint64_t bytes;
};

// Every output range is given, 16-byte aligned, and shares no byte with an
// input or another output (null ones aside).
bool ranges_ok(const Range* in, int n_in, const Range* out, int n_out) {
    auto meet = [](const Range& a, const Range& b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
    };
    auto aligned = [](const Range& a) { return (reinterpret_cast<uintptr_t>(a.p) & 15u) == 0; };
    for (int i = 0; i < n_in; ++i)
        if (!aligned(in[i])) return false;
    for (int i = 0; i < n_out; ++i) {
        if (!aligned(out[i])) return false;
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return false;
    }
    return true;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// CTA pairs that the cutting along K reckons with (a B200's 148 SMs), whatever
// the GPU, so that workspace sizes do not depend on it.
constexpr int kPlanPairs = 74;

// Stages' worth of time that a unit costs beside its stages (filling the
// pipeline, its share of the epilogue).
constexpr int kUnitCost = 4;

size_t part_bytes(int64_t units) { return static_cast<size_t>(units) * kTile * kTile * sizeof(float); }

int64_t tiles_of(int64_t rows, int64_t cols) { return static_cast<int64_t>(ceil_div(rows, kTile)) * ceil_div(cols, kTile); }

// Most parts that `tiles` of `stages` each are cut into along K: where they are
// fewer than CTA pairs, each pair gets at most one part, of at least eight stages.
int most_parts(int64_t tiles, int64_t stages) {
    int64_t split = kPlanPairs / tiles;
    if (split > stages / 8) split = stages / 8;
    return static_cast<int>(split < 1 ? 1 : (split > 16 ? 16 : split));
}

// Y = H Wd^T of the forward call, past gated_some.cu's tokens: 1500 at 512 -> 5632
// take 44.1 us, 53.9 with the tiles whole.  (Parts of eight stages, measured
// with 64 tokens at 1024 -> 2816: 19.7 us, 22.5 with parts of 16, 20.2 with
// parts of four.)
int down_parts(int64_t M, int64_t D, int64_t F) { return most_parts(tiles_of(M, D), ceil_div(F, 64)); }

// Which kernels run the forward call.  gated_few.cu's
// - up to 8 tokens;
// - up to 16, but with weights past 128 MB those of gated_some.cu (16 tokens at
//   5120 -> 13824: 73 us against 90; at 4096 -> 11008 53 and 70; but at 2048 -> 5632
//   24.4 against 22.8);
// - up to 128 where weights and products are small (128 at 256 -> 512: 5.0 us
//   against 8.9, at 1024 -> 1024 13.1 and 14.0; 48 at 1024 -> 2816 14.3 and 16.4; but
//   17 at 1536 -> 4096 24 against 19), in about four blocks an SM at most (17 at
//   512 -> 8192 in 1024 blocks 20 us against 15).
bool few_kernels(int64_t M, int64_t D, int64_t F) {
    if (M <= 8) return true;
    if (M <= 16) return 6 * D * F <= 128000000;
    const int64_t groups = (M + 15) / 16;
    return M <= kFewTokens && 16 * groups * D * F <= 140000000 && groups * ceil_div(F, 16) <= 600;
}

// gated_some.cu's down-projection up to 512 tokens (384 at 512 -> 8192: 24.3 us
// for the call, 30.3 with the tiled one; at 4096 -> 1024 26.5 and 32.0; 256 at
// 5120 -> 13824, the worst case, 110 and 108), with small weights up to 1024 (768
// at 1024 -> 2816 23.9 and 29.0; 1024 at 5120 -> 13824 354 and 339).
bool some_down(int64_t M, int64_t D, int64_t F) { return M <= 512 || (M <= 1024 && D * F <= 12000000); }

// gated_some.cu's gate and up projections
// - where there are enough tiles of 128 channels for the SMs, and the more the
//   more tokens: half of 3 / 2 a token (64 at 5120 -> 13824: 77 us against 88, at
//   2048 -> 5632 27.9 and 28.3, but 18.4 against 16.4 at 1024 -> 2816);
// - where rows are short, so that the epilogue is what counts, and one round of
//   tiles does (128 at 512 -> 8192: 18.3 us against 21.1, 200 there 22.1 and 22.5;
//   at 2472 -> 864 25.8 against 21.4);
// - where the tiled kernel would need a second round of tiles and this one does
//   not, with 208 tokens a tile at most (384 at 2048 -> 5632: 36.1 us against 40.5,
//   160 at 5120 -> 13824 88 and 97; 256 there 114 against 110).
bool some_gate(int64_t M, int64_t D, int64_t F) {
    const int64_t tiles = ceil_div(F, 128), sms = 2 * kPlanPairs;
    if (M <= 256 && 2 * M <= 3 * tiles) return true;
    if (D <= 512) return M <= 128 || (M <= 384 && tiles * ceil_div(M, 256) <= sms);
    return M <= 512 && ceil_div(M, kTile) * tiles > kPlanPairs && tiles * ceil_div(M, 208) <= sms;
}

// Narrow tiles where rounds of them over the pairs end sooner than rounds of
// wide ones, twice as long each: with 200 tokens, 13824 columns of H are 108
// tiles for 74 pairs (two rounds) or 216 (three of half the length).
// 64 tokens at 5120 -> 13824: 92.6 us, 96.7 wide (before they had kernels of their
// own).  Past four rounds wide tiles win by
// reading X half as often (900 at 2048 -> 8192: 81 us, 88 narrow).
bool narrow_tiles(int64_t rows, int64_t wide, int64_t thin, int64_t pairs) {
    return rows * thin <= 4 * pairs && ceil_div(rows * thin, pairs) < 2 * ceil_div(rows * wide, pairs);
}

// dH = dY Wd, where that saves more than the extra kernel costs: at 95 tokens and
// 2472 -> 864 its four tiles have 39 stages each (training step 50 us, 68 with the
// tiles whole).  The gate and up projections are not cut: it made 957 tokens at
// 2000 -> 784 take 25.9 us instead of 20.9, and gained nothing elsewhere.
int dh_parts(int64_t M, int64_t D, int64_t F) {
    const int64_t stages = ceil_div(D, 64);
    return stages < 32 ? 1 : most_parts(tiles_of(M, F), stages);
}

// How the second launch of the backward call is cut: dX has few long tiles
// (K = 2 D_ff) with few tokens, the weights' gradients (K = tokens) with many
// tokens and narrow weights.  Tiles are cut only while a part is longer than
// what a CTA pair has to do on average.
struct BackwardPlan {
    int64_t x_tiles, x_stages, w_tiles, w_stages;  // of dX; of one weight's gradient
    int x_split, w_split;
    int64_t units;  // with fp32 partial tiles

    BackwardPlan(int64_t M, int64_t D, int64_t F, bool x, int weights) {
        x_tiles = x ? tiles_of(M, D) : 0;
        x_stages = 2 * ceil_div(F, 64);
        w_tiles = tiles_of(F, D);
        w_stages = ceil_div(M, 64);
        const int64_t w_all = weights * w_tiles;
        const int64_t average = (x_tiles * (x_stages + kUnitCost) + w_all * (w_stages + kUnitCost)) / kPlanPairs + 1;
        auto parts = [&](int64_t tiles, int64_t stages) {
            if (tiles == 0) return 1;
            const int64_t wanted = (stages + kUnitCost + average - 1) / average;
            const int most = most_parts(tiles, stages);
            return static_cast<int>(wanted < most ? wanted : most);
        };
        x_split = parts(x_tiles, x_stages);
        w_split = parts(w_all, w_stages);
        units = (x_split > 1 ? x_tiles * x_split : 0) + (w_split > 1 ? w_all * w_split : 0);
    }
    int64_t x_cost() const { return x_stages / x_split + kUnitCost; }  // of a unit
    int64_t w_cost() const { return w_stages / w_split + kUnitCost; }
};

struct BackwardLayout {
    size_t dg, du, part, total;
};

// Values from one row of dG and dU to the next: they live in the workspace, so
// their rows start on 128-byte lines whatever D_ff (2047 tokens at 1544 -> 4104:
// training step 276 us with rows of D_ff values, 257 like this, after pauses; 296
// to 302 like this in a long run).
int64_t hidden_pitch(int64_t F) { return (F + 63) / 64 * 64; }

// The workspace does for any choice of gradients.
BackwardLayout backward_layout(int64_t M, int64_t D, int64_t F) {
    BackwardLayout l;
    l.dg = 0;
    l.du = align256(static_cast<size_t>(M) * hidden_pitch(F) * 2);
    l.part = 2 * l.du;
    int64_t units = 0;
    const int dh = dh_parts(M, D, F);
    if (dh > 1) units = tiles_of(M, F) * dh;
    for (int x = 0; x < 2; ++x)
        for (int weights = 0; weights < 4; ++weights) {
            const int64_t u = BackwardPlan(M, D, F, x, weights).units;
            if (u > units) units = u;
        }
    l.total = l.part + part_bytes(units);
    return l;
}

}  // namespace
}  // namespace rtlynx

using namespace rtlynx;

extern "C" {

size_t rtlynx_gated_mlp_block_workspace_size(int64_t M, int64_t D, int64_t D_ff, int mode_down) {
    if (check_sizes(M, D, D_ff, RTLYNX_ACT_SILU) || few_kernels(M, D, D_ff)) return 0;
    if (mode_down != RTLYNX_MODE_DENSE_SKIP) return 0;
    if (some_down(M, D, D_ff)) {
        const int split = down_some_parts(M, D, D_ff);
        return split > 1 ? align256(static_cast<size_t>(split) * M * D * sizeof(float)) : 0;
    }
    const int split = down_parts(M, D, D_ff);
    return split > 1 ? part_bytes(tiles_of(M, D) * split) : 0;
}

int rtlynx_gated_mlp_block(const void* X, const void* W_gate, const void* W_up, const void* W_down,
                           const void* LA_down, const void* LB_down, void* G, void* U, void* low, void* H, void* Y, int64_t M,
                           int64_t D, int64_t D_ff, int64_t R, int act, int mode_down, void* workspace,
                           size_t ws_bytes, void* stream_) {
    int rc = check_sizes(M, D, D_ff, act);
    if (rc) return rc;
    if (!X || !W_gate || !W_up || !W_down || !H || !Y || (G == nullptr) != (U == nullptr) ||
        (G == nullptr) != (low == nullptr))
        return RTLYNX_ERR_INVALID_ARG;
    rc = validate(H, W_down, LA_down, LB_down, Y, M, D_ff, D, R, mode_down);
    if (rc) return rc;
    const bool sparse = mode_down == RTLYNX_MODE_SPARSE;
    const size_t need = sparse ? rtlynx_workspace_size(M, D_ff, D, R, mode_down)
                               : rtlynx_gated_mlp_block_workspace_size(M, D, D_ff, mode_down);
    if (need > 0 && (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return RTLYNX_ERR_INVALID_ARG;
    const uint64_t x_bytes = 2ull * M * D, h_bytes = 2ull * M * D_ff, w_bytes = 2ull * D * D_ff;
    const bool lora = sparse && R > 0;
    const Range in[6] = {{X, x_bytes},
                         {W_gate, w_bytes},
                         {W_up, w_bytes},
                         {W_down, w_bytes},
                         {lora ? LA_down : nullptr, 2ull * D * (lora ? R : 0)},
                         {lora ? LB_down : nullptr, 2ull * D_ff * (lora ? R : 0)}};
    const Range out[6] = {{H, h_bytes}, {Y, x_bytes}, {G, h_bytes}, {U, h_bytes}, {low, h_bytes},
                          {need ? workspace : nullptr, need}};
    if (!ranges_ok(in, 6, out, 6)) return RTLYNX_ERR_INVALID_ARG;
    int num_sms = 0;
    int* err = nullptr;
    rc = device_info(&num_sms, &err);
    if (rc) return rc;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const int pairs = num_sms / 2;
    if (few_kernels(M, D, D_ff)) {
        if (launch_gated_few(X, W_gate, W_up, H, G, U, low, static_cast<int>(M), static_cast<int>(D),
                             static_cast<int>(D_ff), act, stream))
            return RTLYNX_ERR_CUDA;
        if (sparse)
            return rtlynx_linear_ws(H, W_down, LA_down, LB_down, Y, M, D_ff, D, R, mode_down, workspace, ws_bytes,
                                    stream_);
        return launch_down_few(H, W_down, Y, static_cast<int>(M), static_cast<int>(D_ff), static_cast<int>(D), stream)
                   ? RTLYNX_ERR_CUDA
                   : RTLYNX_OK;
    }
    if (some_gate(M, D, D_ff)) {
        if (launch_gated_some(X, W_gate, W_up, H, G, U, low, M, D, D_ff, act, err, stream)) return RTLYNX_ERR_CUDA;
    } else {
        GatedArgs args{};
        Maps maps{args};
        args.problems = 1;
        args.err = err;
        Problem& p = args.p[0];
        p.m_pairs = ceil_div(M, kTile);
        const bool narrow = narrow_tiles(p.m_pairs, ceil_div(D_ff, kHalf), ceil_div(D_ff, kNarrow / 2), pairs);
        const int columns = narrow ? kNarrow / 2 : kHalf;
        p.n_tiles = ceil_div(D_ff, columns);
        p.split = 1;
        p.k0 = p.k = ceil_div(D, 64);
        p.a0 = p.a1 = maps.add(X, M, D, false);
        p.b0 = p.b1 = maps.add(W_gate, D_ff, D, false, columns);
        maps.add(W_up, D_ff, D, false, columns);
        p.out[0] = maps.out(H, M, D_ff);
        p.out[1] = maps.out(G, M, D_ff);
        p.out[2] = maps.out(U, M, D_ff);
        p.out[3] = maps.out(low, M, D_ff);
        if (!maps.ok) return RTLYNX_ERR_CUDA;
        p.group_n = raster_group(p, pairs);
        p.rows = static_cast<int>(M);
        p.cols = static_cast<int>(D_ff);
        args.units = p.m_pairs * p.n_tiles;
        int e;
        if (act == RTLYNX_ACT_SILU)
            e = narrow ? launch_tiles<kGatedForward, RTLYNX_ACT_SILU, kNarrow>(args, num_sms, stream)
                       : launch_tiles<kGatedForward, RTLYNX_ACT_SILU, kTile>(args, num_sms, stream);
        else
            e = narrow ? launch_tiles<kGatedForward, RTLYNX_ACT_GELU, kNarrow>(args, num_sms, stream)
                       : launch_tiles<kGatedForward, RTLYNX_ACT_GELU, kTile>(args, num_sms, stream);
        if (e) return RTLYNX_ERR_CUDA;
    }
    if (sparse)
        return rtlynx_linear_ws(H, W_down, LA_down, LB_down, Y, M, D_ff, D, R, mode_down, workspace, ws_bytes, stream_);
    if (some_down(M, D, D_ff))
        return launch_down_some(H, W_down, Y, static_cast<float*>(workspace), M, D_ff, D, err, stream) ? RTLYNX_ERR_CUDA
                                                                                                       : RTLYNX_OK;
    GatedArgs args{};
    Maps maps{args};
    args.problems = 1;
    args.err = err;
    Problem& p = args.p[0];
    p.m_pairs = ceil_div(M, kTile);
    p.n_tiles = ceil_div(D, kTile);
    p.split = down_parts(M, D, D_ff);
    p.part = static_cast<float*>(workspace);
    p.k0 = p.k = ceil_div(D_ff, 64);
    p.a0 = p.a1 = maps.add(H, M, D_ff, false);
    p.b0 = p.b1 = maps.add(W_down, D, D_ff, false);
    p.out[0] = maps.out(Y, M, D);
    p.sum_out[0] = static_cast<uint16_t*>(Y);
    p.sum_pitch = static_cast<int>(D);
    if (!maps.ok) return RTLYNX_ERR_CUDA;
    p.group_n = raster_group(p, pairs);
    p.rows = static_cast<int>(M);
    p.cols = static_cast<int>(D);
    args.units = p.m_pairs * p.n_tiles * p.split;
    return launch_gated<kStore, 0>(args, num_sms, stream) ? RTLYNX_ERR_CUDA : RTLYNX_OK;
}

size_t rtlynx_gated_mlp_backward_workspace_size(int64_t M, int64_t D, int64_t D_ff) {
    if (check_sizes(M, D, D_ff, RTLYNX_ACT_SILU)) return 0;
    return backward_layout(M, D, D_ff).total;
}

int rtlynx_gated_mlp_backward(const void* dY, const void* X, const void* W_gate, const void* W_up, const void* W_down,
                              const void* G, const void* U, const void* low, const void* H, void* dX, void* dW_gate, void* dW_up,
                              void* dW_down, int64_t M, int64_t D, int64_t D_ff, int act, void* workspace,
                              size_t ws_bytes, void* stream_) {
    int rc = check_sizes(M, D, D_ff, act);
    if (rc) return rc;
    if (!dY || !X || !W_gate || !W_up || !W_down || !G || !U || !low || !H || !workspace)
         return RTLYNX_ERR_INVALID_ARG;
    const BackwardLayout l = backward_layout(M, D, D_ff);
    if (ws_bytes < l.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return RTLYNX_ERR_INVALID_ARG;
    const uint64_t x_bytes = 2ull * M * D, h_bytes = 2ull * M * D_ff, w_bytes = 2ull * D * D_ff;
    const Range in[9] = {{dY, x_bytes}, {X, x_bytes}, {W_gate, w_bytes}, {W_up, w_bytes}, {W_down, w_bytes},
                         {G, h_bytes},  {U, h_bytes}, {low, h_bytes},    {H, h_bytes}};
    const Range out[5] = {{dX, x_bytes}, {dW_gate, w_bytes}, {dW_up, w_bytes}, {dW_down, w_bytes}, {workspace, l.total}};
    if (!ranges_ok(in, 9, out, 5)) return RTLYNX_ERR_INVALID_ARG;
    if (!dX && !dW_gate && !dW_up && !dW_down) return RTLYNX_OK;
    int num_sms = 0;
    int* err = nullptr;
    rc = device_info(&num_sms, &err);
    if (rc) return rc;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    uint16_t* dG = reinterpret_cast<uint16_t*>(base + l.dg);
    uint16_t* dU = reinterpret_cast<uint16_t*>(base + l.du);

    const int64_t h_pitch = hidden_pitch(D_ff);
    const int m_pairs = ceil_div(M, kTile), token_stages = ceil_div(M, 64);
    if (dX || dW_gate || dW_up) {
        // dH = dY Wd, taken to dG and dU before it leaves the chip
        GatedArgs args{};
        Maps maps{args};
        args.problems = 1;
        args.err = err;
        Problem& p = args.p[0];
        p.m_pairs = m_pairs;
        p.split = dh_parts(M, D, D_ff);
        // narrow tiles by the forward call's rule
        const bool narrow = p.split == 1 && narrow_tiles(m_pairs, ceil_div(D_ff, kTile), ceil_div(D_ff, kNarrow), num_sms / 2);
        p.n_tiles = ceil_div(D_ff, narrow ? kNarrow : kTile);
        p.part = reinterpret_cast<float*>(base + l.part);
        p.k0 = p.k = ceil_div(D, 64);
        p.a0 = p.a1 = maps.add(dY, M, D, false);
        p.b0 = p.b1 = maps.add(W_down, D, D_ff, true);
        p.b_mn = 1;
        p.out[0] = maps.out_pitched(dG, M, D_ff, h_pitch);
        p.out[1] = maps.out_pitched(dU, M, D_ff, h_pitch);
        p.sum_out[0] = dG;
        p.sum_out[1] = dU;
        p.sum_pitch = static_cast<int>(h_pitch);
        if (!maps.ok) return RTLYNX_ERR_CUDA;
        p.group_n = raster_group(p, num_sms / 2);
        p.rows = static_cast<int>(M);
        p.cols = static_cast<int>(D_ff);
        p.in[0] = static_cast<const uint16_t*>(G);
        p.in[1] = static_cast<const uint16_t*>(U);
        p.in[2] = static_cast<const uint16_t*>(low);
        args.units = p.m_pairs * p.n_tiles * p.split;
        int e;
        if (act == RTLYNX_ACT_SILU)
            e = narrow ? launch_gated<kGatedBackward, RTLYNX_ACT_SILU, kNarrow>(args, num_sms, stream)
                       : launch_gated<kGatedBackward, RTLYNX_ACT_SILU>(args, num_sms, stream);
        else
            e = narrow ? launch_gated<kGatedBackward, RTLYNX_ACT_GELU, kNarrow>(args, num_sms, stream)
                       : launch_gated<kGatedBackward, RTLYNX_ACT_GELU>(args, num_sms, stream);
        if (e) return RTLYNX_ERR_CUDA;
    }

    GatedArgs args{};
    Maps maps{args};
    args.err = err;
    const int pairs = num_sms / 2;
    auto close = [&](Problem& p, int64_t rows, int64_t cols, void* out) {
        p.m_pairs = ceil_div(rows, kTile);
        p.n_tiles = ceil_div(cols, kTile);
        p.rows = static_cast<int>(rows);
        p.cols = static_cast<int>(cols);
        p.out[0] = maps.out(out, rows, cols);
        p.sum_out[0] = static_cast<uint16_t*>(out);
        p.sum_pitch = static_cast<int>(cols);
        p.group_n = raster_group(p, pairs);
        p.first_unit = args.units;
        args.units += p.m_pairs * p.n_tiles * p.split;
        ++args.problems;
    };
    const int weights = (dW_gate != nullptr) + (dW_up != nullptr) + (dW_down != nullptr);
    const BackwardPlan plan(M, D, D_ff, dX != nullptr, weights);
    float* part = reinterpret_cast<float*>(base + l.part);
    auto parts_of = [&](Problem& p, int64_t tiles, int split) {
        p.split = split;
        p.part = part;
        if (split > 1) part += part_bytes(tiles * split) / sizeof(float);
    };
    auto add_dx = [&]() {
        if (!dX) return;
        Problem& p = args.p[args.problems];
        p.k0 = ceil_div(D_ff, 64);
        p.k = 2 * p.k0;
        p.a0 = maps.add_pitched(dG, M, D_ff, h_pitch, false);
        p.b0 = maps.add(W_gate, D_ff, D, true);
        p.a1 = maps.add_pitched(dU, M, D_ff, h_pitch, false);
        p.b1 = maps.add(W_up, D_ff, D, true);
        p.b_mn = 1;
        parts_of(p, plan.x_tiles, plan.x_split);
        close(p, M, D, dX);
    };
    auto weight_grad = [&](const void* a, int64_t a_cols, int64_t a_pitch, const void* b, int64_t b_cols, void* out) {
        if (!out) return;
        Problem& p = args.p[args.problems];
        p.k0 = p.k = token_stages;
        p.a0 = p.a1 = maps.add_pitched(a, M, a_cols, a_pitch, true);
        p.b0 = p.b1 = maps.add(b, M, b_cols, true);
        p.a_mn = p.b_mn = 1;
        parts_of(p, plan.w_tiles, plan.w_split);
        close(p, a_cols, b_cols, out);
    };
    auto add_weights = [&]() {
        weight_grad(dG, D_ff, h_pitch, X, D, dW_gate);
        weight_grad(dU, D_ff, h_pitch, X, D, dW_up);
        weight_grad(dY, D, D, H, D_ff, dW_down);
    };
    // The longer units first; see Units for what the pairs with one of them
    // less take instead.
    const bool x_first = plan.x_cost() >= plan.w_cost();
    if (x_first) add_dx(); else add_weights();
    args.longs = args.units;
    if (x_first) add_weights(); else add_dx();
    if (!maps.ok) return RTLYNX_ERR_CUDA;
    const int rest = args.longs % pairs;
    if (rest > 0) {
        const int64_t extra = x_first ? plan.x_cost() / plan.w_cost() : plan.w_cost() / plan.x_cost();
        const int64_t fair = (args.units - args.longs + pairs - rest - 1) / (pairs - rest);
        args.extra = static_cast<int>(extra < fair ? extra : fair);
    }
    return launch_gated<kStore, 0>(args, num_sms, stream) ? RTLYNX_ERR_CUDA : RTLYNX_OK;
}

}  // extern "C"
