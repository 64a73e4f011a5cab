// The gated feed-forward block for some tokens: too many for gated_few.cu,
// too few to fill the tiles of gated.cu.
//
// The weights' bytes still bound it, so they take the MMA's long side: a CTA
// computes D[128 weight rows, tokens], the weights are the A operand (128 rows
// of 64 K values a stage, of both Wg and Wu in the first kernel), the tokens
// its B (N = tokens rounded up to 16, 256 at most).  Nearly all of shared memory
// holds weights on their way, 32 KB a stage for 64 tokens' 8 KB, which is what
// keeps HBM busy: a CTA pair of gated.cu has 128 KB in flight of which it can use
// half, here every SM has up to 160 KB.  Wg's and Wu's products for the same rows
// lie in the same tensor-memory lanes, so the activation needs no exchange.
//
// Measured at 5120 -> 13824 (424.7 MB of weights, 64.9 us at the measured copy
// rate): 17 tokens 73 us, 64 tokens 76, 128 tokens 82, 200 tokens 99; with
// gated.cu's kernels 92, 97, 103 and 105.  At 2048 -> 5632: 129 tokens 29.6 us, 384
// 36.1; with gated.cu's kernels 37.4 and 45.9.
//
// One output tile a CTA.  The second kernel's tiles are cut along K so that
// every SM has a part; the parts are left in fp32 in the caller's workspace and
// added in order.  Where SMs are left, several CTAs share a tile's tokens (256
// tokens at 384 -> 1024: 11.0 us, 14.2 with all tokens in one).  The second kernel
// requests its first weights before the first kernel has finished.
#include "../../include/rtlynx.h"
#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace rtlynx {
namespace {

constexpr int kSomeThreads = 64 + 512;           // at most: loads, MMAs, sixteen warps of epilogue
constexpr int kRows = 128;                       // weight rows of a tile
constexpr int kWeightBytes = kRows * 64 * 2;     // of one weight, a stage
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 220 * 1024;
constexpr int kSomeSmem = kRingBytes + 1024 + 1024;
static_assert(kSomeSmem <= 232448, "shared memory budget");

struct SomeArgs {
    CUtensorMap w[2], x;
    uint16_t* out[4];  // [tokens, rows]: H, G, U, low (the last three may be null, see gated.cu); or the one output
    float* part;       // [split][tokens, rows] where K is cut
    int tokens, rows;
    int n;             // tokens of a CTA, a multiple of 16
    int k, split;      // stages of a row, parts they are cut into
    int ring, columns; // pipeline stages; tensor-memory columns
    int* err;
};

template <bool GATED, int ACT>
__global__ void __launch_bounds__(kSomeThreads, 1) rtlynx_gated_some_kernel(const __grid_constant__ SomeArgs args) {
    constexpr int kMats = GATED ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes);
    uint64_t* empty = full + kMaxStages;
    uint64_t* done = empty + kMaxStages;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * kRows;
    const int part = blockIdx.y;
    const int token0 = blockIdx.z * args.n;
    const int kb = part * args.k / args.split, ke = (part + 1) * args.k / args.split;
    const uint32_t stage_bytes = static_cast<uint32_t>(kMats * kWeightBytes + args.n * 128);
    int* err = args.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < args.ring; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&args.w[0]);
        if (GATED) prefetch_tmap(&args.w[1]);
        prefetch_tmap(&args.x);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, static_cast<uint32_t>(args.columns));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    if (warp == 0) {
        auto weights = [&](int stage, int kt) {
            uint8_t* dst = smem + stage * stage_bytes;
            mbar_arrive_expect_tx(&full[stage], stage_bytes);
            tma_load_2d(dst, &args.w[0], &full[stage], kt * 64, row0);
            if (GATED) tma_load_2d(dst + kWeightBytes, &args.w[1], &full[stage], kt * 64, row0);
        };
        auto tokens = [&](int stage, int kt) {
            tma_load_2d(smem + stage * stage_bytes + kMats * kWeightBytes, &args.x, &full[stage], kt * 64, token0);
        };
        const int ahead = min(args.ring, ke - kb);
        if constexpr (GATED) {
            // what came before this call has finished: the kernel that follows
            // may start, and read all but this kernel's outputs
            grid_dependency_wait();
            launch_dependents();
        } else if (lane == 0) {
            // follows the gated kernel, which does not write these weights
            for (int s = 0; s < ahead; ++s) weights(s, kb + s);
        }
        if constexpr (!GATED) {
            grid_dependency_wait();
            launch_dependents();
            if (lane == 0)
                for (int s = 0; s < ahead; ++s) tokens(s, kb + s);
        }
        __syncwarp();
        int stage = GATED || ahead == args.ring ? 0 : ahead;
        uint32_t phase = !GATED && ahead == args.ring ? 1u : 0u;
        for (int kt = GATED ? kb : kb + ahead; kt < ke; ++kt) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, err))) break;
            if (elect_one()) {
                weights(stage, kt);
                tokens(stage, kt);
            }
            if (++stage == args.ring) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        // (see gemm.cu: the whole warp runs the loop, one elected lane issues)
        const uint32_t idesc = make_idesc_bf16(kRows, args.n, false);
        const uint32_t smem0 = smem_u32(smem);
        const uint64_t desc_w = make_sdesc(smem0, 16, 1024, kSw128);
        const uint64_t desc_x = make_sdesc(smem0 + kMats * kWeightBytes, 16, 1024, kSw128);
        const uint64_t step = stage_bytes >> 4;
        int stage = 0;
        uint32_t phase = 0;
        uint64_t off = 0;
        for (int kt = kb; kt < ke; ++kt) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, err))) break;
            tc_fence_after();
            const uint64_t w = desc_w + off, x = desc_x + off;
            const uint32_t acc = kt != kb;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_f16(tmem_base, w + 2 * i, x + 2 * i, idesc, i > 0 ? 1u : acc);
                    if (GATED)
                        mma_f16(tmem_base + static_cast<uint32_t>(args.n), w + (kWeightBytes >> 4) + 2 * i, x + 2 * i, idesc,
                                i > 0 ? 1u : acc);
                }
            }
            if (elect_one()) tc_commit(&empty[stage]);
            off += step;
            if (++stage == args.ring) {
                stage = 0;
                off = 0;
                phase ^= 1u;
            }
        }
        if (elect_one()) tc_commit(done);
        mbar_wait(done, 0, nullptr);
        __syncwarp();
    } else {
        grid_dependency_wait();  // the outputs may be what an earlier kernel reads
        const int quad = warp & 3;
        const int row = row0 + quad * 32 + lane;
        const uint32_t acc = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        uint32_t ok = 0;
        if (lane == 0) ok = mbar_wait(done, 0, err) ? 1u : 0u;
        if (__shfl_sync(0xFFFFFFFFu, ok, 0) && !error_seen(err)) {
            tc_fence_after();
            // sixteen tokens at a time, shared out over the two or four warps of
            // a quadrant; the warp's lanes are consecutive channels, so each
            // token's store is 64 contiguous bytes
            const int round = static_cast<int>(blockDim.x - 64) / 8;
            const int tokens = min(args.n, args.tokens - token0);
            const size_t first = static_cast<size_t>(token0) * args.rows + row;
            float* const out_part = GATED ? nullptr : args.part + static_cast<size_t>(part) * args.tokens * args.rows;
            for (int t0 = 16 * ((warp - 2) >> 2); t0 < tokens; t0 += round) {
                size_t at = first + static_cast<size_t>(t0) * args.rows;
                uint32_t g[16], u[16];
                tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(t0), g);
                if (GATED) tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(args.n + t0), u);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j, at += args.rows) {
                    if (t0 + j >= tokens || row >= args.rows) continue;
                    const float v = __uint_as_float(g[j]);
                    if constexpr (GATED) {
                        args.out[0][at] = __bfloat16_as_ushort(__float2bfloat16_rn(act_value<ACT>(v) * __uint_as_float(u[j])));
                        if (args.out[1]) {
                            args.out[1][at] = static_cast<uint16_t>(g[j] >> 16);
                            args.out[2][at] = static_cast<uint16_t>(u[j] >> 16);
                            args.out[3][at] = static_cast<uint16_t>((g[j] >> 8 & 0xFFu) | (u[j] & 0xFF00u));
                        }
                    } else if (args.split > 1) {
                        out_part[at] = v;
                    } else {
                        args.out[0][at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                    }
                }
            }
            tc_fence_before();
        }
    }

    __syncwarp();
    // after an abort, copies still in flight get time to land before the
    // shared memory they target is released
    if (error_seen(err)) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, static_cast<uint32_t>(args.columns));
    }
}

// Adds the parts in order and rounds; a thread owns eight channels of a token.
__global__ void __launch_bounds__(256) rtlynx_gated_some_sum_kernel(const float* part, uint16_t* out, int split, int64_t n) {
    grid_dependency_wait();
    launch_dependents();
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    float sum[8] = {};
    for (int s = 0; s < split; ++s) {
        const float4* src = reinterpret_cast<const float4*>(part + s * n + i);
        const float4 a = src[0], b = src[1];
        sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
        sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
    }
    *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]),
                                                     pack_bf16x2(sum[4], sum[5]), pack_bf16x2(sum[6], sum[7]));
}

// How many CTAs share the tokens of one tile of rows: while there are SMs left,
// so that the epilogue, which no other tile's main loop hides, is spread over
// them.  No fewer than 32 tokens each, one round of the epilogue's eight warps,
// and no more than the MMA takes.
int64_t least_groups(int64_t tokens) { return (tokens + 255) / 256; }
int token_groups(int64_t tokens, int64_t tiles) {
    const int64_t least = least_groups(tokens), most = (tokens + 31) / 32, fill = 148 / tiles;
    return static_cast<int>(fill < least ? least : (fill < most ? fill : most));
}

template <bool GATED, int ACT>
int launch_some(SomeArgs& args, const void* x, const void* w0, const void* w1, int64_t tokens, int64_t rows, int64_t K,
                int split, int groups, cudaStream_t stream) {
    auto kernel = rtlynx_gated_some_kernel<GATED, ACT>;
    static std::atomic<uint64_t> smem_set{0};
    int e = allow_max_dynamic_smem(kernel, smem_set);
    if (e) return e;
    constexpr int kMats = GATED ? 2 : 1;
    args.tokens = static_cast<int>(tokens);
    args.rows = static_cast<int>(rows);
    const int64_t sixteens = (tokens + 15) / 16;
    args.n = static_cast<int>((sixteens + groups - 1) / groups * 16);
    args.k = static_cast<int>((K + 63) / 64);
    args.split = split;
    const int stage = kMats * kWeightBytes + args.n * 128;
    args.ring = kRingBytes / stage < kMaxStages ? kRingBytes / stage : kMaxStages;
    args.columns = 32;
    while (args.columns < kMats * args.n) args.columns *= 2;
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
    e = encode_tmap_uncached(&args.w[0], type, w0, K, rows, K * 2, 64, kRows, swizzle);
    if (!e && GATED) e = encode_tmap_uncached(&args.w[1], type, w1, K, rows, K * 2, 64, kRows, swizzle);
    if (!e) e = encode_tmap_uncached(&args.x, type, x, K, tokens, K * 2, 64, args.n, swizzle);
    if (e) return e;
    const dim3 grid(static_cast<unsigned>((rows + kRows - 1) / kRows), split,
                    static_cast<unsigned>((tokens + args.n - 1) / args.n));
    // Eight epilogue warps, sixteen from 64 tokens on: 128 tokens at 512 -> 8192
    // take 18.2 us, 20.2 with eight; 17 at 2048 -> 5632 24.9, 26.0 with sixteen.
    const int threads = args.n >= 64 ? kSomeThreads : 64 + 256;
    return launch_dependent(kernel, grid, dim3(threads), kSomeSmem, stream, args);
}

}  // namespace

int launch_gated_some(const void* X, const void* W_gate, const void* W_up, void* H, void* G, void* U, void* low, int64_t M,
                      int64_t D, int64_t D_ff, int act, int* err, cudaStream_t stream) {
    SomeArgs args{};
    args.out[0] = static_cast<uint16_t*>(H);
    args.out[1] = static_cast<uint16_t*>(G);
    args.out[2] = static_cast<uint16_t*>(U);
    args.out[3] = static_cast<uint16_t*>(low);
    args.err = err;
    const int groups = token_groups(M, (D_ff + kRows - 1) / kRows);
    return act == RTLYNX_ACT_SILU ? launch_some<true, RTLYNX_ACT_SILU>(args, X, W_gate, W_up, M, D_ff, D, 1, groups, stream)
                                  : launch_some<true, RTLYNX_ACT_GELU>(args, X, W_gate, W_up, M, D_ff, D, 1, groups, stream);
}

int down_some_parts(int64_t M, int64_t D, int64_t D_ff) {
    const int64_t ctas = (D + kRows - 1) / kRows * least_groups(M), stages = (D_ff + 63) / 64;
    // parts of twelve stages at least (384 tokens at 512 -> 8192: 24.3 us, 26.1 with
    // eight, 24.6 with sixteen; 64 at 2048 -> 5632 25.1, 26.4 and 25.7)
    int64_t split = 148 / ctas;
    if (split > stages / 12) split = stages / 12;
    return static_cast<int>(split < 1 ? 1 : (split > 16 ? 16 : split));
}

int launch_down_some(const void* H, const void* W_down, void* Y, float* part, int64_t M, int64_t D_ff, int64_t D, int* err,
                     cudaStream_t stream) {
    SomeArgs args{};
    args.out[0] = static_cast<uint16_t*>(Y);
    args.part = part;
    args.err = err;
    const int split = down_some_parts(M, D, D_ff);
    const int e = launch_some<false, 0>(args, H, W_down, nullptr, M, D, D_ff, split,
                                        token_groups(M, (D + kRows - 1) / kRows * split), stream);
    if (e || split == 1) return e;
    const int64_t n = M * D;
    return launch_dependent(rtlynx_gated_some_sum_kernel, dim3(static_cast<unsigned>((n / 8 + 255) / 256)), dim3(256), 0,
                            stream, static_cast<const float*>(part), static_cast<uint16_t*>(Y), split, n);
}

}  // namespace rtlynx
