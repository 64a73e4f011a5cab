// The gated feed-forward block for a few tokens.
//
// With a handful of tokens the block reads 6 D D_ff bytes of weights and does
// little else, so HBM bounds it, and the tiles of the many-token kernel
// (gated.cu, 256 rows by 256 columns a CTA pair) are both too empty and too
// few: 13824 channels make 108 tiles for 74 pairs, 5120 make 20.  Here a block
// takes 16 output channels and all K; its warps deal the K chunks out between
// them, so 864 and 320 blocks keep every SM reading.
//
// The weights are the MMA's A operand (m16n8k16, 16 channels), the tokens its
// B.  The MMA's K order is free as long as both operands share it, so a lane
// reads 16 contiguous bytes of each row: of a chunk of 32 K values lane
// (g, t) holds values 8t .. 8t + 7 of rows g and g + 8, which are the operands
// of two MMAs.  Weights go straight from global memory to registers, each byte
// once, with all loads of kUnroll chunks in flight before the first MMA.  At
// this rate the legacy MMA is no limit: 1 KB of weights per MMA pair.
//
// The warps' fp32 sums meet in shared memory and are added in warp order.
//
// Small weights stay in L2, and then more tokens do as well: blocks of 16 tokens
// each, side by side, reading the same weights (64 tokens at 256 -> 512: 4.9 us,
// 8.9 with gated_some.cu's kernels; 32 at 2472 -> 864 9.7 and 18.0).
//
// Measured at D = 5120, D_ff = 13824 (424.7 MB of weights, 64.9 us at the
// measured copy rate): 1 token 67 us (6.4 TB/s), 8 tokens 69; 16 tokens 88, as a
// block re-reads the tokens from L2 half as often as it reads weights, which is
// where gated_some.cu takes over.  11 tokens at 2056 -> 5512: 20.8 us.
#include "../../include/rtlynx.h"
#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace rtlynx {
namespace {

constexpr int kFewRows = 16;  // output channels of a block

struct FewArgs {
    const uint16_t* x;      // [M, K]
    const uint16_t* w[2];   // [N, K]: gate and up, or the one matrix
    uint16_t* out[4];       // [M, N]: H, G, U, low (the last three may be null, see gated.cu), or the one output
    int M, N, K;
};

// Not the read-only path: this kernel may have been launched while the one
// that writes its weights was still running.
__device__ __forceinline__ uint4 load_weights(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// GATED: two matrices, act(first) * second; otherwise the one product.
// TILES: a block's tokens in eights.  WARPS: warps of a block.  BLOCKS: resident on
// an SM, which settles the registers of a thread.
template <bool GATED, int TILES, int ACT, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS) rtlynx_gated_few_kernel(const FewArgs args) {
    constexpr int kFewWarps = WARPS, kFewThreads = 32 * WARPS;
    constexpr int kMats = GATED ? 2 : 1;
    constexpr int kUnroll = GATED ? 2 : 4;
    constexpr int kSums = kMats * TILES * 4;
    __shared__ float sums[kFewWarps][kSums][32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int row0 = blockIdx.x * kFewRows + g;
    const int token0 = blockIdx.y * 8 * TILES, tokens = args.M - token0;
    const uint16_t* const x0 = args.x + static_cast<size_t>(token0) * args.K;
    const bool row_ok[2] = {row0 < args.N, row0 + 8 < args.N};
    const size_t row_at[2] = {static_cast<size_t>(row0) * args.K, static_cast<size_t>(row0 + 8) * args.K};
    const int chunks = (args.K + 31) / 32;

    float c[kMats][TILES][4];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int n = 0; n < TILES; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[m][n][j] = 0.0f;

    uint4 w[kUnroll][kMats][2];
    auto fetch_weights = [&](int first) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = (first + u * kFewWarps) * 32 + 8 * t;
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[u][m][h] = make_uint4(0, 0, 0, 0);
                    if (row_ok[h] && k < args.K) w[u][m][h] = load_weights(args.w[m] + row_at[h] + k);
                }
        }
    };
    if constexpr (GATED) {
        // Whatever came before this call has finished here, so the kernel that
        // follows may start and read all but this kernel's outputs.
        grid_dependency_wait();
        launch_dependents();
        fetch_weights(warp);
    } else {
        // Follows the gated kernel, which does not write these weights: the
        // first of them are on their way while it drains.
        fetch_weights(warp);
        grid_dependency_wait();
    }

    for (int first = warp; first < chunks; first += kUnroll * kFewWarps) {
        uint4 x[kUnroll][TILES];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = (first + u * kFewWarps) * 32 + 8 * t;
#pragma unroll
            for (int n = 0; n < TILES; ++n) {
                const int token = 8 * n + g;
                x[u][n] = make_uint4(0, 0, 0, 0);
                if (token < tokens && k < args.K)
                    x[u][n] = *reinterpret_cast<const uint4*>(x0 + static_cast<size_t>(token) * args.K + k);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                    mma_16816(c[m][n], w[u][m][0].x, w[u][m][1].x, w[u][m][0].y, w[u][m][1].y, x[u][n].x, x[u][n].y);
                    mma_16816(c[m][n], w[u][m][0].z, w[u][m][1].z, w[u][m][0].w, w[u][m][1].w, x[u][n].z, x[u][n].w);
                }
        fetch_weights(first + kUnroll * kFewWarps);
    }

#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int n = 0; n < TILES; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[warp][(m * TILES + n) * 4 + j][lane] = c[m][n][j];
    __syncthreads();
    // thread -> (token, channel), channels fastest; in the accumulators channel
    // g (+ 8) and token 2 t (+ 1) of a tile are lane (g, t), element 2 (+ 1)
    for (int i = threadIdx.x; i < kFewRows * 8 * TILES; i += kFewThreads) {
        const int ch = i % kFewRows, token = i / kFewRows;
        const int n = token / 8, col = token % 8;
        const int from = (ch % 8) * 4 + col / 2, j = (ch / 8) * 2 + col % 2;
        const int row = blockIdx.x * kFewRows + ch;
        if (token >= tokens || row >= args.N) continue;
        float total[kMats];
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            total[m] = 0.0f;
#pragma unroll
            for (int k = 0; k < kFewWarps; ++k) total[m] += sums[k][(m * TILES + n) * 4 + j][from];
        }
        const size_t at = static_cast<size_t>(token0 + token) * args.N + row;
        if constexpr (GATED) {
            args.out[0][at] = __bfloat16_as_ushort(__float2bfloat16_rn(act_value<ACT>(total[0]) * total[1]));
            if (args.out[1]) {
                const uint32_t gate = __float_as_uint(total[0]), up = __float_as_uint(total[1]);
                args.out[1][at] = static_cast<uint16_t>(gate >> 16);
                args.out[2][at] = static_cast<uint16_t>(up >> 16);
                args.out[3][at] = static_cast<uint16_t>((gate >> 8 & 0xFFu) | (up & 0xFF00u));
            }
        } else {
            args.out[0][at] = __bfloat16_as_ushort(__float2bfloat16_rn(total[0]));
        }
    }
}

template <bool GATED, int ACT, int WARPS, int BLOCKS>
int launch_warps(const FewArgs& args, const dim3& grid, cudaStream_t stream) {
    const dim3 block(32 * WARPS);
    if (args.M <= 8)
        return launch_dependent(rtlynx_gated_few_kernel<GATED, 1, ACT, WARPS, WARPS == 8 ? 3 : 1>, grid, block, 0, stream, args);
    return launch_dependent(rtlynx_gated_few_kernel<GATED, 2, ACT, WARPS, BLOCKS>, grid, block, 0, stream, args);
}

template <bool GATED, int ACT>
int launch_few(const FewArgs& args, cudaStream_t stream) {
    int num_sms = 0;
    int* err = nullptr;
    if (device_info(&num_sms, &err)) return static_cast<int>(cudaErrorInvalidDevice);
    const dim3 grid((args.N + kFewRows - 1) / kFewRows, (args.M + 15) / 16);
    const int blocks = static_cast<int>(grid.x * grid.y);
    // Sixteen warps where there are no more blocks than SMs, so that enough
    // loads are in flight: at 2056 -> 5512 and 11 tokens, where that is the
    // down-projection, the call takes 20.8 us, 23.7 with eight.  With more blocks eight are as good or better (70 against
    // 77 us at 5120 -> 13824, one token).
    if (blocks <= num_sms) return launch_warps<GATED, ACT, 16, 1>(args, grid, stream);
    // Past eight tokens two blocks of 128 registers a thread on an SM, three of
    // 80 where they are all resident then (11 tokens at 1536 -> 4096: 12.0 us,
    // 13.6 with three; at 2056 -> 5512 22.1 and 21.2, although 80 registers spill 52
    // bytes of the gated kernel).  Up to eight tokens three (one at 5120 -> 13824:
    // 66.6 us, 75.4 with two).
    if (blocks > 2 * num_sms && blocks <= 3 * num_sms) return launch_warps<GATED, ACT, 8, 3>(args, grid, stream);
    return launch_warps<GATED, ACT, 8, 2>(args, grid, stream);
}

}  // namespace

int launch_gated_few(const void* X, const void* W_gate, const void* W_up, void* H, void* G, void* U, void* low, int M,
                     int D, int D_ff, int act, cudaStream_t stream) {
    FewArgs args{};
    args.x = static_cast<const uint16_t*>(X);
    args.w[0] = static_cast<const uint16_t*>(W_gate);
    args.w[1] = static_cast<const uint16_t*>(W_up);
    args.out[0] = static_cast<uint16_t*>(H);
    args.out[1] = static_cast<uint16_t*>(G);
    args.out[2] = static_cast<uint16_t*>(U);
    args.out[3] = static_cast<uint16_t*>(low);
    args.M = M, args.N = D_ff, args.K = D;
    return act == RTLYNX_ACT_SILU ? launch_few<true, RTLYNX_ACT_SILU>(args, stream)
                                  : launch_few<true, RTLYNX_ACT_GELU>(args, stream);
}

int launch_down_few(const void* H, const void* W_down, void* Y, int M, int D_ff, int D, cudaStream_t stream) {
    FewArgs args{};
    args.x = static_cast<const uint16_t*>(H);
    args.w[0] = args.w[1] = static_cast<const uint16_t*>(W_down);
    args.out[0] = static_cast<uint16_t*>(Y);
    args.M = M, args.N = D, args.K = D_ff;
    return launch_few<false, 0>(args, stream);
}

}  // namespace rtlynx
