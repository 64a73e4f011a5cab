// Query and key heads between the qkv layer and attention: rotary positions
// with several axes, RMS norm of each head fused with the rotation, and the
// gradients of both.
//
//   n = x r,  r = (mean_c x_c^2 + eps)^(-1/2)     (norm forms only)
//   y = R(p) (n w)                                 pair i of axis a turned by
//                                                  p_a f_i radians
//   backward, g = R(p)^T dy:
//   dw = sum over tokens and heads of g n
//   dx = r (g w - n mean_c(g w n))
//
// Every element is read once and written once and needs a handful of
// operations, so memory bounds it.  A group of lanes owns one token of one
// tensor and walks over that token's heads, eight channels a lane: a lane keeps
// the same channels of every head, so the cosines, sines and norm weights of
// its channels are computed or loaded once a token and stay in registers, and
// no table of angles is read.  Eight channels are 16 bytes of a 16-bit type; a
// head of d channels takes d / 8 lanes, and a warp as many tokens as fit (four
// at 64 channels, two at 128).  (A warp's lanes on several heads of one token
// instead repeat its angles: 55 us against 23 on 31077 tokens of 12 + 6 heads of
// 48, and nothing gained with many heads.)  Pairs are computed two at a time
// (f32x2): the norm's gradient took 195 us without, 179 with.
//
// Measured (32760 tokens, 40 + 40 heads of 128, bf16, 1.34 GB): rotation 207 us
// (6.5 TB/s, the measured copy rate), with the norm 218 us (6.1 TB/s); gradient
// of both on 16384 tokens (1.01 GB) 160 us (6.3 TB/s).  That is after pauses: in a
// long run, which reaches the power cap (980 W, 1.7 GHz of 1.97), 209, 231 and
// 181 us (the last 5.6 TB/s).
//
// Angles: position x frequency / 2 pi in 64 bits, reduced to an eighth of a
// turn there, so a position of 2^24 loses nothing; sine and cosine of the
// remainder in 32.  Sums of squares and all other sums are held in 32 bits,
// outputs rounded once.
//
// The weights' gradients: each block sums its tokens in a fixed order into a
// row of the caller's workspace, and a second kernel adds the rows in order;
// no atomics, so equal calls give equal bits.
#include <cuda_fp16.h>
#include <math.h>

#include "../../include/rtlynx.h"
#include "internal.h"
#include "ptx.cuh"

namespace rtlynx {
namespace {

constexpr int kHeadThreads = 256;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kMaxDim = 256;
constexpr int kMaxPairs = kMaxDim / 2;
constexpr int kHeadGradRows = 512;  // rows of partial sums the workspace holds for each tensor
constexpr double kTwoPi = 6.283185307179586476925286766559;

enum Kind { kRope = 0, kNorm = 1, kNormBackward = 2 };

// One tensor of the call: x is read (the gradient dy too in backward), y written.
struct HeadTensor {
    const void* x;
    const void* dy;
    void* y;
    const void* w;
    float* part;  // backward: [blocks, dim] partial sums of the weight's gradient
    int64_t xb, xs, xh, gb, gs, gh, yb, ys, yh;  // strides of batch, token, head, in elements
    uint32_t heads, groups, run;  // a token's heads are cut into `groups` runs of `run`
    uint32_t rows;                // tokens of all sequences
    uint32_t items, blocks;       // items: (as many tokens as fit a warp) x groups
};

struct HeadArgs {
    HeadTensor t[2];  // queries, keys
    const void* positions;
    int64_t pb, ps, pa;  // strides of the positions: batch, token, axis
    int pos_type;
    uint32_t tokens;  // per sequence
    int dim, pairs;
    float eps, sin_sign;
    uint8_t axis[kMaxPairs];
    double turns[kMaxPairs];  // frequency / 2 pi
};

template <typename T>
struct Raw {
    uint32_t r[2 * sizeof(T)];
};

// Two floats in one 64-bit register: sm_100 multiplies and adds both at once.
using F2 = unsigned long long;

__device__ __forceinline__ F2 make_f2(float lo, float hi) {
    F2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float lo(F2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi(F2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ F2 negate(F2 v) { return v ^ 0x8000000080000000ull; }

__device__ __forceinline__ float widen_lo(uint32_t u, __nv_bfloat16) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float widen_hi(uint32_t u, __nv_bfloat16) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ float widen_lo(uint32_t u, __half) { return __low2float(*reinterpret_cast<__half2*>(&u)); }
__device__ __forceinline__ float widen_hi(uint32_t u, __half) { return __high2float(*reinterpret_cast<__half2*>(&u)); }

__device__ __forceinline__ uint32_t narrow(float a, float b, __nv_bfloat16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t narrow(float a, float b, __half) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

// A lane's four pairs: x[i] holds the first channels of pairs 2 i and 2 i + 1,
// y[i] the second ones.
struct Pairs {
    F2 x[2], y[2];
};

template <typename T, bool HALF>
__device__ __forceinline__ Pairs unpack(const Raw<T>& raw) {
    Pairs p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (sizeof(T) == 4) {
            const uint32_t* r = raw.r;
            const int x0 = HALF ? 2 * i : 4 * i, x1 = HALF ? 2 * i + 1 : 4 * i + 2, y = HALF ? 4 : 1;
            p.x[i] = make_f2(__uint_as_float(r[x0]), __uint_as_float(r[x1]));
            p.y[i] = make_f2(__uint_as_float(r[x0 + y]), __uint_as_float(r[x1 + y]));
        } else if constexpr (HALF) {
            p.x[i] = make_f2(widen_lo(raw.r[i], T()), widen_hi(raw.r[i], T()));
            p.y[i] = make_f2(widen_lo(raw.r[2 + i], T()), widen_hi(raw.r[2 + i], T()));
        } else {
            p.x[i] = make_f2(widen_lo(raw.r[2 * i], T()), widen_lo(raw.r[2 * i + 1], T()));
            p.y[i] = make_f2(widen_hi(raw.r[2 * i], T()), widen_hi(raw.r[2 * i + 1], T()));
        }
    }
    return p;
}

template <typename T, bool HALF>
__device__ __forceinline__ Raw<T> pack(const Pairs& p) {
    Raw<T> raw;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (sizeof(T) == 4) {
            const int x0 = HALF ? 2 * i : 4 * i, x1 = HALF ? 2 * i + 1 : 4 * i + 2, y = HALF ? 4 : 1;
            raw.r[x0] = __float_as_uint(lo(p.x[i]));
            raw.r[x1] = __float_as_uint(hi(p.x[i]));
            raw.r[x0 + y] = __float_as_uint(lo(p.y[i]));
            raw.r[x1 + y] = __float_as_uint(hi(p.y[i]));
        } else if constexpr (HALF) {
            raw.r[i] = narrow(lo(p.x[i]), hi(p.x[i]), T());
            raw.r[2 + i] = narrow(lo(p.y[i]), hi(p.y[i]), T());
        } else {
            raw.r[2 * i] = narrow(lo(p.x[i]), lo(p.y[i]), T());
            raw.r[2 * i + 1] = narrow(hi(p.x[i]), hi(p.y[i]), T());
        }
    }
    return raw;
}

// A lane's eight channels are two runs of four, at offsets a and b.  They
// are one run of eight (b = a + 4) unless HALF pairs channel i with channel
// i + rotated / 2.  Outputs may be the inputs' own memory, so these are plain
// loads, not the read-only path.
template <typename T, bool HALF>
__device__ __forceinline__ void load8(const T* p, int a, int b, Raw<T>& raw) {
    if constexpr (sizeof(T) == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + a), v = *reinterpret_cast<const uint4*>(p + b);
        raw.r[0] = u.x, raw.r[1] = u.y, raw.r[2] = u.z, raw.r[3] = u.w;
        raw.r[4] = v.x, raw.r[5] = v.y, raw.r[6] = v.z, raw.r[7] = v.w;
    } else if constexpr (HALF) {
        const uint2 u = *reinterpret_cast<const uint2*>(p + a), v = *reinterpret_cast<const uint2*>(p + b);
        raw.r[0] = u.x, raw.r[1] = u.y, raw.r[2] = v.x, raw.r[3] = v.y;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p + a);
        raw.r[0] = u.x, raw.r[1] = u.y, raw.r[2] = u.z, raw.r[3] = u.w;
    }
}

template <typename T, bool HALF>
__device__ __forceinline__ void store8(T* p, int a, int b, const Raw<T>& raw) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4*>(p + a) = make_uint4(raw.r[0], raw.r[1], raw.r[2], raw.r[3]);
        *reinterpret_cast<uint4*>(p + b) = make_uint4(raw.r[4], raw.r[5], raw.r[6], raw.r[7]);
    } else if constexpr (HALF) {
        *reinterpret_cast<uint2*>(p + a) = make_uint2(raw.r[0], raw.r[1]);
        *reinterpret_cast<uint2*>(p + b) = make_uint2(raw.r[2], raw.r[3]);
    } else {
        *reinterpret_cast<uint4*>(p + a) = make_uint4(raw.r[0], raw.r[1], raw.r[2], raw.r[3]);
    }
}

// Turns the lane's four pairs: (x, y) -> (x a - y b, x c + y d).  Where not the
// whole head is turned, the other pairs are (x a, y d): their b and c are zero,
// but zero times an infinity in the other channel would be NaN.
__device__ __forceinline__ void turn(Pairs& p, const F2 (&a)[2], const F2 (&nb)[2], const F2 (&c)[2], const F2 (&d)[2],
                                     bool whole, uint32_t turned) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const F2 x = mul(p.x[i], a[i]), y = mul(p.y[i], d[i]);
        F2 tx = fma2(p.y[i], nb[i], x), ty = fma2(p.x[i], c[i], y);
        if (!whole) {
            const bool t0 = turned >> (2 * i) & 1u, t1 = turned >> (2 * i + 1) & 1u;
            tx = make_f2(t0 ? lo(tx) : lo(x), t1 ? hi(tx) : hi(x));
            ty = make_f2(t0 ? lo(ty) : lo(y), t1 ? hi(ty) : hi(y));
        }
        p.x[i] = tx;
        p.y[i] = ty;
    }
}

// Sum over a head's lanes, in every one of them.  LANES = 0: heads of up to ten
// lanes, side by side without a gap; head_lane is the first of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float v, int chunk, int lanes, int head_lane) {
    if constexpr (LANES > 0) {
#pragma unroll
        for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        return v;
    } else {
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) {
            const float other = __shfl_down_sync(0xFFFFFFFFu, v, m);
            if (chunk + m < lanes) v += other;
        }
        return __shfl_sync(0xFFFFFFFFu, v, head_lane);
    }
}

template <typename T, int LANES, bool HALF, int KIND>
__global__ void __launch_bounds__(kHeadThreads, KIND == kNormBackward ? 2 : 4) rtlynx_heads_kernel(const __grid_constant__ HeadArgs args) {
    // Heads loaded before the first is used, and whether the next ones are
    // loaded before these are computed.  Registers decide: forward, 64 of them
    // leave 32 warps an SM, which hide the latency without looking ahead
    // (video workload's norm: 229 us when measured; two heads and looking
    // ahead 235, 80 registers 249), though the norm's instances spill 16 to 92
    // bytes a thread for it (24 at 128 channels in 16 bits, 48 with half pairing); backward, with two tensors read and the weights' sums
    // kept, 128 and 16 warps, looking ahead (179 us when
    // measured; without 205, two heads 190).
    // Half pairing of a 16-bit type takes two loads for a lane's channels: two
    // heads at a time backward (25286 tokens of 20 + 20 heads of 128: 154 us; four
    // spill registers, 241 us).
    constexpr bool kTwoLoads = HALF && sizeof(T) == 2;
    constexpr int kUnroll = sizeof(T) == 4 || (kTwoLoads && KIND == kNormBackward) ? 2 : 4;
    constexpr int kGrads = KIND == kNormBackward ? kUnroll : 1;
    constexpr bool kPipe = KIND == kNormBackward;
    __shared__ double turns[kMaxPairs];
    __shared__ uint8_t axis[kMaxPairs];
    __shared__ float sums[KIND == kNormBackward ? kHeadWarps * 32 * 8 : 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < args.pairs; i += kHeadThreads) {
        turns[i] = args.turns[i];
        axis[i] = args.axis[i];
    }
    __syncthreads();
    grid_dependency_wait();
    launch_dependents();

    const bool keys = blockIdx.x >= args.t[0].blocks;
    const HeadTensor& t = args.t[keys ? 1 : 0];
    const uint32_t block = blockIdx.x - (keys ? args.t[0].blocks : 0u);

    // a head takes `lanes` lanes (some of them idle where they are LANES), and
    // the warp as many tokens as fit
    const int lanes = LANES > 0 ? LANES : args.dim / 8;
    const int per_pass = 32 / lanes;
    const int chunk = lane % lanes, sub = lane / lanes;
    const bool active = LANES > 0 ? 8 * chunk < args.dim : sub < per_pass;
    auto sum_head = [&](float v) { return head_sum<LANES>(v, chunk, lanes, lane - chunk); };
    const int rotated = 2 * args.pairs;
    const bool whole = rotated == args.dim;
    // channel offsets of the lane's two runs of four
    int a = 8 * chunk, b = 8 * chunk + 4;
    if (HALF && 8 * chunk < rotated) {
        a = 4 * chunk;
        b = args.pairs + 4 * chunk;
    }

    const F2 one = make_f2(1.0f, 1.0f), zero = make_f2(0.0f, 0.0f);
    Pairs w{{one, one}, {one, one}};
    auto load_weights = [&]() {
        if (active && t.w) {
            Raw<T> raw;
            load8<T, HALF>(static_cast<const T*>(t.w), a, b, raw);
            w = unpack<T, HALF>(raw);
        }
    };
    if constexpr (KIND == kNormBackward) load_weights();
    Pairs dw{{zero, zero}, {zero, zero}};
    const float inv_dim = 1.0f / static_cast<float>(args.dim);

    for (uint32_t item = block * kHeadWarps + warp; item < t.items; item += t.blocks * kHeadWarps) {
        const uint32_t slot = item / t.groups, group = item - slot * t.groups;
        const uint32_t token = slot * per_pass + sub;
        const bool live = active && token < t.rows;
        const uint32_t bi = token / args.tokens, si = token - bi * args.tokens;
        const T* x = static_cast<const T*>(t.x) + bi * t.xb + si * t.xs;
        const T* dy = KIND == kNormBackward ? static_cast<const T*>(t.dy) + bi * t.gb + si * t.gs : nullptr;
        T* y = static_cast<T*>(t.y) + bi * t.yb + si * t.ys;
        const uint32_t first = group * t.run;
        const uint32_t last = min(first + t.run, t.heads);
        auto fetch = [&](uint32_t h0, Raw<T>(&rx)[kUnroll], Raw<T>(&rg)[kGrads]) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const uint32_t h = h0 + u;
#pragma unroll
                for (int j = 0; j < static_cast<int>(2 * sizeof(T)); ++j) {
                    rx[u].r[j] = 0u;
                    if (KIND == kNormBackward) rg[u % kGrads].r[j] = 0u;
                }
                if (live && h < last) {
                    load8<T, HALF>(x + h * t.xh, a, b, rx[u]);
                    if constexpr (KIND == kNormBackward) load8<T, HALF>(dy + h * t.gh, a, b, rg[u]);
                }
            }
        };
        Raw<T> rx[kUnroll], rg[kGrads];
        fetch(first, rx, rg);  // on their way while the angles are computed

        float c[4], s[4];
        uint32_t turned = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = 1.0f;
            s[j] = 0.0f;
            const int i = 4 * chunk + j;
            if (live && i < args.pairs) {
                const int64_t at = bi * args.pb + si * args.ps + axis[i] * args.pa;
                double p;
                if (args.pos_type == RTLYNX_POS_INT32)
                    p = static_cast<double>(static_cast<const int32_t*>(args.positions)[at]);
                else if (args.pos_type == RTLYNX_POS_INT64)
                    p = static_cast<double>(static_cast<const int64_t*>(args.positions)[at]);
                else
                    p = static_cast<double>(static_cast<const float*>(args.positions)[at]);
                double turn = p * turns[i];
                turn -= rint(turn);
                const double quarter = rint(4.0 * turn);
                const float rest = static_cast<float>(turn - 0.25 * quarter);
                float sn, cs;
                sincospif(2.0f * rest, &sn, &cs);
                const int q = static_cast<int>(quarter) & 3;
                c[j] = q == 0 ? cs : (q == 1 ? -sn : (q == 2 ? -cs : sn));
                s[j] = args.sin_sign * (q == 0 ? sn : (q == 1 ? cs : (q == 2 ? -sn : -cs)));
                turned |= 1u << j;
            }
        }
        // the turn's coefficients; the norm's weights are part of them going
        // forward (and not kept beside them)
        if constexpr (KIND == kNorm) load_weights();
        F2 ca[2], nb[2], cc[2], cd[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const F2 c2 = make_f2(c[2 * i], c[2 * i + 1]), s2 = make_f2(s[2 * i], s[2 * i + 1]);
            ca[i] = cd[i] = c2;
            cc[i] = s2;
            nb[i] = negate(s2);
            if constexpr (KIND == kNorm) {
                ca[i] = mul(ca[i], w.x[i]);
                cc[i] = mul(cc[i], w.x[i]);
                nb[i] = mul(nb[i], w.y[i]);
                cd[i] = mul(cd[i], w.y[i]);
            }
        }

        auto head = [&](uint32_t h, const Raw<T>& xr, const Raw<T>& gr) {
            Pairs v = unpack<T, HALF>(xr);
            if constexpr (KIND == kRope) {
                turn(v, ca, nb, cc, cd, whole, turned);
            } else {
                const F2 squares = fma2(v.y[1], v.y[1], fma2(v.x[1], v.x[1], fma2(v.y[0], v.y[0], mul(v.x[0], v.x[0]))));
                const float r = rsqrtf(fmaf(sum_head(lo(squares) + hi(squares)), inv_dim, args.eps));
                const F2 r2 = make_f2(r, r);
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // n
                    v.x[i] = mul(v.x[i], r2);
                    v.y[i] = mul(v.y[i], r2);
                }
                if constexpr (KIND == kNorm) {
                    turn(v, ca, nb, cc, cd, whole, turned);
                } else {
                    Pairs g = unpack<T, HALF>(gr);
                    turn(g, ca, nb, cc, cd, whole, turned);
                    F2 dot = zero;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        dw.x[i] = fma2(g.x[i], v.x[i], dw.x[i]);
                        dw.y[i] = fma2(g.y[i], v.y[i], dw.y[i]);
                        g.x[i] = mul(g.x[i], w.x[i]);
                        g.y[i] = mul(g.y[i], w.y[i]);
                        dot = fma2(g.x[i], v.x[i], dot);
                        dot = fma2(g.y[i], v.y[i], dot);
                    }
                    const float mean = -sum_head(lo(dot) + hi(dot)) * inv_dim;
                    const F2 mean2 = make_f2(mean, mean);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v.x[i] = mul(r2, fma2(v.x[i], mean2, g.x[i]));
                        v.y[i] = mul(r2, fma2(v.y[i], mean2, g.y[i]));
                    }
                }
            }
            if (live) store8<T, HALF>(y + h * t.yh, a, b, pack<T, HALF>(v));
        };
        for (uint32_t h0 = first; h0 < last; h0 += kUnroll) {
            Raw<T> nx[kUnroll], ng[kGrads];
            if (kPipe) fetch(h0 + kUnroll, nx, ng);
            // The same in the whole warp.  (Heads past the last computed as zeros:
            // 39201 tokens of 5 + 1 heads of 192 took 197 us backward, now 149.)
            if (h0 + kUnroll <= last) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) head(h0 + u, rx[u], rg[u % kGrads]);
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll - 1; ++u)
                    if (h0 + u < last) head(h0 + u, rx[u], rg[u % kGrads]);
            }
            if (kPipe) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) rx[u] = nx[u];
#pragma unroll
                for (int u = 0; u < kGrads; ++u) rg[u] = ng[u];
            } else {
                fetch(h0 + kUnroll, rx, rg);
            }
        }
    }

    if constexpr (KIND == kNormBackward) {
        // Heads that shared a pass hold the same channels in different lanes.
        // In channel order: the lane's runs of four at a and at b.
        float sum[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int x0 = HALF ? 2 * i : 4 * i, x1 = HALF ? 2 * i + 1 : 4 * i + 2, to_y = HALF ? 4 : 1;
            sum[x0] = lo(dw.x[i]);
            sum[x1] = hi(dw.x[i]);
            sum[x0 + to_y] = lo(dw.y[i]);
            sum[x1 + to_y] = hi(dw.y[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float own = sum[j];
            for (int k = 1; k < per_pass; ++k) sum[j] += __shfl_sync(0xFFFFFFFFu, own, (chunk + k * lanes) & 31);
            if (sub == 0) sums[(warp * 32 + chunk) * 8 + j] = sum[j];
        }
        __syncthreads();
        if (t.part && warp == 0 && sub == 0 && active) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float total = 0.0f;
                for (int k = 0; k < kHeadWarps; ++k) total += sums[(k * 32 + chunk) * 8 + j];
                t.part[static_cast<size_t>(block) * args.dim + (j < 4 ? a + j : b + j - 4)] = total;
            }
        }
    }
}

// Adds the rows of partial sums: block (channel / 32, tensor); a warp takes
// every 32nd row, in order, then the warps' sums are added in order.  (A row for
// each of 148 SMs: five loads one after the other in each warp, not nineteen.)
constexpr int kGradWarps = 32;
struct WeightGradArgs {
    const float* part[2];
    float* dw[2];
    uint32_t rows[2];
    int dim;
};

__global__ void __launch_bounds__(32 * kGradWarps) rtlynx_heads_weight_grad_kernel(const WeightGradArgs args) {
    __shared__ float sums[kGradWarps][32];
    grid_dependency_wait();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.y, c = blockIdx.x * 32 + lane;
    if (!args.dw[t]) return;
    float total = 0.0f;
    if (c < args.dim)
        for (uint32_t r = warp; r < args.rows[t]; r += kGradWarps)
            total += args.part[t][static_cast<size_t>(r) * args.dim + c];
    sums[warp][lane] = total;
    __syncthreads();
    if (warp == 0 && c < args.dim) {
        float all = 0.0f;
        for (int k = 0; k < kGradWarps; ++k) all += sums[k][lane];
        args.dw[t][c] = all;
    }
}

// ---------------------------------------------------------------- host side
using Wide = __int128;

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A view with the sizes it is used at.
struct View {
    const rtlynx_heads* v;
    int64_t B, S, D;
    int bytes;
    Wide within() const { return Wide(S - 1) * v->stride_s + Wide(v->heads - 1) * v->stride_h + D; }  // one sequence
    Wide token() const { return Wide(v->heads - 1) * v->stride_h + D; }
    Wide extent() const { return Wide(B - 1) * v->stride_b + within(); }
    Wide begin() const { return Wide(reinterpret_cast<uintptr_t>(v->ptr)); }
    Wide end() const { return begin() + extent() * bytes; }
};

bool same_view(const View& a, const View& b) {
    return a.v->ptr == b.v->ptr && a.v->heads == b.v->heads && (a.B == 1 || a.v->stride_b == b.v->stride_b) &&
           (a.S == 1 || a.v->stride_s == b.v->stride_s) && (a.v->heads == 1 || a.v->stride_h == b.v->stride_h);
}

// Whether two views may share an element: their ranges meet, and they are not
// seen to be different parts of the same rows (tokens or sequences).
bool may_meet(const View& a, const View& b) {
    if (a.end() <= b.begin() || b.end() <= a.begin()) return false;
    const Wide bytes = b.begin() - a.begin();
    if (bytes % a.bytes) return true;
    const Wide delta = bytes / a.bytes;
    auto apart = [&](Wide period, Wide ea, Wide eb) {
        if (period <= 0) return false;
        const Wide r = ((delta % period) + period) % period;
        return r >= ea && r + eb <= period;
    };
    if (a.B > 1 && a.v->stride_b == b.v->stride_b && apart(a.v->stride_b, a.within(), b.within())) return false;
    const int64_t s = a.v->stride_s;
    if (a.S > 1 && s > 0 && s == b.v->stride_s &&
        (a.B == 1 || (a.v->stride_b % s == 0 && b.v->stride_b % s == 0)) && apart(s, a.token(), b.token()))
        return false;
    return true;
}

// Whether an output view writes an element twice.
bool self_overlap(const View& a) {
    struct Dim {
        int64_t n, stride;
    } d[3] = {{a.B, a.v->stride_b}, {a.S, a.v->stride_s}, {a.v->heads, a.v->stride_h}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (d[j].stride < d[i].stride) {
                const Dim t = d[i];
                d[i] = d[j];
                d[j] = t;
            }
    Wide span = a.D;
    for (const Dim& k : d) {
        if (k.n == 1) continue;
        if (k.stride < span) return true;
        span += Wide(k.n - 1) * k.stride;
    }
    return false;
}

int check_view(const View& a) {
    if (!a.v->ptr || !aligned(a.v->ptr) || a.v->heads <= 0) return RTLYNX_ERR_INVALID_ARG;
    const rtlynx_heads& v = *a.v;
    auto bad = [](int64_t n, int64_t stride) { return n > 1 && (stride < 0 || stride % 8); };
    if (bad(a.B, v.stride_b) || bad(a.S, v.stride_s) || bad(v.heads, v.stride_h)) return RTLYNX_ERR_INVALID_ARG;
    if (v.heads > 65536 || a.extent() > (Wide(1) << 45)) return RTLYNX_ERR_UNSUPPORTED;
    return RTLYNX_OK;
}

bool meets(const View& a, const void* p, Wide bytes) {
    const Wide b = Wide(reinterpret_cast<uintptr_t>(p));
    return p && bytes > 0 && a.begin() < b + bytes && b < a.end();
}

bool ranges_meet(const void* p, Wide np, const void* q, Wide nq) {
    if (!p || !q) return false;
    const Wide a = Wide(reinterpret_cast<uintptr_t>(p)), b = Wide(reinterpret_cast<uintptr_t>(q));
    return a < b + nq && b < a + np;
}

int elem_bytes(int dtype) { return dtype == RTLYNX_FP32 ? 4 : 2; }

// Lanes that a head takes: as many as it has eights of channels where that lets
// more heads into a warp pass than the next power of two, whose sums need
// fewer steps.
int lanes_of(int64_t dim) {
    const int exact = static_cast<int>(dim / 8);
    int power = 8;
    while (power < exact) power *= 2;
    return 32 / exact > 32 / power ? exact : power;
}
int heads_per_pass(int64_t dim) { return 32 / lanes_of(dim); }

int64_t slots_of(int64_t rows, int64_t dim) { return (rows + heads_per_pass(dim) - 1) / heads_per_pass(dim); }

// Heads that a group of lanes takes of its token: all of them, so that angles
// are computed once, unless that leaves the tensor with more heads fewer than
// `want` warps; then shorter runs, as long for the other tensor.
int64_t run_length(int64_t rows, int64_t most_heads, int64_t dim, int64_t want) {
    const int64_t slots = slots_of(rows, dim);
    int64_t groups = slots >= want ? 1 : (want + slots - 1) / slots;
    if (groups > most_heads) groups = most_heads;
    return (most_heads + groups - 1) / groups;
}

void deal(HeadTensor& t, int64_t rows, int64_t heads, int64_t run, int64_t dim, int64_t most_blocks) {
    t.run = static_cast<uint32_t>(run < heads ? run : heads);
    t.groups = static_cast<uint32_t>((heads + t.run - 1) / t.run);
    t.heads = static_cast<uint32_t>(heads);
    t.rows = static_cast<uint32_t>(rows);
    const int64_t items = slots_of(rows, dim) * t.groups;
    t.items = static_cast<uint32_t>(items);
    const int64_t blocks = (items + kHeadWarps - 1) / kHeadWarps;
    t.blocks = static_cast<uint32_t>(blocks < most_blocks ? blocks : most_blocks);
}

// Both tensors' work.  Forward, as many blocks as there are items for, 16 warps
// an SM asked for.  Backward, where a block keeps a row of partial sums, the two
// blocks an SM that run at once, shared out by the tensors' heads (three more
// for a token's angles).
void deal_all(HeadTensor (&t)[2], const int64_t (&heads)[2], int tensors, int64_t rows, int64_t dim, int num_sms,
              bool backward) {
    const int big = tensors == 2 && heads[1] > heads[0] ? 1 : 0;
    int64_t blocks[2] = {int64_t(1) << 30, int64_t(1) << 30}, want = 16ll * num_sms;
    if (backward) {
        const int64_t all = 2 * num_sms < kHeadGradRows ? 2 * num_sms : kHeadGradRows;
        blocks[big] = all;
        if (tensors == 2) {
            const int64_t mine = heads[big] + 3, other = heads[1 - big] + 3;
            blocks[1 - big] = all * other / (mine + other);
            if (blocks[1 - big] < 1) blocks[1 - big] = 1;
            blocks[big] = all - blocks[1 - big];
        }
        want = blocks[big] * kHeadWarps;
    }
    const int64_t run = run_length(rows, heads[big], dim, want);
    for (int i = 0; i < tensors; ++i) deal(t[i], rows, heads[i], run, dim, blocks[i]);
}

template <typename T, int LANES>
int launch_lanes(const HeadArgs& args, bool half, int kind, cudaStream_t stream) {
    const dim3 grid(args.t[0].blocks + args.t[1].blocks), block(kHeadThreads);
    if (half) {
        if (kind == kRope) return launch_dependent(rtlynx_heads_kernel<T, LANES, true, kRope>, grid, block, 0, stream, args);
        if (kind == kNorm) return launch_dependent(rtlynx_heads_kernel<T, LANES, true, kNorm>, grid, block, 0, stream, args);
        return launch_dependent(rtlynx_heads_kernel<T, LANES, true, kNormBackward>, grid, block, 0, stream, args);
    }
    if (kind == kRope) return launch_dependent(rtlynx_heads_kernel<T, LANES, false, kRope>, grid, block, 0, stream, args);
    if (kind == kNorm) return launch_dependent(rtlynx_heads_kernel<T, LANES, false, kNorm>, grid, block, 0, stream, args);
    return launch_dependent(rtlynx_heads_kernel<T, LANES, false, kNormBackward>, grid, block, 0, stream, args);
}

template <typename T>
int launch_type(const HeadArgs& args, bool half, int kind, cudaStream_t stream) {
    switch (lanes_of(args.dim)) {
        case 8: return launch_lanes<T, 8>(args, half, kind, stream);
        case 16: return launch_lanes<T, 16>(args, half, kind, stream);
        case 32: return launch_lanes<T, 32>(args, half, kind, stream);
        default: return launch_lanes<T, 0>(args, half, kind, stream);
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

struct Call {
    const rtlynx_heads *x[2], *dy[2], *y[2];  // queries, keys; keys NULL when the call has none
    const void* w[2];
    float* dw[2];
};

// Checks and runs one call of any kind.
int run_heads(int kind, float sin_sign, const Call& call, int64_t B, int64_t S, int64_t D, int dtype,
              const rtlynx_rope_spec* spec, const void* positions, int64_t pos_stride_b, int64_t pos_stride_s,
              int64_t pos_stride_a, float eps, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    if (dtype != RTLYNX_BF16 && dtype != RTLYNX_FP16 && dtype != RTLYNX_FP32) return RTLYNX_ERR_INVALID_ARG;
    if (B <= 0 || S <= 0 || D <= 0 || D % 8) return RTLYNX_ERR_INVALID_ARG;
    if (D > kMaxDim || B > INT32_MAX || S > INT32_MAX || B * S > INT32_MAX) return RTLYNX_ERR_UNSUPPORTED;
    if (!spec || !positions || !call.x[0] || !call.y[0]) return RTLYNX_ERR_INVALID_ARG;
    if ((call.x[1] == nullptr) != (call.y[1] == nullptr)) return RTLYNX_ERR_INVALID_ARG;
    if (kind == kNormBackward && (!call.dy[0] || (call.x[1] == nullptr) != (call.dy[1] == nullptr)))
        return RTLYNX_ERR_INVALID_ARG;
    if (kind != kRope && !(eps > 0.0f && eps < INFINITY)) return RTLYNX_ERR_INVALID_ARG;
    // the rotation
    if (spec->n_axes < 1) return RTLYNX_ERR_INVALID_ARG;
    if (spec->n_axes > RTLYNX_MAX_AXES) return RTLYNX_ERR_UNSUPPORTED;
    if (spec->pairing != RTLYNX_ROPE_INTERLEAVED && spec->pairing != RTLYNX_ROPE_HALF) return RTLYNX_ERR_INVALID_ARG;
    if (spec->pos_type != RTLYNX_POS_INT32 && spec->pos_type != RTLYNX_POS_INT64 && spec->pos_type != RTLYNX_POS_FP32)
        return RTLYNX_ERR_INVALID_ARG;
    int64_t rotated = 0;
    for (int a = 0; a < spec->n_axes; ++a) {
        if (spec->axis_dim[a] < 2 || spec->axis_dim[a] % 2 || spec->axis_dim[a] > D) return RTLYNX_ERR_INVALID_ARG;
        rotated += spec->axis_dim[a];
    }
    if (rotated > D) return RTLYNX_ERR_INVALID_ARG;
    if (spec->pairing == RTLYNX_ROPE_HALF && rotated % 8) return RTLYNX_ERR_UNSUPPORTED;
    if (!spec->inv_freq && !(spec->theta > 0.0 && spec->theta < INFINITY)) return RTLYNX_ERR_INVALID_ARG;
    const uintptr_t pos_align = spec->pos_type == RTLYNX_POS_INT64 ? 8 : 4;
    if (reinterpret_cast<uintptr_t>(positions) % pos_align) return RTLYNX_ERR_INVALID_ARG;
    if ((B > 1 && pos_stride_b < 0) || (S > 1 && pos_stride_s < 0) || (spec->n_axes > 1 && pos_stride_a < 0))
        return RTLYNX_ERR_INVALID_ARG;
    const Wide pos_extent = Wide(B - 1) * pos_stride_b + Wide(S - 1) * pos_stride_s +
                            Wide(spec->n_axes - 1) * pos_stride_a + 1;
    if (pos_extent > (Wide(1) << 45)) return RTLYNX_ERR_UNSUPPORTED;
    const Wide pos_bytes = pos_extent * Wide(pos_align);

    // the tensors
    const int bytes = elem_bytes(dtype);
    const int tensors = call.x[1] ? 2 : 1;
    auto view = [&](const rtlynx_heads* v) { return View{v, B, S, D, bytes}; };
    for (int t = 0; t < tensors; ++t) {
        const rtlynx_heads* used[3] = {call.x[t], call.y[t], kind == kNormBackward ? call.dy[t] : nullptr};
        for (const rtlynx_heads* v : used) {
            if (!v) continue;
            const int rc = check_view(view(v));
            if (rc) return rc;
            if (v->heads != call.x[t]->heads) return RTLYNX_ERR_INVALID_ARG;
        }
        if (call.w[t] && !aligned(call.w[t])) return RTLYNX_ERR_INVALID_ARG;
        if (call.dw[t] && !aligned(call.dw[t])) return RTLYNX_ERR_INVALID_ARG;
        if (self_overlap(view(call.y[t]))) return RTLYNX_ERR_INVALID_ARG;
    }
    // An output may be exactly its own input (or incoming gradient); it may
    // share no element with anything else.
    for (int t = 0; t < tensors; ++t) {
        const View y = view(call.y[t]);
        for (int o = 0; o < tensors; ++o) {
            const View x = view(call.x[o]);
            if (!(o == t && same_view(y, x)) && may_meet(y, x)) return RTLYNX_ERR_INVALID_ARG;
            if (kind == kNormBackward) {
                const View g = view(call.dy[o]);
                if (!(o == t && same_view(y, g)) && may_meet(y, g)) return RTLYNX_ERR_INVALID_ARG;
            }
            if (o != t && may_meet(y, view(call.y[o]))) return RTLYNX_ERR_INVALID_ARG;
            if (meets(y, call.w[o], Wide(D) * bytes) || meets(y, call.dw[o], Wide(D) * 4)) return RTLYNX_ERR_INVALID_ARG;
        }
        if (meets(y, positions, pos_bytes)) return RTLYNX_ERR_INVALID_ARG;
    }

    HeadArgs args{};
    const bool grads = kind == kNormBackward && (call.dw[0] || call.dw[1]);
    size_t need = 0;
    if (grads) {
        need = rtlynx_qk_norm_rope_workspace_size(D);
        if (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return RTLYNX_ERR_INVALID_ARG;
        for (int t = 0; t < tensors; ++t) {
            const rtlynx_heads* used[3] = {call.x[t], call.y[t], call.dy[t]};
            for (const rtlynx_heads* v : used)
                if (meets(view(v), workspace, Wide(need))) return RTLYNX_ERR_INVALID_ARG;
            const rtlynx_heads* read[2] = {call.x[t], call.dy[t]};
            for (int o = 0; o < tensors; ++o) {
                for (const rtlynx_heads* v : read)
                    if (meets(view(v), call.dw[o], Wide(D) * 4)) return RTLYNX_ERR_INVALID_ARG;
                if (ranges_meet(call.dw[t], Wide(D) * 4, call.w[o], Wide(D) * bytes)) return RTLYNX_ERR_INVALID_ARG;
            }
            if (ranges_meet(call.w[t], Wide(D) * bytes, workspace, Wide(need)) ||
                ranges_meet(call.dw[t], Wide(D) * 4, workspace, Wide(need)) ||
                ranges_meet(call.dw[t], Wide(D) * 4, positions, pos_bytes))
                return RTLYNX_ERR_INVALID_ARG;
        }
        if (ranges_meet(call.dw[0], Wide(D) * 4, call.dw[1], Wide(D) * 4) ||
            ranges_meet(positions, pos_bytes, workspace, Wide(need)))
            return RTLYNX_ERR_INVALID_ARG;
    }
    int num_sms = 0;
    int* err = nullptr;
    const int rc = device_info(&num_sms, &err);
    if (rc) return rc;

    const int64_t rows = B * S;
    int64_t heads[2] = {};
    for (int t = 0; t < tensors; ++t) {
        HeadTensor& h = args.t[t];
        h.x = call.x[t]->ptr;
        h.xb = call.x[t]->stride_b, h.xs = call.x[t]->stride_s, h.xh = call.x[t]->stride_h;
        h.y = call.y[t]->ptr;
        h.yb = call.y[t]->stride_b, h.ys = call.y[t]->stride_s, h.yh = call.y[t]->stride_h;
        if (kind == kNormBackward) {
            h.dy = call.dy[t]->ptr;
            h.gb = call.dy[t]->stride_b, h.gs = call.dy[t]->stride_s, h.gh = call.dy[t]->stride_h;
        }
        h.w = call.w[t];
        if (rows * call.x[t]->heads > (int64_t(1) << 31)) return RTLYNX_ERR_UNSUPPORTED;  // items fit 32 bits
        heads[t] = call.x[t]->heads;
        if (call.dw[t])
            h.part = static_cast<float*>(workspace) + static_cast<size_t>(t) * kHeadGradRows * D;
    }
    deal_all(args.t, heads, tensors, rows, D, num_sms, kind == kNormBackward);
    args.positions = positions;
    args.pb = pos_stride_b, args.ps = pos_stride_s, args.pa = pos_stride_a;
    args.pos_type = spec->pos_type;
    args.tokens = static_cast<uint32_t>(S);
    args.dim = static_cast<int>(D);
    args.pairs = static_cast<int>(rotated / 2);
    args.eps = eps;
    args.sin_sign = sin_sign;
    for (int a = 0, i = 0; a < spec->n_axes; ++a)
        for (int j = 0; j < spec->axis_dim[a] / 2; ++j, ++i) {
            args.axis[i] = static_cast<uint8_t>(a);
            const double f = spec->inv_freq ? spec->inv_freq[i] : pow(spec->theta, -2.0 * j / spec->axis_dim[a]);
            args.turns[i] = f / kTwoPi;
        }
    const bool half = spec->pairing == RTLYNX_ROPE_HALF;
    int e = dtype == RTLYNX_BF16   ? launch_type<__nv_bfloat16>(args, half, kind, stream)
            : dtype == RTLYNX_FP16 ? launch_type<__half>(args, half, kind, stream)
                                   : launch_type<float>(args, half, kind, stream);
    if (e) return RTLYNX_ERR_CUDA;
    if (grads) {
        WeightGradArgs wg{};
        wg.dim = static_cast<int>(D);
        for (int t = 0; t < tensors; ++t) {
            wg.part[t] = args.t[t].part;
            wg.dw[t] = call.dw[t];
            wg.rows[t] = args.t[t].blocks;
        }
        e = launch_dependent(rtlynx_heads_weight_grad_kernel, dim3((D + 31) / 32, 2), dim3(32 * kGradWarps), 0, stream, wg);
        if (e) return RTLYNX_ERR_CUDA;
    }
    return RTLYNX_OK;
}

}  // namespace
}  // namespace rtlynx

using namespace rtlynx;

extern "C" {

int rtlynx_rope(const rtlynx_heads* q, const rtlynx_heads* k, const rtlynx_heads* q_out, const rtlynx_heads* k_out,
                int64_t B, int64_t S, int64_t D_head, int dtype, const rtlynx_rope_spec* spec, const void* positions,
                int64_t pos_stride_b, int64_t pos_stride_s, int64_t pos_stride_a, void* stream) {
    const Call call{{q, k}, {nullptr, nullptr}, {q_out, k_out}, {nullptr, nullptr}, {nullptr, nullptr}};
    return run_heads(kRope, 1.0f, call, B, S, D_head, dtype, spec, positions, pos_stride_b, pos_stride_s, pos_stride_a,
                     0.0f, nullptr, 0, static_cast<cudaStream_t>(stream));
}

int rtlynx_rope_backward(const rtlynx_heads* dq_out, const rtlynx_heads* dk_out, const rtlynx_heads* dq,
                         const rtlynx_heads* dk, int64_t B, int64_t S, int64_t D_head, int dtype,
                         const rtlynx_rope_spec* spec, const void* positions, int64_t pos_stride_b,
                         int64_t pos_stride_s, int64_t pos_stride_a, void* stream) {
    const Call call{{dq_out, dk_out}, {nullptr, nullptr}, {dq, dk}, {nullptr, nullptr}, {nullptr, nullptr}};
    return run_heads(kRope, -1.0f, call, B, S, D_head, dtype, spec, positions, pos_stride_b, pos_stride_s, pos_stride_a,
                     0.0f, nullptr, 0, static_cast<cudaStream_t>(stream));
}

int rtlynx_qk_norm_rope(const rtlynx_heads* q, const rtlynx_heads* k, const void* w_q, const void* w_k,
                        const rtlynx_heads* q_out, const rtlynx_heads* k_out, int64_t B, int64_t S, int64_t D_head,
                        int dtype, float eps, const rtlynx_rope_spec* spec, const void* positions,
                        int64_t pos_stride_b, int64_t pos_stride_s, int64_t pos_stride_a, void* stream) {
    const Call call{{q, k}, {nullptr, nullptr}, {q_out, k_out}, {w_q, k ? w_k : nullptr}, {nullptr, nullptr}};
    return run_heads(kNorm, 1.0f, call, B, S, D_head, dtype, spec, positions, pos_stride_b, pos_stride_s, pos_stride_a,
                     eps, nullptr, 0, static_cast<cudaStream_t>(stream));
}

size_t rtlynx_qk_norm_rope_workspace_size(int64_t D_head) {
    if (D_head <= 0 || D_head % 8 || D_head > kMaxDim) return 0;
    return round256(2 * static_cast<size_t>(kHeadGradRows) * static_cast<size_t>(D_head) * sizeof(float));
}

int rtlynx_qk_norm_rope_backward(const rtlynx_heads* dq_out, const rtlynx_heads* dk_out, const rtlynx_heads* q,
                                 const rtlynx_heads* k, const void* w_q, const void* w_k, const rtlynx_heads* dq,
                                 const rtlynx_heads* dk, float* dw_q, float* dw_k, int64_t B, int64_t S,
                                 int64_t D_head, int dtype, float eps, const rtlynx_rope_spec* spec,
                                 const void* positions, int64_t pos_stride_b, int64_t pos_stride_s,
                                 int64_t pos_stride_a, void* workspace, size_t ws_bytes, void* stream) {
    const Call call{{q, k}, {dq_out, dk_out}, {dq, dk}, {w_q, k ? w_k : nullptr}, {dw_q, k ? dw_k : nullptr}};
    return run_heads(kNormBackward, -1.0f, call, B, S, D_head, dtype, spec, positions, pos_stride_b, pos_stride_s,
                     pos_stride_a, eps, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
