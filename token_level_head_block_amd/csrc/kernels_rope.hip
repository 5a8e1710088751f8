// kernels_rope.hip -- RMSNorm of each query and key head with a weight, and the
// rotation by the token's positions, in one pass; and its gradients.
//
//   u = x rsqrt(mean(x^2) + eps),  n = w u,  a pair (a, b) of n at angle
//   th = position * frequency becomes (a cos th - b sin th, b cos th + a sin th).
// Backwards, dn is the pair turned by -th, dw = sum dn u, and
//   dx = rsqrt(..) (w dn - u mean(w dn u)).
// Bound by the rows' bytes.  A lane has eight neighbouring values of a row, so that a
// row is D / 8 lanes of one wave and the norm a few lane exchanges; a token's sines are
// computed once for all of its heads.  Measured in bf16: forwards 32 x 4096 tokens, 6 + 6 heads
// of 64: 87 us for 403 MB, 4.6 TB/s; 48 tokens, 12 + 4 heads of 128: 4.0 us; backwards 65536
// tokens, 12 + 12 heads of 128: 230 us for 1.2 GB, 5.2 TB/s, as a large copy.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "gated.h"

namespace mhla {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 8;      // tokens whose sines a workgroup holds at a time

struct Row8 {
    float x[8];
};
__device__ __forceinline__ Row8 load8(const uint16_t* p) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
    Row8 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.x[2 * j] = bf_lo(w[j]);
        r.x[2 * j + 1] = bf_hi(w[j]);
    }
    return r;
}
__device__ __forceinline__ Row8 load8(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return Row8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store8(uint16_t* p, const Row8& r) {
    *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16(r.x[0], r.x[1]), pack_bf16(r.x[2], r.x[3]),
                                         pack_bf16(r.x[4], r.x[5]), pack_bf16(r.x[6], r.x[7])};
}
__device__ __forceinline__ void store8(float* p, const Row8& r) {
    *reinterpret_cast<f32x4*>(p) = f32x4{r.x[0], r.x[1], r.x[2], r.x[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.x[4], r.x[5], r.x[6], r.x[7]};
}

// Sum over the L lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = 1; m < L; m <<= 1) x += shfl_xor(x, m);
    return x;
}

// Cosine and sine of position * frequency.  The product and its turns are taken in 64
// bits: at position 2^20 an fp32 angle would be off by up to 2^-4.
__device__ __forceinline__ float2 turn(int32_t pos, float freq) {
    const double t = (double)pos * (double)freq * 0.15915494309189535;   // 1 / (2 pi)
    const float f = (float)(t - rint(t));
    float2 cs;
    sincospif(2.f * f, &cs.y, &cs.x);
    return cs;
}

// The pairs of a row turned by their angles (BACK: by the opposite ones).  cs: the token's
// (cos, sin) of each pair; l: the lane's place in its row.
template <bool BACK>
__device__ __forceinline__ Row8 rotate(const Row8& n, const float2* cs, int l, int rot, int style) {
    Row8 y = n;
    if (style == 0) {
        // members rot / 2 apart: the other one lies rot / 16 lanes away
        const int half = rot / 16;
        const bool first = l < half, in = l < 2 * half;
        const int lane = threadIdx.x & 63, other = in ? (first ? lane + half : lane - half) : lane;
        const int p0 = 8 * (first ? l : l - half);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float o = __shfl(n.x[j], other, 64);
            if (in) {
                const float2 t = cs[p0 + j];
                const float s = (first != BACK) ? -t.y : t.y;
                y.x[j] = fmaf(o, s, n.x[j] * t.x);
            }
        }
    } else if (8 * l < rot) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = cs[4 * l + j];
            const float s = BACK ? -t.y : t.y;
            y.x[2 * j] = fmaf(-n.x[2 * j + 1], s, n.x[2 * j] * t.x);
            y.x[2 * j + 1] = fmaf(n.x[2 * j], s, n.x[2 * j + 1] * t.x);
        }
    }
    return y;
}

struct Args {
    QkRope r;
    FastDiv div_h, div_hk;
    int64_t first, tokens;  // this launch's first token, and the end of all tokens
    int tile;               // tokens of a workgroup's tile
};

// Sines of the tile's tokens.  Ends with a barrier.
__device__ __forceinline__ void tile_turns(const Args& a, int64_t tok0, int n, float2* cs) {
    const int pairs = a.r.rot / 2;
    for (int p = threadIdx.x; p < n * pairs; p += THREADS) {
        const int t = p / pairs, i = p - t * pairs;
        const int ax = i < a.r.sec[0] ? 0 : i < a.r.sec[0] + a.r.sec[1] ? 1 : 2;
        cs[t * pairs + i] = turn(a.r.pos[(tok0 + t) * a.r.axes + ax], a.r.freq[i]);
    }
    __syncthreads();
}

template <typename E, int D>
__global__ void __launch_bounds__(THREADS) qk_rope_fwd(Args a) {
    constexpr int L = D / 8, RP = THREADS / L;   // lanes of a row, rows of a pass
    __shared__ float2 cs[MAX_TOKENS * D / 2];
    const QkRope& r = a.r;
    const int l = threadIdx.x % L, r0 = threadIdx.x / L;
    const int64_t tok0 = a.first + (int64_t)blockIdx.x * a.tile;
    const int n = (int)min((int64_t)a.tile, a.tokens - tok0);
    tile_turns(a, tok0, n, cs);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int H = which ? r.HK : r.H;
        const FastDiv dv = which ? a.div_hk : a.div_h;
        const E* x = static_cast<const E*>(which ? r.k : r.q);
        E* y = static_cast<E*>(which ? r.ko : r.qo);
        const int64_t xs = which ? r.ks : r.qs;
        const float* wp = which ? r.wk : r.wq;
        Row8 w = {{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
        if (wp) w = load8(wp + 8 * l);
        const int rows = n * H;
        // every lane of a wave runs every pass: the rows' lanes exchange values
        for (int p0 = 0; p0 < rows; p0 += RP) {
            const int p = p0 + r0;
            const bool in = p < rows;
            const int pc = in ? p : rows - 1;
            const int t = (int)fdiv((uint32_t)pc, dv), h = pc - t * H;
            const int64_t tk = tok0 + t;
            Row8 v = load8(x + tk * xs + (int64_t)h * D + 8 * l);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v.x[j], v.x[j], ss);
            const float rs = 1.f / sqrtf(row_sum<L>(ss) * (1.f / D) + r.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) v.x[j] = v.x[j] * rs * w.x[j];
            const Row8 o = rotate<false>(v, cs + t * (r.rot / 2), l, r.rot, r.style);
            if (in) store8(y + (tk * H + h) * D + 8 * l, o);
        }
    }
}

// A workgroup takes tiles of tokens in turn and leaves the sums of its rows' dw as one
// partial [2][D]; a second launch adds the partials in 64 bits, in their order.
template <typename E, int D>
__global__ void __launch_bounds__(THREADS) qk_rope_bwd(Args a) {
    constexpr int L = D / 8, RP = THREADS / L;
    __shared__ float2 cs[MAX_TOKENS * D / 2];
    __shared__ float red[4][2][D];
    const QkRope& r = a.r;
    const int l = threadIdx.x % L, r0 = threadIdx.x / L, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    float dw[2][8];
    Row8 w[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float* wp = which ? r.wk : r.wq;
        w[which] = Row8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
        if (wp) w[which] = load8(wp + 8 * l);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[which][j] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * a.tile;
    for (int64_t tok0 = (int64_t)blockIdx.x * a.tile; tok0 < a.tokens; tok0 += step) {
        const int n = (int)min((int64_t)a.tile, a.tokens - tok0);
        __syncthreads();                 // the last tile's sines are read
        tile_turns(a, tok0, n, cs);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int H = which ? r.HK : r.H;
            const FastDiv dv = which ? a.div_hk : a.div_h;
            const E* x = static_cast<const E*>(which ? r.k : r.q);
            const E* dy = static_cast<const E*>(which ? r.dko : r.dqo);
            E* dx = static_cast<E*>(which ? r.ko : r.qo);
            const int64_t xs = which ? r.ks : r.qs;
            const int rows = n * H;
            for (int p0 = 0; p0 < rows; p0 += RP) {
                const int p = p0 + r0;
                const bool in = p < rows;
                const int pc = in ? p : rows - 1;
                const int t = (int)fdiv((uint32_t)pc, dv), h = pc - t * H;
                const int64_t tk = tok0 + t;
                Row8 v = load8(x + tk * xs + (int64_t)h * D + 8 * l);
                const Row8 g = load8(dy + (tk * H + h) * D + 8 * l);
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v.x[j], v.x[j], ss);
                const float rs = 1.f / sqrtf(row_sum<L>(ss) * (1.f / D) + r.eps);
                Row8 dn = rotate<true>(g, cs + t * (r.rot / 2), l, r.rot, r.style);
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v.x[j] *= rs;
                    if (in) dw[which][j] = fmaf(dn.x[j], v.x[j], dw[which][j]);
                    dn.x[j] *= w[which].x[j];
                    m = fmaf(dn.x[j], v.x[j], m);
                }
                m = row_sum<L>(m) * (1.f / D);
#pragma unroll
                for (int j = 0; j < 8; ++j) dn.x[j] = rs * fmaf(-v.x[j], m, dn.x[j]);
                if (in) store8(dx + (tk * H + h) * D + 8 * l, dn);
            }
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s = dw[which][j];
#pragma unroll
            for (int m = L; m < 64; m <<= 1) s += shfl_xor(s, m);
            if (lane < L) red[wave][which][8 * l + j] = s;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
        const int which = i / D, c = i % D;
        r.part[(int64_t)blockIdx.x * 2 * D + i] =
            (red[0][which][c] + red[1][which][c]) + (red[2][which][c] + red[3][which][c]);
    }
}

// dw[c] = sum of the partials: a workgroup per value, 256 runs added by a tree.
__global__ void __launch_bounds__(THREADS) qk_rope_dw(const float* part, int groups, int D, float* dwq, float* dwk) {
    __shared__ double red[4];
    const int i = blockIdx.x;
    double s = 0.0;
    for (int g = threadIdx.x; g < groups; g += THREADS) s += (double)part[(int64_t)g * 2 * D + i];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float* d = i < D ? dwq : dwk;
        if (d) d[i < D ? i : i - D] = (float)((red[0] + red[1]) + (red[2] + red[3]));
    }
}

template <typename E, int D>
hipError_t launch(Args a, bool backward) {
    if (!backward) {
        // a launch has fewer than 2^32 threads: more tokens are taken in runs
        constexpr int64_t MOST = ((int64_t)1 << 32) / THREADS - 1;
        for (; a.first < a.tokens; a.first += MOST * a.tile) {
            const int64_t n = (a.tokens - a.first + a.tile - 1) / a.tile;
            qk_rope_fwd<E, D><<<dim3((unsigned)(n < MOST ? n : MOST)), THREADS, 0, a.r.stream>>>(a);
        }
        return hipGetLastError();
    }
    qk_rope_bwd<E, D><<<dim3((unsigned)a.r.groups), THREADS, 0, a.r.stream>>>(a);
    if (a.r.dwq || a.r.dwk)
        qk_rope_dw<<<dim3(2 * D), THREADS, 0, a.r.stream>>>(a.r.part, a.r.groups, D, a.r.dwq, a.r.dwk);
    return hipGetLastError();
}

}  // namespace

int qk_rope_groups(int64_t tokens) { return tokens < 1024 ? (int)tokens : 1024; }

hipError_t run_qk_rope(const QkRope& r, bool backward) {
    Args a;
    a.r = r;
    a.first = 0;
    a.tokens = (int64_t)r.B * r.T;
    a.div_h = make_fastdiv((uint32_t)(r.H > 0 ? r.H : 1));
    a.div_hk = make_fastdiv((uint32_t)(r.HK > 0 ? r.HK : 1));
    // few tokens: one a workgroup, so that they spread over the compute units
    a.tile = a.tokens >= 2048 * MAX_TOKENS ? MAX_TOKENS : a.tokens >= 2048 ? 2 : 1;
    if (r.bf16)
        return r.D == 32 ? launch<uint16_t, 32>(a, backward) : r.D == 64 ? launch<uint16_t, 64>(a, backward)
                                                                       : launch<uint16_t, 128>(a, backward);
    return r.D == 32 ? launch<float, 32>(a, backward) : r.D == 64 ? launch<float, 64>(a, backward)
                                                                  : launch<float, 128>(a, backward);
}

}  // namespace mhla
