// kernels_gated.hip -- gated linear attention: a state S [d, d] for every
// key-value head, S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
//
// Chunk form.  With G the running sum of the gates inside a chunk of 64 tokens
// and S the state before it,
//   o_t  = scale (exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s)
//   S'   = exp(G_end) S + sum_s exp(G_end - G_s) k_s v_s^T.
// All three gradients have the same form with the roles exchanged.  A walk has
// a query role X, a key role Y and a value role Z:
//   out: X = q, Y = k, Z = v, forwards        dq: X = do, Y = v, Z = k, forwards
//   dv:  X = k, Y = q, Z = do, backwards      dk: X = v, Y = do, Z = q, backwards
// (backwards: token s sees the tokens t >= s with exp(G_t - G_s), the state
// holds the tokens behind the chunk and is taken with exp(G_end - G_s)).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "gated.h"

namespace mhla {
namespace {

constexpr int GC = GATED_CHUNK;
constexpr int THREADS = 256;   // a group of four waves
constexpr float LOG2E = 1.44269504088896341f;
constexpr float LOG2E_LOW = 1.92596299e-8f;    // log2(e) - LOG2E

// ---------------------------------------------------------------- operands
// A 16-row operand over 32 contraction values: lane (g = lane / 16, i = lane % 16)
// holds row i's values in one of two orders, the same for both operands of a product:
// "row" order, 8g + j (j < 8), or "token" order, 16 (j / 4) + 4g + j % 4, in which a
// pair of accumulator tiles (rows 4g + 0..3 of column i) is an operand as it stands.
// Where a product's rows are value columns, two tiles take them interleaved: row 4g + j of
// tiles 2k and 2k + 1 is column 32k + 8g + j and 32k + 8g + 4 + j, so that a lane ends up with
// the eight neighbouring columns that it has of an operand in row order.
// bf16: one 16x16x32 product; fp32: eight 16x16x4 products.
template <typename E>
struct Frag;
template <>
struct Frag<uint16_t> {
    u32x4 v;
};
template <>
struct Frag<float> {
    f32x4 a, b;
};

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, const f32x4& c) {
    return mfma_bf16(a.v, b.v, c);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mfma_f32(a.a[j], b.a[j], c);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mfma_f32(a.b[j], b.b[j], c);
    return c;
}

// A packed pair that the compiler takes as a word: it would otherwise round the first value
// once more by itself to widen it.
__device__ __forceinline__ uint32_t pack_opaque(float a, float b) {
    uint32_t w = pack_bf16(a, b);
    asm("" : "+v"(w));
    return w;
}

// Eight fp32 values as the sum of N operands.  bf16: each rounded to nearest, the
// remainder to the next (the subtractions are exact): one keeps 8 significant bits,
// two 17, three all 24.
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], Frag<uint16_t> (&f)[N]) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = pack_opaque(r[2 * j], r[2 * j + 1]);
            f[n].v[j] = w;
            if (n + 1 < N) {
                r[2 * j] -= bf_lo(w);
                r[2 * j + 1] -= bf_hi(w);
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], Frag<float> (&f)[N]) {
    static_assert(N == 1, "fp32 operands need no split");
    f[0].a = f32x4{x[0], x[1], x[2], x[3]};
    f[0].b = f32x4{x[4], x[5], x[6], x[7]};
}

__device__ __forceinline__ void widen(const Frag<uint16_t>& f, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf_lo(f.v[j]);
        x[2 * j + 1] = bf_hi(f.v[j]);
    }
}
__device__ __forceinline__ void widen(const Frag<float>& f, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = f.a[j];
        x[4 + j] = f.b[j];
    }
}

// ---------------------------------------------------------------- tiles in LDS
// Rows of W values, in 16-byte pieces whose place in the row is XORed with a number of
// the row, so that the lanes of a read that hold 16 rows of one piece (row order) or 4
// or 8 rows of two neighbouring pieces (token order) fall on different banks.
template <typename E, int W>
struct Tile {
    static constexpr int ROWB = W * (int)sizeof(E);
    static constexpr int NP = ROWB / 16;
    static constexpr int RP = ROWB >= 256 ? 1 : 256 / ROWB;   // rows in a pass over all banks

    __device__ static __forceinline__ int at(int row, int piece) {
        int f;
        if constexpr (sizeof(E) == 2) {
            // 16-byte reads of one piece run over rows 0-3, 12-15 of it and 4-11 of the next piece
            // together, transposing reads over 8 rows of two neighbouring pieces
            constexpr int H = NP / 2;
            const int m = (row / RP) & (NP - 1), up = m / H;
            f = (((m & (H - 1)) ^ (up * (H / 2))) << 1) | up;
        } else {
            f = (row / RP) & ((NP < 16 ? NP : 16) - 1);
        }
        return row * ROWB + ((piece ^ f) << 4);
    }
    // 16 rows from row0, contraction over columns 32 kk .. 32 kk + 31, row order
    __device__ static __forceinline__ Frag<E> rows(const char* t, int row0, int kk, int lane) {
        const int row = row0 + (lane & 15), g = lane >> 4;
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            f.v = *reinterpret_cast<const u32x4*>(t + at(row, 4 * kk + g));
        } else {
            f.a = *reinterpret_cast<const f32x4*>(t + at(row, 8 * kk + 2 * g));
            f.b = *reinterpret_cast<const f32x4*>(t + at(row, 8 * kk + 2 * g + 1));
        }
        return f;
    }
    // columns of tile n (INTER: interleaved with its neighbour's), contraction over rows
    // 32 kk .. 32 kk + 31, token order
    template <bool INTER>
    __device__ static __forceinline__ Frag<E> cols(const char* t, int kk, int n, int lane) {
        const int i = lane & 15, g = lane >> 4;
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            // transposing reads: in a group of 16 lanes, 4 lanes address 8 bytes each of one row, lane i gets
            // the i-th of these columns of the group's 4 rows
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int row = 32 * kk + 4 * g + (i >> 2);
            const int piece = INTER ? 4 * (n >> 1) + (i & 3) : 2 * n + ((i & 3) >> 1), half = (INTER ? n & 1 : i & 1) * 8;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + at(row, piece) + half));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + at(row + 16, piece) + half));
            const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
            f.v = u32x4{ua[0], ua[1], ub[0], ub[1]};
        } else {
            const int c = INTER ? 32 * (n >> 1) + 8 * (i >> 2) + 4 * (n & 1) + (i & 3) : 16 * n + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 32 * kk + 4 * g + j;
                f.a[j] = *reinterpret_cast<const float*>(t + at(row, c >> 2) + (c & 3) * 4);
                f.b[j] = *reinterpret_cast<const float*>(t + at(row + 16, c >> 2) + (c & 3) * 4);
            }
        }
        return f;
    }
};
// The row of S^T in LDS that holds value column e: the 16 rows of a tile, as interleaved
// tiles take them, lie together.
__device__ __forceinline__ int state_row(int e) { return (e & ~31) + 16 * ((e >> 2) & 1) + 4 * ((e >> 3) & 3) + (e & 3); }

// Four fp32 values to columns c .. c + 3 (c a multiple of 4) of a row, split over N tiles.
template <typename E, int W, int N>
__device__ __forceinline__ void put4(char* t, int tile_bytes, int row, int c, const f32x4& x) {
    if constexpr (sizeof(E) == 2) {
        f32x4 r = x;
        char* p = t + Tile<E, W>::at(row, c >> 3) + (c & 4) * 2;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const u32x2 w = {pack_opaque(r[0], r[1]), pack_opaque(r[2], r[3])};
            *reinterpret_cast<u32x2*>(p + n * tile_bytes) = w;
            if (n + 1 < N) {
                r[0] -= bf_lo(w[0]);
                r[1] -= bf_hi(w[0]);
                r[2] -= bf_lo(w[1]);
                r[3] -= bf_hi(w[1]);
            }
        }
    } else {
        *reinterpret_cast<f32x4*>(t + Tile<E, W>::at(row, c >> 2)) = x;
    }
}

// ---------------------------------------------------------------- global memory
// Rows of a chunk go through buffer descriptors over exactly its live rows: a load past
// them gives zero, whatever the memory holds there, and a store past them is dropped, with
// no branch and no 64-bit address arithmetic in a lane.  32-bit byte offsets: 64 rows of at
// most 2^23 values each (checked by the host).
constexpr int RSRC_FLAGS = 0x00027000;   // raw buffer of dwords

template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* p, int64_t tok, int64_t stride, int col, int rows,
                                                          int width) {
    const E* base = static_cast<const E*>(p) + tok * stride + col;
    const int bytes = rows > 0 ? ((rows - 1) * (int)stride + width) * (int)sizeof(E) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(base), 0, bytes, RSRC_FLAGS);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// 16-byte pieces of a chunk's rows (W values) held in registers between their load and
// their store to LDS.
template <typename E, int W>
struct Staged {
    using TL = Tile<E, W>;
    static constexpr int PIECES = GC * TL::NP / THREADS, STEP = THREADS / TL::NP;   // rows between a thread's pieces
    static constexpr bool SAME = STEP % (TL::RP * (TL::NP < 16 ? TL::NP : 16)) == 0;   // and their XOR
    u32x4 r[PIECES];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int stride, int tid) {
        const int off = (tid / TL::NP) * stride * (int)sizeof(E) + (tid % TL::NP) * 16;
#pragma unroll
        for (int n = 0; n < PIECES; ++n) r[n] = load16(rs, off + n * (STEP * stride * (int)sizeof(E)));
    }
    __device__ __forceinline__ void store(char* t, int tid) const {
        const int row0 = tid / TL::NP, pc = tid % TL::NP;
        const int a0 = TL::at(row0, pc);
#pragma unroll
        for (int n = 0; n < PIECES; ++n) {
            const int a = SAME ? a0 + n * STEP * TL::ROWB : TL::at(row0 + n * STEP, pc);
            *reinterpret_cast<u32x4*>(t + a) = r[n];
        }
    }
};

// One row's operand in row order: off at value 8 g.
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t r, int off, Frag<uint16_t>& f) { f.v = load16(r, off); }
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t r, int off, Frag<float>& f) {
    f.a = __builtin_bit_cast(f32x4, load16(r, off));
    f.b = __builtin_bit_cast(f32x4, load16(r, off + 16));
}
// Eight neighbouring values of a row, from two interleaved tiles.
__device__ __forceinline__ void store_row8(__amdgpu_buffer_rsrc_t r, int off, const f32x4& x, const f32x4& y, uint16_t) {
    const u32x4 w = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, off, 0, 0);
}
__device__ __forceinline__ void store_row8(__amdgpu_buffer_rsrc_t r, int off, const f32x4& x, const f32x4& y, float) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), r, off + 16, 0, 0);
}

__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    return f32x4{bf_lo(w[0]), bf_hi(w[0]), bf_lo(w[1]), bf_hi(w[1])};
}
__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void store4(uint16_t* p, const f32x4& x) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}
__device__ __forceinline__ void store4(float* p, const f32x4& x) { *reinterpret_cast<f32x4*>(p) = x; }

// ---------------------------------------------------------------- gates
// Running sum of a chunk's gates in powers of two, a token a lane, as a whole part h
// (exact) and a fraction f in [-1/2, 1/2]: exp(G_t - G_s) = 2^((h_t - h_s) + (f_t - f_s))
// keeps the precision of its own size however far the sums have run.  A gate below
// 2^-256 counts as 2^-256, which is 0 in fp32 like itself; so -infinity is a gate of 0.
struct Gates {
    float h, f;
};
template <int CTRL, int ROWS>
__device__ __forceinline__ float lanes_below(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(Gates& s) {
    s.h += lanes_below<CTRL, ROWS>(s.h);
    s.f += lanes_below<CTRL, ROWS>(s.f);
    const float r = rintf(s.f);
    s.h += r;
    s.f -= r;
}
__device__ __forceinline__ Gates gate_sums(float g) {
    Gates s;
    const float x = g * LOG2E;
    if (x < -256.f) {
        s.h = -256.f;
        s.f = 0.f;
    } else {
        s.h = rintf(x);
        s.f = fmaf(g, LOG2E, -s.h) + g * LOG2E_LOW;
    }
    scan_step<0x111, 0xf>(s);   // lanes 1, 2, 4, 8 below in a row of 16 (0 past its start),
    scan_step<0x112, 0xf>(s);
    scan_step<0x114, 0xf>(s);
    scan_step<0x118, 0xf>(s);
    scan_step<0x142, 0xa>(s);   // then the last lane of rows 0 and 2 into rows 1 and 3,
    scan_step<0x143, 0xc>(s);   // and lane 31 into rows 2 and 3
    return s;
}
__device__ __forceinline__ float lane_value(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// Gate sums and weights of a chunk in LDS, a row of 64 each (row 2 is spare):
// h, f; kw, weights of the keys in the state; rw, weights of the state in the rows; cw, of
// a token within its group of 16: 2^(G_b - G_s), G_b the sum at the group's end (backwards
// 2^(G_s - G_b), G_b the sum before its start), times the pairs' scale.
constexpr int GATE_ROWS = 6;
template <bool REV>
__device__ __forceinline__ void put_gates(float* gh, const Gates& gs, float eh, float ef, float pair_scale,
                                          float row_scale, float key_scale, int wave, int lane) {
    // wave 1: kw, wave 2: rw, wave 3: cw (wave 0 fills the spare row), each a power of two of the gate sum's
    // distance from 0, the chunk's end, or its group's end (backwards: its group's start)
    const int at = REV ? ((lane & 48) - 1) & 63 : lane | 15;
    const float gbh = __shfl(gs.h, at, 64), gbf = __shfl(gs.f, at, 64);
    const bool from0 = REV ? wave == 1 : wave == 2;
    const float bh = wave == 3 ? gbh : from0 ? 0.f : eh, bf = wave == 3 ? gbf : from0 ? 0.f : ef;
    const float d = (bh - gs.h) + (bf - gs.f);
    const float sc = wave == 3 ? pair_scale : wave == 2 ? row_scale : key_scale;
    gh[(2 + wave) * GC + lane] = sc * pow2(from0 || (REV && wave == 3) ? -d : d);
    gh[lane] = gs.h;
    gh[GC + lane] = gs.f;
}
// Weights of the tokens of group st in this lane's row (gate sum th + tf): of another group
// the product of cw and this factor, 0 for a group that the row does not see.
template <bool REV>
__device__ __forceinline__ float group_factor(const float* gh, float th, float tf, int st, int wave) {
    const int at = 16 * st + (REV ? -1 : 15);
    const float d = (th - gh[at]) + (tf - gh[GC + at]);
    return pow2((REV ? st > wave : st < wave) ? (REV ? -d : d) : -INFINITY);
}
// Of the row's own group, token s = 4 (lane / 16) + j.
template <bool REV>
__device__ __forceinline__ f32x4 own_weights(const float* gh, float th, float tf, float scale, int wave, int lane) {
    const f32x4 sh = *reinterpret_cast<const f32x4*>(gh + 16 * wave + 4 * (lane >> 4));
    const f32x4 sf = *reinterpret_cast<const f32x4*>(gh + GC + 16 * wave + 4 * (lane >> 4));
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float d = (th - sh[j]) + (tf - sf[j]);
        r[j] = scale * pow2(REV ? -d : d);
    }
    return r;
}

// ---------------------------------------------------------------- the state in accumulators
// Tiles of 16 x 16 of the D x EB state, spread over the four waves: wave w holds the row
// tiles w, w + 4, .. with all column tiles, or at D = 32 row tile w % 2 and half the columns.
template <int D, int EB>
struct StateTiles {
    static constexpr int CT = D / 16, ET = EB / 16;
    static constexpr int CW = CT >= 4 ? CT / 4 : 1;
    static constexpr int EW = CT >= 4 ? ET : ET / 2;
    typedef f32x4 Acc[CW][EW];
    __device__ static __forceinline__ int ct(int wave, int n) { return CT >= 4 ? wave + 4 * n : (wave & 1); }
    __device__ static __forceinline__ int et(int wave, int n) { return CT >= 4 ? n : (wave >> 1) * EW + n; }
};

// S = decay S + sum_s w_s y_s z_s^T over a chunk's tiles.  The weighted keys enter the
// matrix cores as fp32 values split into three bf16 terms: the state is an fp32 sum of
// products rounded as in fp32, which the terms' three products per tile pay for.
template <typename E, int D, int EB>
__device__ __forceinline__ void update_state(typename StateTiles<D, EB>::Acc& S, const char* yt,
                                             const char* zt, const float* w, float decay, int wave, int lane) {
    using ST = StateTiles<D, EB>;
    constexpr int N = sizeof(E) == 2 ? 3 : 1;
#pragma unroll
    for (int a = 0; a < ST::CW; ++a)
#pragma unroll
        for (int b = 0; b < ST::EW; ++b) S[a][b] = S[a][b] * decay;
#pragma unroll
    for (int kk = 0; kk < GC / 32; ++kk) {
        const int g = lane >> 4;
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(w + 32 * kk + 4 * g);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(w + 32 * kk + 16 + 4 * g);
        Frag<E> ys[ST::CW][N];
#pragma unroll
        for (int a = 0; a < ST::CW; ++a) {
            float x[8];
            widen(Tile<E, D>::template cols<false>(yt, kk, ST::ct(wave, a), lane), x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] *= w0[j];
                x[4 + j] *= w1[j];
            }
            split<N>(x, ys[a]);
        }
#pragma unroll
        for (int b = 0; b < ST::EW; ++b) {
            const Frag<E> z = Tile<E, EB>::template cols<false>(zt, kk, ST::et(wave, b), lane);
#pragma unroll
            for (int a = 0; a < ST::CW; ++a)
#pragma unroll
                for (int n = 0; n < N; ++n) S[a][b] = mma(ys[a][N - 1 - n], z, S[a][b]);
        }
    }
}

// Where a state lies in memory: element (c, e) of the walk at c * sc + e * se.
template <int D, int EB>
__device__ __forceinline__ void load_state(typename StateTiles<D, EB>::Acc& S, const float* p,
                                           int sc, int se, int wave, int lane) {
    using ST = StateTiles<D, EB>;
#pragma unroll
    for (int a = 0; a < ST::CW; ++a)
#pragma unroll
        for (int b = 0; b < ST::EW; ++b) {
            const int c = 16 * ST::ct(wave, a) + 4 * (lane >> 4), e = 16 * ST::et(wave, b) + (lane & 15);
#pragma unroll
            for (int j = 0; j < 4; ++j) S[a][b][j] = p ? p[(c + j) * sc + e * se] : 0.f;
        }
}
template <int D, int EB>
__device__ __forceinline__ void store_state(const typename StateTiles<D, EB>::Acc& S, float* p,
                                            int sc, int se, int wave, int lane) {
    using ST = StateTiles<D, EB>;
#pragma unroll
    for (int a = 0; a < ST::CW; ++a)
#pragma unroll
        for (int b = 0; b < ST::EW; ++b) {
            const int c = 16 * ST::ct(wave, a) + 4 * (lane >> 4), e = 16 * ST::et(wave, b) + (lane & 15);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[(c + j) * sc + e * se] = S[a][b][j];
        }
}

// Keeps reads of the tiles inside the loop over heads and chunks: hoisted out of it, they fill
// the registers.  FRESH: their addresses too (the lane number comes back as a value that the
// compiler knows nothing of).
template <bool FRESH>
__device__ __forceinline__ int in_loop(int lane) {
    if constexpr (FRESH) asm volatile("" : "+v"(lane) : : "memory");
    else asm volatile("" : : : "memory");
    return lane;
}

// ---------------------------------------------------------------- the walk
// Whether groups of 16 tokens that none of a wave's rows sees are left out.  Worth its branches
// at D = 128 in bf16, where the matrix cores have most to do (forwards, 16 x 4096 tokens, 8
// heads: 273 -> 233 us; backwards 2 x 4097 tokens, 12 heads over 4: 164 -> 160); at D = 64 it
// costs as much as it saves (16 x 4096, 16 heads: 144 -> 152), and fp32 loses a workgroup of a
// compute unit to its registers (2 x 4096, 70 heads of 32: 122 -> 126).
template <typename E, int D>
constexpr bool SKIP_UNSEEN = sizeof(E) == 2 && D == 128;

// One role: [B, T, heads, D] with a token stride.
struct Role {
    const void* p;
    int64_t stride;
};

struct Walk {
    Role x, y, z, x2;
    void* out;           // [B, T, HK * nx, D]
    float* r;            // x2 . out without a token's own term, [blocks][B, T, HK * nx]
    const float* g;
    const int32_t* lens;
    const float* start;  // state before the walk's first chunk
    int64_t start_pair, start_seg;   // offsets of a (b, kv head) and of a segment
    float* end;          // state after the sequence, or nullptr
    int sc, se;          // strides of a state's key-role and value-role index
    int B, T, HK, nx, ny, nseg, seg_chunks;
    float pair_scale, row_scale, key_scale;
};

// Workgroups go to the eight XCDs in turn; this numbering gives each XCD a run of
// consecutive numbers, so that the heads and value blocks of the same tokens, which read
// neighbouring (or the same) lines, share an L2 at the same time.
__device__ __forceinline__ int xcd_run(int blk, int n) {
    const int x = blk & 7, q = n >> 3, r = n & 7;
    return x * q + min(x, r) + (blk >> 3);
}

// A workgroup walks the chunks of one segment of one (b, kv head), for EB of the value
// columns, with two groups of four waves side by side: one has the rows (its wave w the
// chunk's tokens 16 w .. 16 w + 15) and computes the outputs from tiles and state in LDS, the
// other has the state in its accumulators, adds the chunk to it, and brings the next tiles.
// Between two barriers, while the outputs are stored, it replaces tiles and state.  As eight
// waves the two shorter chains of a chunk run at once and fit 128 registers, four waves a
// SIMD (whole calls, one group doing both and two: forwards 65536 tokens, 6 heads of 64 bf16
// 82.4 and 79 us; 2 x 4096 tokens, 70 heads of 32 fp32 129 and 122; backwards 65536 tokens 232
// and 221, both with 79 segments).
// What bounds it: at D <= 64 in bf16 the tokens' bytes (65536 tokens, 6 heads of 64: 47 us
// forwards, 201 MB at 4.3 TB/s, the matrix cores busy a fifth of it); in fp32 the matrix cores,
// whose 16x16x4 products of a chunk take half of the time (70 heads of 32: 89 us, 294 MB at 3.3
// TB/s); where walks are few and short, the chain from the first load through state, products
// and stores (4 x 1000 tokens, 8 heads over 2 of 128, one chunk each: 13 us).
// Products are formed transposed (Y X^T, then Z^T P^T), so that P leaves the accumulators as
// the next product's operand and a lane stores four neighbouring values of one token.
// P and S are taken as two bf16 terms (three for the sums r, which are fp32 results), so
// that the output is rounded once.
// Pair weights: inside the wave's own 16 tokens each from its two gate sums; with an earlier
// (later) group of 16 as 2^(G_t - G_b) 2^(G_b - G_s) over the sum at the group's end (before
// its start), one exponential a row and one a token instead of one a pair.
template <typename E, int D, int EB, bool DOT>
constexpr int walk_lds() {
    return (GC * D + GC * EB + (sizeof(E) == 4 ? 1 : DOT ? 3 : 2) * EB * D) * (int)sizeof(E) + GATE_ROWS * GC * 4;
}

template <typename E, int D, int EB, bool REV, bool DOT, bool SPLIT>
__device__ __forceinline__ void walk(const Walk& w, int id, char* lds) {
    using TY = Tile<E, D>;
    using TZ = Tile<E, EB>;
    using ST = StateTiles<D, EB>;
    constexpr int NS = sizeof(E) == 4 ? 1 : DOT ? 3 : 2;   // terms of S
    constexpr int NP = sizeof(E) == 4 ? 1 : 2;             // terms of P
    constexpr int KD = D / 32, KE = EB / 32, ET = EB / 16;
    constexpr int YB = GC * TY::ROWB, ZB = GC * TZ::ROWB, SB = EB * TY::ROWB;
    char* yt = lds;
    char* zt = lds + YB;
    char* stt = lds + YB + ZB;   // S transposed, [e][c], NS terms
    float* gh = reinterpret_cast<float*>(lds + YB + ZB + NS * SB);
    const float* kw = gh + 3 * GC;
    const float* rw = kw + GC;
    const float* cw = rw + GC;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;         // in its group
    const int tid = threadIdx.x & (THREADS - 1), lane = tid & 63, li = lane & 15, lg = lane >> 4;
    constexpr int NB = D / EB;
    const int number = id;
    const int eb = id % NB;
    id /= NB;
    const int hk = id % w.HK;
    id /= w.HK;
    const int seg = id % w.nseg, b = id / w.nseg;

    const int T = w.T;
    int len = T;
    if (w.lens) len = min(max(w.lens[b], 0), T);
    const int c0 = seg * w.seg_chunks, c1 = min(c0 + w.seg_chunks, (T + GC - 1) / GC);
    const int live_end = min(c1, (len + GC - 1) / GC);   // chunks from here on hold no live token
    const int64_t tok0 = (int64_t)b * T;
    const int chunks = max(live_end - c0, 0);
    const int first = REV ? live_end - 1 : c0, dir = REV ? -1 : 1;
    const int nx = REV ? 1 : w.nx, ny = REV ? w.ny : 1;   // backwards it is Y and Z that a group has several of
    const bool keep = w.end && (REV ? seg == 0 : seg == w.nseg - 1);   // the state after the last chunk is wanted
    constexpr int ES = (int)sizeof(E);
    constexpr bool FRESH = D == 128;

    // ---- the state's part: tiles, gates and the state
    typename ST::Acc S;
    Staged<E, D> ys;
    Staged<E, EB> zs;
    float graw = 0.f, eh = 0.f, ef = 0.f;
    Gates gs = {0.f, 0.f};
    // a chunk past the walk's end has no rows
    auto fetch = [&](int ci, int hy) {
        const int c = first + dir * ci;
        const int live = ci < chunks ? min(len - c * GC, GC) : 0;
        const int64_t tk = tok0 + (int64_t)c * GC;
        const int h = hk * ny + hy;
        ys.load(rows_of<E>(w.y.p, tk, w.y.stride, h * D, live, D), (int)w.y.stride, tid);
        zs.load(rows_of<E>(w.z.p, tk, w.z.stride, h * D + eb * EB, live, EB), (int)w.z.stride, tid);
        graw = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows_of<float>(w.g, tk, w.HK, hk, live, 1), lane * w.HK * 4, 0, 0));
    };
    auto next_gates = [&]() {
        gs = gate_sums(graw);
        eh = lane_value(gs.h, 63);
        ef = lane_value(gs.f, 63);
    };
    auto begin_state = [&]() {
        load_state<D, EB>(S, w.start ? w.start + ((int64_t)b * w.HK + hk) * w.start_pair + seg * w.start_seg + eb * EB * w.se : nullptr,
                          w.sc, w.se, wave, lane);
        fetch(0, 0);
        next_gates();
    };
    auto put_tiles = [&]() {
        ys.store(yt, tid);
        zs.store(zt, tid);
    };
    auto publish = [&](int at) {
        put_gates<REV>(gh, gs, eh, ef, w.pair_scale, w.row_scale, w.key_scale, wave, at);
#pragma unroll
        for (int a = 0; a < ST::CW; ++a)
#pragma unroll
            for (int e = 0; e < ST::EW; ++e)
                put4<E, D, NS>(stt, SB, state_row(16 * ST::et(wave, e) + (at & 15)), 16 * ST::ct(wave, a) + 4 * (at >> 4), S[a][e]);
    };
    auto end_state = [&]() {
        if (keep)
            store_state<D, EB>(S, w.end + ((int64_t)b * w.HK + hk) * D * D + eb * EB * w.se, w.sc, w.se, wave, lane);
    };

    if constexpr (SPLIT) {
        if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0) {
            begin_state();
            if (chunks > 0) {
                put_tiles();
                publish(lane);
                __syncthreads();
            }
            for (int ci = 0; ci < chunks; ++ci) {
                float decay = pow2(eh + ef);
                for (int hy = 0; hy < ny; ++hy) {
                    const bool last_y = hy + 1 == ny;
                    const int at = in_loop<FRESH>(lane);
                    fetch(last_y ? ci + 1 : ci, last_y ? 0 : hy + 1);
                    if (keep || ci + 1 < chunks) update_state<E, D, EB>(S, yt, zt, kw, decay, wave, at);
                    decay = 1.f;
                    if (last_y) next_gates();
                    __syncthreads();              // the tiles' and the state's reads are over
                    put_tiles();
                    if (last_y) publish(at);
                    __syncthreads();
                }
            }
            end_state();
            return;
        }
    }

    // ---- the rows' part
    const int hx_all = w.HK * w.nx;
    float* const rout = DOT ? w.r + (int64_t)eb * w.B * T * hx_all : nullptr;
    // which wave has which rows turns with the workgroup, so that the long ones spread over the SIMDs
    constexpr bool SKIP = SKIP_UNSEEN<E, D>;
    const int own_group = SKIP ? (wave + number) & 3 : wave;
    const int tl = 16 * own_group + li;                   // this lane's token in a chunk
    Frag<E> xf[KD], x2f[DOT ? KE : 1];
    auto fetch_x = [&](int ci, int hx, Frag<E> (&x)[KD], Frag<E> (&x2)[DOT ? KE : 1]) {
        const int c = first + dir * ci;
        const int live = ci < chunks ? min(len - c * GC, GC) : 0;
        const int64_t tk = tok0 + (int64_t)c * GC;
        const int h = hk * nx + hx;
        const __amdgpu_buffer_rsrc_t rx = rows_of<E>(w.x.p, tk, w.x.stride, h * D, live, D);
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) load_row(rx, (tl * (int)w.x.stride + 8 * lg + 32 * kk) * ES, x[kk]);
        if constexpr (DOT) {
            const __amdgpu_buffer_rsrc_t r2 = rows_of<E>(w.x2.p, tk, w.x2.stride, h * D + eb * EB, live, EB);
#pragma unroll
            for (int kk = 0; kk < KE; ++kk) load_row(r2, (tl * (int)w.x2.stride + 8 * lg + 32 * kk) * ES, x2[kk]);
        }
    };
    fetch_x(0, 0, xf, x2f);

    // rows of dead chunks are zero
    {
        const int t0 = max(c0, live_end) * GC, n = min(c1 * GC, T) - t0;
        constexpr int PC = EB / 4;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        for (int64_t p = tid; p < (int64_t)n * w.nx * PC; p += THREADS) {
            const int row = (int)(p / (w.nx * PC)), rest = (int)(p % (w.nx * PC));
            const int64_t tk = tok0 + t0 + row;
            const int h = hk * w.nx + rest / PC;
            store4(static_cast<E*>(w.out) + (tk * hx_all + h) * D + eb * EB + (rest % PC) * 4, zero);
            if (DOT && rest % PC == 0) rout[tk * hx_all + h] = 0.f;
        }
    }

    f32x4 o[ET];
    float rsum = 0.f;
    auto store_rows = [&](int ci, int hx) {
        const int c = first + dir * ci;
        const bool live = c * GC + tl < len, whole = (c + 1) * GC <= len;
        const int rows = min(T - c * GC, GC);
        const int64_t tk0 = tok0 + (int64_t)c * GC;
        const int h = hk * nx + hx;
        const __amdgpu_buffer_rsrc_t ro = rows_of<E>(w.out, tk0, (int64_t)hx_all * D, h * D + eb * EB, rows, EB);
        if (!whole) {
#pragma unroll
            for (int e = 0; e < ET; ++e)
                if (!live) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int k = 0; k < KE; ++k)
            store_row8(ro, (tl * hx_all * D + 32 * k + 8 * lg) * ES, o[2 * k], o[2 * k + 1], E());
        if constexpr (DOT) {
            float s = rsum + shfl_xor(rsum, 16);
            s += shfl_xor(s, 32);             // all four lanes of a token store the same sum
            const __amdgpu_buffer_rsrc_t rr = rows_of<float>(rout, tk0, hx_all, h, rows, 1);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(live ? s : 0.f), rr, tl * hx_all * 4, 0, 0);
        }
    };
    // the outputs of the tiles in LDS, all heads of X; all but the last head's are stored
    auto compute_rows = [&](int ci, int hy) {
        const bool last_y = hy + 1 == ny;
        const float th = gh[tl], tf = gh[GC + tl], trw = rw[tl];
        for (int hx = 0; hx < nx; ++hx) {
            const bool last_x = hx + 1 == nx;
            const int at = in_loop<FRESH>(lane);
            Frag<E> xn[KD], x2n[DOT ? KE : 1];
            if (!REV || last_y) fetch_x(last_x ? ci + 1 : ci, last_x ? 0 : hx + 1, xn, x2n);
            if (!REV || hy == 0) {
                // from the state: o = S^T x
                rsum = 0.f;
#pragma unroll
                for (int e = 0; e < ET; ++e) {
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = NS - 1; n >= 0; --n)
#pragma unroll
                        for (int kk = 0; kk < KD; ++kk)
                            acc = mma(TY::rows(stt + n * SB, 16 * e, kk, at), xf[kk], acc);
                    o[e] = acc * trw;
                }
                if constexpr (DOT) {
#pragma unroll
                    for (int kk = 0; kk < KE; ++kk) {
                        float u[8];
                        widen(x2f[kk], u);
#pragma unroll
                        for (int j = 0; j < 4; ++j) rsum += u[j] * o[2 * kk][j] + u[4 + j] * o[2 * kk + 1][j];
                    }
                }
            }
            // the chunk's tokens s, 32 at a time: the row's own group of 16 and the groups that come before
            // (backwards: after) it, the others' weight being 0
            float own[4];
            {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f}, m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KD; ++k) acc = mma(TY::rows(yt, 16 * own_group, k, at), xf[k], acc);
                if constexpr (DOT) {
#pragma unroll
                    for (int k = 0; k < KE; ++k) m = mma(TZ::rows(zt, 16 * own_group, k, at), x2f[k], m);
                }
                const f32x4 ow = own_weights<REV>(gh, th, tf, w.pair_scale, own_group, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int s = 4 * lg + j;
                    const float v = acc[j] * ow[j];
                    own[j] = (REV ? s >= li : s <= li) ? v : 0.f;
                    if constexpr (DOT) rsum += s != li ? own[j] * m[j] : 0.f;
                }
            }
#pragma unroll
            for (int kk = 0; kk < GC / 32; ++kk) {
                if (SKIP && (REV ? 2 * kk + 1 < own_group : 2 * kk > own_group)) continue;
                float q[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int st = 2 * kk + u;
                    if (st == (REV ? 0 : GC / 16 - 1) || (SKIP && (REV ? st <= own_group : st >= own_group))) {   // no other group's
#pragma unroll
                        for (int j = 0; j < 4; ++j) q[4 * u + j] = st == own_group ? own[j] : 0.f;
                        continue;
                    }
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f}, m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KD; ++k) acc = mma(TY::rows(yt, 16 * st, k, at), xf[k], acc);
                    if constexpr (DOT) {
#pragma unroll
                        for (int k = 0; k < KE; ++k) m = mma(TZ::rows(zt, 16 * st, k, at), x2f[k], m);
                    }
                    const float rf = group_factor<REV>(gh, th, tf, st, own_group);
                    const f32x4 cs = *reinterpret_cast<const f32x4*>(cw + 16 * st + 4 * lg);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = acc[j] * (cs[j] * rf);
                        if constexpr (DOT) rsum += v * m[j];
                        q[4 * u + j] = st == own_group ? own[j] : v;
                    }
                }
                Frag<E> pf[NP];
                split<NP>(q, pf);
#pragma unroll
                for (int e = 0; e < ET; ++e) {
                    const Frag<E> z = TZ::template cols<true>(zt, kk, e, at);
#pragma unroll
                    for (int n = NP - 1; n >= 0; --n) o[e] = mma(z, pf[n], o[e]);
                }
            }
            if (!REV || last_y) {
#pragma unroll
                for (int kk = 0; kk < KD; ++kk) xf[kk] = xn[kk];
                if constexpr (DOT) {
#pragma unroll
                    for (int kk = 0; kk < KE; ++kk) x2f[kk] = x2n[kk];
                }
            }
            if (!last_x) store_rows(ci, hx);
        }
    };
    if constexpr (SPLIT) {
        if (chunks > 0) __syncthreads();
        for (int ci = 0; ci < chunks; ++ci)
            for (int hy = 0; hy < ny; ++hy) {
                compute_rows(ci, hy);
                __syncthreads();                  // the tiles' and the state's reads are over
                if (!REV || hy + 1 == ny) store_rows(ci, nx - 1);
                __syncthreads();
            }
    } else {
        begin_state();
        for (int ci = 0; ci < chunks; ++ci) {
            float decay = pow2(eh + ef);
            for (int hy = 0; hy < ny; ++hy) {
                const bool last_y = hy + 1 == ny;
                __syncthreads();                  // the tiles' and the state's reads are over
                put_tiles();
                if (hy == 0) publish(lane);
                __syncthreads();
                fetch(last_y ? ci + 1 : ci, last_y ? 0 : hy + 1);
                compute_rows(ci, hy);
                if (!REV || last_y) store_rows(ci, nx - 1);
                if (keep || ci + 1 < chunks) update_state<E, D, EB>(S, yt, zt, kw, decay, wave, lane);
                decay = 1.f;
                if (last_y) next_gates();
            }
        }
        end_state();
    }
}

// At D = 128 in bf16 one group of waves does both parts in turn: split, the rows' part does
// not fit 128 registers, and past them a compute unit holds one workgroup of eight waves
// instead of two of four (backwards, 2 x 4097 tokens, 12 heads over 4: 117 us, split 148).
// In fp32 either way it holds one, and eight waves are better than four (forwards, 4 x 2048
// tokens, 8 heads: 111 us, not split 125).
template <typename E, int D>
constexpr bool split_walk() { return D <= 64 || sizeof(E) == 4; }
template <typename E, int D>
constexpr int walk_threads() { return split_walk<E, D>() ? 2 * THREADS : THREADS; }

template <typename E, int D, int EB>
__global__ void __launch_bounds__((walk_threads<E, D>()), (!split_walk<E, D>() || D == 128 ? 2 : 4)) gated_walk(Walk w) {
    __shared__ __attribute__((aligned(16))) char lds[walk_lds<E, D, EB, false>()];
    walk<E, D, EB, false, false, split_walk<E, D>()>(w, xcd_run(blockIdx.x, gridDim.x), lds);
}

// ---------------------------------------------------------------- dk and dv together
// Backwards over a segment with X = k and v, Y = q, Z = do: the pair products q . k and
// do . v serve dk, dv and k . dk alike, the tiles are read once and the state's gradient D is
// summed once, where two walks would do each twice.  D lies in LDS once, transposed ([e][c]):
// dv contracts it over c (its columns), dk over e (its rows, by transposing reads).  D <= 64:
// at 128 the state of all columns leaves room for one workgroup of a compute unit, and dk and
// dv are walks of their own.
// One group of waves computes dk and k . dk and brings the tiles of q, the other dv, with D
// in its accumulators, and the tiles of do.
// Bound by vector instructions and LDS reads together: at 65536 tokens, 6 heads of 64 bf16 the
// launch of all gradients takes 157 us, 538 MB at 3.4 TB/s, with the vector units busy half of
// it, LDS two fifths (a third of that are bank conflicts of the transposing reads of
// interleaved tiles) and the matrix cores a fifth.
struct Back {
    Role q, k, v, dout;
    void* dk;
    void* dv;            // [B, T, HK, D]
    float* r;            // k . dk without a token's own term, [B, T, HK]
    const float* g;
    const int32_t* lens;
    const float* start;  // gradient of the state behind each segment, [B*HK][nseg][D*D], or nullptr (zero)
    float* end;          // gradient of the initial state, or nullptr
    int B, T, HK, G, nseg, seg_chunks;
    float scale;
};

template <typename E, int D>
__device__ __forceinline__ void back(const Back& w, int id, char* lds) {
    using TL = Tile<E, D>;
    using ST = StateTiles<D, D>;
    constexpr int NS = sizeof(E) == 4 ? 1 : 3;             // terms of D (two for dv, three for k . dk)
    constexpr int NSV = sizeof(E) == 4 ? 1 : 2;
    constexpr int NP = sizeof(E) == 4 ? 1 : 2;
    constexpr int KD = D / 32, DT = D / 16, ES = (int)sizeof(E);
    constexpr int TB = GC * TL::ROWB, SB = D * TL::ROWB;
    char* yt = lds;
    char* zt = lds + TB;
    char* stt = lds + 2 * TB;
    float* gh = reinterpret_cast<float*>(lds + 2 * TB + NS * SB);
    const float* kw = gh + 3 * GC;
    const float* rw = kw + GC;
    const float* cw = rw + GC;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;         // in its group
    const bool dk_group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) == 0;
    const int tid = threadIdx.x & (THREADS - 1), lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int hk = id % w.HK;
    id /= w.HK;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int T = w.T;
    int len = T;
    if (w.lens) len = min(max(w.lens[b], 0), T);
    const int c0 = seg * w.seg_chunks, c1 = min(c0 + w.seg_chunks, (T + GC - 1) / GC);
    const int live_end = min(c1, (len + GC - 1) / GC);
    const int64_t tok0 = (int64_t)b * T, pair = (int64_t)b * w.HK + hk;
    const int chunks = max(live_end - c0, 0);
    const int tl = 16 * wave + li;
    const bool keep = w.end && seg == 0;
    constexpr bool FRESH = true;

    // k or v of a chunk's rows, this lane's token; a chunk past the walk's end has no rows
    auto fetch_x = [&](int ci, const Role& x, Frag<E> (&f)[KD]) {
        const int c = live_end - 1 - ci;
        const int live = ci < chunks ? min(len - c * GC, GC) : 0;
        const __amdgpu_buffer_rsrc_t r = rows_of<E>(x.p, tok0 + (int64_t)c * GC, x.stride, hk * D, live, D);
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) load_row(r, (tl * (int)x.stride + 8 * lg + 32 * kk) * ES, f[kk]);
    };
    auto store_rows = [&](int c, void* out, f32x4 (&o)[DT]) {
        const __amdgpu_buffer_rsrc_t r = rows_of<E>(out, tok0 + (int64_t)c * GC, (int64_t)w.HK * D, hk * D, min(T - c * GC, GC), D);
        if ((c + 1) * GC > len) {
#pragma unroll
            for (int e = 0; e < DT; ++e)
                if (c * GC + tl >= len) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int k = 0; k < KD; ++k) store_row8(r, (tl * w.HK * D + 32 * k + 8 * lg) * ES, o[2 * k], o[2 * k + 1], E());
    };
    // rows of dead chunks are zero
    auto zero_rows = [&](void* out) {
        const int t0 = max(c0, live_end) * GC, n = min(c1 * GC, T) - t0;
        constexpr int PC = D / 4;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        for (int p = tid; p < n * PC; p += THREADS)
            store4(static_cast<E*>(out) + ((tok0 + t0 + p / PC) * w.HK + hk) * D + (p % PC) * 4, zero);
    };
    // The row's own group of 16 tokens: t >= this one
    auto own_pairs = [&](const f32x4& a, const f32x4& ow, float (&o)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = 4 * lg + j >= li ? a[j] * ow[j] : 0.f;
    };

    if (!dk_group) {
        typename ST::Acc S;
        load_state<D, D>(S, w.start ? w.start + (pair * w.nseg + seg) * D * D : nullptr, D, 1, wave, lane);
        Staged<E, D> zs;
        float graw = 0.f;
        auto fetch = [&](int ci, int hy) {
            const int c = live_end - 1 - ci;
            const int live = ci < chunks ? min(len - c * GC, GC) : 0;
            const int64_t tk = tok0 + (int64_t)c * GC;
            zs.load(rows_of<E>(w.dout.p, tk, w.dout.stride, (hk * w.G + hy) * D, live, D), (int)w.dout.stride, tid);
            graw = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows_of<float>(w.g, tk, w.HK, hk, live, 1), lane * w.HK * 4, 0, 0));
        };
        fetch(0, 0);
        Frag<E> kf[KD], kn[KD];
        fetch_x(0, w.k, kf);
        zero_rows(w.dv);
        Gates gs = gate_sums(graw);
        float eh = lane_value(gs.h, 63), ef = lane_value(gs.f, 63);
        auto publish = [&](int at) {
            put_gates<true>(gh, gs, eh, ef, w.scale, 1.f, w.scale, wave, at);
#pragma unroll
            for (int a = 0; a < ST::CW; ++a)
#pragma unroll
                for (int e = 0; e < ST::EW; ++e)
                    put4<E, D, NS>(stt, SB, state_row(16 * ST::et(wave, e) + (at & 15)), 16 * ST::ct(wave, a) + 4 * (at >> 4), S[a][e]);
        };
        if (chunks > 0) {
            zs.store(zt, tid);
            publish(lane);
            __syncthreads();
        }
        f32x4 ov[DT];
        for (int ci = 0; ci < chunks; ++ci) {
            float decay = pow2(eh + ef);
            for (int hy = 0; hy < w.G; ++hy) {
                const bool last = hy + 1 == w.G;
                const int at = in_loop<FRESH>(lane);
                fetch(last ? ci + 1 : ci, last ? 0 : hy + 1);
                if (hy == 0) {
                    fetch_x(ci + 1, w.k, kn);
                    // from the state: dv = D^T k
                    const float trw = rw[tl];
#pragma unroll
                    for (int e = 0; e < DT; ++e) {
                        f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int n = NSV - 1; n >= 0; --n)
#pragma unroll
                            for (int kk = 0; kk < KD; ++kk) a = mma(TL::rows(stt + n * SB, 16 * e, kk, at), kf[kk], a);
                        ov[e] = a * trw;
                    }
                }
                const float th = gh[tl], tf = gh[GC + tl];
                float pown[4];
                {
                    f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KD; ++k) a = mma(TL::rows(yt, 16 * wave, k, at), kf[k], a);
                    own_pairs(a, own_weights<true>(gh, th, tf, w.scale, wave, lane), pown);
                }
#pragma unroll
                for (int kk = 0; kk < GC / 32; ++kk) {
                    float pq[8];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int st = 2 * kk + u;
                        if (st == 0) {   // no other group's
#pragma unroll
                            for (int j = 0; j < 4; ++j) pq[4 * u + j] = st == wave ? pown[j] : 0.f;
                            continue;
                        }
                        f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < KD; ++k) a = mma(TL::rows(yt, 16 * st, k, at), kf[k], a);
                        const float rf = group_factor<true>(gh, th, tf, st, wave);
                        const f32x4 cs = *reinterpret_cast<const f32x4*>(cw + 16 * st + 4 * lg);
#pragma unroll
                        for (int j = 0; j < 4; ++j) pq[4 * u + j] = st == wave ? pown[j] : a[j] * (cs[j] * rf);
                    }
                    Frag<E> pf[NP];
                    split<NP>(pq, pf);
#pragma unroll
                    for (int e = 0; e < DT; ++e) {
                        const Frag<E> z = TL::template cols<true>(zt, kk, e, at);
#pragma unroll
                        for (int n = NP - 1; n >= 0; --n) ov[e] = mma(z, pf[n], ov[e]);
                    }
                }
                if (keep || ci + 1 < chunks) update_state<E, D, D>(S, yt, zt, kw, decay, wave, at);
                decay = 1.f;
                if (last) {
                    gs = gate_sums(graw);
                    eh = lane_value(gs.h, 63);
                    ef = lane_value(gs.f, 63);
                }
                __syncthreads();                  // the tiles' and the state's reads are over
                zs.store(zt, tid);
                if (last) publish(at);
                __syncthreads();
            }
            store_rows(live_end - 1 - ci, w.dv, ov);
#pragma unroll
            for (int kk = 0; kk < KD; ++kk) kf[kk] = kn[kk];
        }
        if (keep) store_state<D, D>(S, w.end + pair * D * D, D, 1, wave, lane);
        return;
    }

    Staged<E, D> ys;
    auto fetch = [&](int ci, int hy) {
        const int c = live_end - 1 - ci;
        const int live = ci < chunks ? min(len - c * GC, GC) : 0;
        ys.load(rows_of<E>(w.q.p, tok0 + (int64_t)c * GC, w.q.stride, (hk * w.G + hy) * D, live, D), (int)w.q.stride, tid);
    };
    fetch(0, 0);
    Frag<E> kf[KD], vf[KD], kn[KD], vn[KD];
    fetch_x(0, w.k, kf);
    fetch_x(0, w.v, vf);
    zero_rows(w.dk);
    for (int t = max(c0, live_end) * GC + tid; t < min(c1 * GC, T); t += THREADS) w.r[(tok0 + t) * w.HK + hk] = 0.f;
    f32x4 ok[DT];
    float rsum = 0.f;
    if (chunks > 0) {
        ys.store(yt, tid);
        __syncthreads();
    }
    for (int ci = 0; ci < chunks; ++ci) {
        const int c = live_end - 1 - ci;
        const int64_t tk0 = tok0 + (int64_t)c * GC;
        for (int hy = 0; hy < w.G; ++hy) {
            const bool last = hy + 1 == w.G;
            const int at = in_loop<FRESH>(lane);
            fetch(last ? ci + 1 : ci, last ? 0 : hy + 1);
            if (hy == 0) {
                fetch_x(ci + 1, w.k, kn);
                fetch_x(ci + 1, w.v, vn);
                // from the state: dk = D v
                const float trw = rw[tl];
                rsum = 0.f;
#pragma unroll
                for (int e = 0; e < DT; ++e) {
                    f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = NS - 1; n >= 0; --n)
#pragma unroll
                        for (int kk = 0; kk < KD; ++kk)
                            a = mma(TL::template cols<true>(stt + n * SB, kk, e, at), vf[kk], a);   // rows by state_row(): e in row order
                    ok[e] = a * trw;
                }
#pragma unroll
                for (int kk = 0; kk < KD; ++kk) {
                    float u[8];
                    widen(kf[kk], u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) rsum += u[j] * ok[2 * kk][j] + u[4 + j] * ok[2 * kk + 1][j];
                }
            }
            const float th = gh[tl], tf = gh[GC + tl];
            float mown[4];
            {
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, m = a;
#pragma unroll
                for (int k = 0; k < KD; ++k) {
                    a = mma(TL::rows(yt, 16 * wave, k, at), kf[k], a);
                    m = mma(TL::rows(zt, 16 * wave, k, at), vf[k], m);
                }
                own_pairs(m, own_weights<true>(gh, th, tf, w.scale, wave, lane), mown);
#pragma unroll
                for (int j = 0; j < 4; ++j) rsum += 4 * lg + j != li ? mown[j] * a[j] : 0.f;
            }
#pragma unroll
            for (int kk = 0; kk < GC / 32; ++kk) {
                float mq[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int st = 2 * kk + u;
                    if (st == 0) {   // no other group's
#pragma unroll
                        for (int j = 0; j < 4; ++j) mq[4 * u + j] = st == wave ? mown[j] : 0.f;
                        continue;
                    }
                    f32x4 a = {0.f, 0.f, 0.f, 0.f}, m = a;
#pragma unroll
                    for (int k = 0; k < KD; ++k) {
                        a = mma(TL::rows(yt, 16 * st, k, at), kf[k], a);
                        m = mma(TL::rows(zt, 16 * st, k, at), vf[k], m);
                    }
                    const float rf = group_factor<true>(gh, th, tf, st, wave);
                    const f32x4 cs = *reinterpret_cast<const f32x4*>(cw + 16 * st + 4 * lg);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float mv = m[j] * (cs[j] * rf);
                        rsum += mv * a[j];
                        mq[4 * u + j] = st == wave ? mown[j] : mv;
                    }
                }
                Frag<E> mf[NP];
                split<NP>(mq, mf);
#pragma unroll
                for (int e = 0; e < DT; ++e) {
                    const Frag<E> y = TL::template cols<true>(yt, kk, e, at);
#pragma unroll
                    for (int n = NP - 1; n >= 0; --n) ok[e] = mma(y, mf[n], ok[e]);
                }
            }
            __syncthreads();                      // the tiles' and the state's reads are over
            ys.store(yt, tid);
            if (last) {
                store_rows(c, w.dk, ok);
                float s = rsum + shfl_xor(rsum, 16);
                s += shfl_xor(s, 32);             // all four lanes of a token store the same sum
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(c * GC + tl < len ? s : 0.f),
                                                      rows_of<float>(w.r, tk0, w.HK, hk, min(T - c * GC, GC), 1), tl * w.HK * 4, 0, 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) {
            kf[kk] = kn[kk];
            vf[kk] = vn[kk];
        }
    }
}

// All three gradients in one launch: the walks for dq and for dk and dv (at D = 128 for dv
// and for dk) do not wait for each other, short problems run them side by side and long ones
// fill the last round (2 x 4097 tokens, 12 heads over 4 of 128, whole call: 196 us in launches
// of their own, 165 in one).  The walks of one segment have neighbouring numbers, the longest
// first; numbered from the last they took as long.
struct Grads {
    Walk q, v, k;   // D = 128: v and k
    Back kv;        // D <= 64
};
template <typename E, int D, int EB>
__global__ void __launch_bounds__((walk_threads<E, D>()), (!split_walk<E, D>() ? 2 : sizeof(E) == 2 || D == 32 ? 4 : 2))
    gated_grads(Grads w) {
    constexpr bool SPLIT = split_walk<E, D>();
    constexpr int NB = D / EB;
    constexpr int LDS = walk_lds<E, D, EB, true>();   // of D <= 64 the same for back()
    __shared__ __attribute__((aligned(16))) char lds[LDS];
    const int n = xcd_run(blockIdx.x, gridDim.x);
    if constexpr (NB == 1) {
        static_assert(D == EB, "back() has all columns");
        if ((n & 1) == 0) back<E, D>(w.kv, n >> 1, lds);
        else walk<E, D, EB, false, true, true>(w.q, n >> 1, lds);
    } else {
        const int role = (n / NB) % 3, id = n / (3 * NB) * NB + n % NB;
        if (role == 0) walk<E, D, EB, true, true, SPLIT>(w.k, id, lds);
        else if (role == 1) walk<E, D, EB, false, true, SPLIT>(w.q, id, lds);
        else walk<E, D, EB, true, false, SPLIT>(w.v, id, lds);
    }
}

// ---------------------------------------------------------------- segments
// What each segment adds to the state, from zero, for the forward state (Y = k, Z = v) and,
// with two roles, for the backward one (Y = q, Z = do of all the group's heads), and the
// segment's decay.  Bound by the bytes of what it reads: 65536 tokens, 6 heads of 64 bf16: 26 us
// for 101 MB (3.9 TB/s) with one role, 43 us for 201 MB (4.7) with two; a wave has its state
// tiles in registers and stages the next chunk's rows while it adds this one's.
struct Local {
    Role y[2], z[2];
    int ny[2];
    float* st[2];
    int64_t pair[2], first[2];   // offset of a (b, kv head); of segment 0's place in it
    float key_scale[2];
    int roles;
    float* dec;
    const float* g;
    const int32_t* lens;
    int B, T, HK, nseg, seg_chunks;
};

template <typename E, int D, int EB>
__global__ void __launch_bounds__(THREADS) gated_local(Local w) {
    using TY = Tile<E, D>;
    using TZ = Tile<E, EB>;
    using ST = StateTiles<D, EB>;
    constexpr int YB = GC * TY::ROWB, ZB = GC * TZ::ROWB;
    __shared__ __attribute__((aligned(16))) char lds[YB + ZB + GC * 4];
    char* yt = lds;
    char* zt = lds + YB;
    float* kw = reinterpret_cast<float*>(lds + YB + ZB);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    constexpr int NB = D / EB;
    int id = xcd_run(blockIdx.x, gridDim.x);
    const int eb = id % NB;
    id /= NB;
    const int hk = id % w.HK;
    id /= w.HK;
    const int role = id % w.roles;
    id /= w.roles;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int T = w.T;
    int len = T;
    if (w.lens) len = min(max(w.lens[b], 0), T);
    const int c0 = seg * w.seg_chunks, c1 = min(c0 + w.seg_chunks, (T + GC - 1) / GC);
    const int live_end = min(c1, (len + GC - 1) / GC);
    const int ny = role ? w.ny[1] : w.ny[0];
    const Role ry = role ? w.y[1] : w.y[0], rz = role ? w.z[1] : w.z[0];
    const float key_scale = role ? w.key_scale[1] : w.key_scale[0];
    const int64_t tok0 = (int64_t)b * T;

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    typename ST::Acc S;
#pragma unroll
    for (int a = 0; a < ST::CW; ++a)
#pragma unroll
        for (int e = 0; e < ST::EW; ++e) S[a][e] = zero;
    float dec = 1.f;

    const int chunks = max(live_end - c0, 0);
    const int first = role ? live_end - 1 : c0, dir = role ? -1 : 1;
    Staged<E, D> ys;
    Staged<E, EB> zs;
    float graw = 0.f;
    auto fetch = [&](int ci, int hy) {
        const int c = first + dir * ci;
        const int live = ci < chunks ? min(len - c * GC, GC) : 0;
        const int64_t tk = tok0 + (int64_t)c * GC;
        const int h = hk * ny + hy;
        ys.load(rows_of<E>(ry.p, tk, ry.stride, h * D, live, D), (int)ry.stride, tid);
        zs.load(rows_of<E>(rz.p, tk, rz.stride, h * D + eb * EB, live, EB), (int)rz.stride, tid);
        graw = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows_of<float>(w.g, tk, w.HK, hk, live, 1), lane * w.HK * 4, 0, 0));
    };
    fetch(0, 0);
    for (int ci = 0; ci < chunks; ++ci) {
        const Gates gs = gate_sums(graw);
        const float eh = lane_value(gs.h, 63), ef = lane_value(gs.f, 63);
        float decay = pow2(eh + ef);
        dec *= decay;
        const float key = key_scale * (role ? pow2(gs.h + gs.f) : pow2((eh - gs.h) + (ef - gs.f)));
        for (int hy = 0; hy < ny; ++hy) {
            __syncthreads();
            ys.store(yt, tid);
            zs.store(zt, tid);
            kw[lane] = key;                       // every wave the same
            __syncthreads();
            const bool last_y = hy + 1 == ny;
            fetch(last_y ? ci + 1 : ci, last_y ? 0 : hy + 1);
            update_state<E, D, EB>(S, yt, zt, kw, decay, wave, lane);
            decay = 1.f;
        }
    }
    const int64_t pair = (int64_t)b * w.HK + hk;
    float* st = (role ? w.st[1] : w.st[0]) + pair * (role ? w.pair[1] : w.pair[0]) + (role ? w.first[1] : w.first[0]) +
                (int64_t)seg * D * D;
    store_state<D, EB>(S, st + eb * EB, D, 1, wave, lane);
    if (tid == 0 && eb == 0 && role == 0) w.dec[pair * w.nseg + seg] = dec;
}

// Joins the segments: fst[j] becomes the state before segment j (j = nseg: after the last),
// rst[j] the gradient of the state after segment j.  A workgroup has 64 elements of one
// pair's states, each of its waves a run of up to JOIN_RUN segments of them: all of a run's
// loads are in flight at once, the runs are joined through LDS.  Bound by its states' bytes and,
// where they are few, by the latency of one read, one exchange and one write: 79 segments of 6
// heads of 64 forwards 6.3 us (16 MB), 128 both ways 12.5 us (50 MB at 4.0 TB/s); 8 pairs of 128, 22 segments both
// ways 11.3 us (46 MB at 4.1 TB/s).
constexpr int JOIN_WAVES = 16, JOIN_RUN = 16;
__global__ void __launch_bounds__(64 * JOIN_WAVES) gated_join(float* fst, const float* s0, float* rst, const float* ds1,
                                                             const float* dec, int nseg, int DD) {
    __shared__ float sums[JOIN_WAVES][64];
    __shared__ float decays[JOIN_WAVES];
    const int64_t pair = blockIdx.y;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6, lane = threadIdx.x & 63;
    const bool rev = (int)blockIdx.x * 64 >= DD;     // backwards segment nseg - 1 comes first
    const int i = blockIdx.x * 64 - (rev ? DD : 0) + lane;
    const float* d = dec + pair * nseg;
    const float* start = rev ? ds1 : s0;
    float* p = rev ? rst + pair * nseg * DD + i : fst + pair * (nseg + 1) * DD + i;
    float carry = start ? start[pair * DD + i] : 0.f;
    // segment j's own sum lies at place j + 1 forwards and j backwards; what comes before
    // it goes to place j
    const int64_t own = rev ? 0 : DD;
    for (int base = 0; base < nseg; base += waves * JOIN_RUN) {
        const int n = min(nseg - base, waves * JOIN_RUN), per = (n + waves - 1) / waves;
        const int k0 = wave * per, mine = min(per, n - k0);     // may be none
        float loc[JOIN_RUN], a[JOIN_RUN];
        float s = 0.f, prod = 1.f;
#pragma unroll
        for (int u = 0; u < JOIN_RUN; ++u) {
            const int k = base + k0 + u, j = rev ? nseg - 1 - k : k;
            loc[u] = 0.f;
            a[u] = 1.f;
            if (u < mine) {
                loc[u] = p[(int64_t)j * DD + own];
                a[u] = d[j];
            }
        }
#pragma unroll
        for (int u = 0; u < JOIN_RUN; ++u) {
            s = a[u] * s + loc[u];
            prod *= a[u];
        }
        sums[wave][lane] = s;
        if (lane == 0) decays[wave] = prod;
        __syncthreads();                              // also: every load above is done before a store below
        float before = carry;
        for (int k = 0; k < waves; ++k) {
            if (k == wave) before = carry;
            carry = decays[k] * carry + sums[k][lane];
        }
#pragma unroll
        for (int u = 0; u < JOIN_RUN; ++u) {
            const int k = base + k0 + u, j = rev ? nseg - 1 - k : k;
            if (u < mine) {
                p[(int64_t)j * DD] = before;
                before = a[u] * before + loc[u];
            }
        }
        __syncthreads();
    }
    if (!rev && wave == 0) p[(int64_t)nseg * DD] = carry;
}

// ---------------------------------------------------------------- gradient of the gates
// dg_t sums the products of pairs s < t <= t', which is
//   sum_{t' >= t} q_t' . dq_t' - sum_{s >= t} k_s . dk_s + <S, dL/dS> at the segment's end
// (a token's product with itself left out of both sums, where it would only cancel).  A
// workgroup takes one segment of one (b, kv head): at most 16 chunks, four tokens a thread
// from the last; the sums run in 64 bits, since they cancel.  A gate of 0 passes no gradient,
// and no pair crosses it: the sums start again there, so that packed sequences leave nothing
// in each other's gradients, not even what a cancelled sum rounds to.
// Bound by latency: few bytes, and two rounds of loads (65536 tokens, 6 heads of 64: 10.1 us; 2 x
// 4097, 12 heads over 4 of 128: 8.4 us, 15.8 with the loads one after the other).
struct GateGrad {
    const float* rq;
    const float* rk;
    const float* fst;    // state after each segment
    int64_t fst_pair;
    const float* rst;    // its gradient, or nullptr (zero)
    const float* g;
    const int32_t* lens;
    float* dg;
    int B, T, HK, nx, nb, nseg, seg_chunks;
};
template <int D>
__global__ void __launch_bounds__(THREADS) gated_gate_grad(GateGrad w) {
    constexpr int DD = D * D;
    constexpr int N = GATED_MAX_CHUNKS * GC / THREADS;
    constexpr float ZERO_GATE = -104.f;               // exp of less is zero in fp32
    __shared__ double part[2][4];
    __shared__ int s_cut[4];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    int id = xcd_run(blockIdx.x, gridDim.x);
    const int hk = id % w.HK;
    id /= w.HK;
    const int seg = id % w.nseg, b = id / w.nseg;
    const int64_t pair = (int64_t)b * w.HK + hk;
    const int T = w.T;
    int len = T;
    if (w.lens) len = min(max(w.lens[b], 0), T);
    const int t0 = seg * w.seg_chunks * GC, t1 = min(t0 + w.seg_chunks * GC, T), live = max(min(t1, len), t0);
    const int64_t tok0 = (int64_t)b * T, tokens = (int64_t)w.B * T;
    // this thread's tokens, descending: thread 0 has the last ones.  Loads of all four are under
    // way at once, those behind the segment's start with an address in it
    const int last = live - 1 - tid * N;
    double v[N];
    float gate[N];
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0.0;
        gate[n] = 0.f;
    }
    if (live > t0) {
        int64_t tk[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            tk[n] = (tok0 + max(last - n, t0)) * w.HK + hk;
            gate[n] = w.g[tk[n]];
        }
        const int64_t block = tokens * w.HK;
        for (int e = 0; e < w.nb; ++e) {
            for (int h = 0; h < w.nx; ++h)
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] += (double)w.rq[(e * block + tk[n]) * w.nx + h];
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] -= (double)w.rk[e * block + tk[n]];
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (last - n < t0) {
                v[n] = 0.0;
                gate[n] = 0.f;
            }
    }
    double cross = 0.0;
    if (w.rst) {
        const float* S = w.fst + pair * w.fst_pair + (int64_t)seg * DD;
        const float* R = w.rst + (pair * w.nseg + seg) * DD;
        constexpr int RUN = THREADS * 4, UN = DD / RUN < 4 ? DD / RUN : 4;
        for (int i = tid * 4; i < DD; i += UN * RUN) {
            f32x4 x[UN], y[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                x[u] = load4(S + i + u * RUN);
                y[u] = load4(R + i + u * RUN);
            }
#pragma unroll
            for (int u = 0; u < UN; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) cross += (double)x[u][j] * (double)y[u][j];
        }
    }
    int cut = 0;                                      // a gate of 0 among the tokens so far
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bool zero = gate[n] < ZERO_GATE;
        sum = zero ? 0.0 : sum + v[n];
        v[n] = sum;
        cut |= zero;
    }
    double s = sum;                                   // sum since the last cut, up to this lane's tokens
    int f = cut;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(s, o, 64);
        const int uf = __shfl_up(f, o, 64);
        if (lane >= o) {
            s += f ? 0.0 : u;
            f |= uf;
        }
        cross += __shfl_xor(cross, o, 64);
    }
    if (lane == 63) {
        part[0][wave] = s;
        s_cut[wave] = f;
    }
    if (lane == 0) part[1][wave] = cross;
    s = __shfl_up(s, 1, 64);
    f = __shfl_up(f, 1, 64);
    __syncthreads();
    double before = (part[1][0] + part[1][1]) + (part[1][2] + part[1][3]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < wave) before = part[0][k] + (s_cut[k] ? 0.0 : before);
    if (lane) before = s + (f ? 0.0 : before);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int t = last - n;
        if (gate[n] < ZERO_GATE) before = 0.0;        // v[n] is 0 there, and counts from there on
        if (t >= t0) w.dg[(tok0 + t) * w.HK + hk] = (float)(before + v[n]);
    }
    for (int t = live + tid; t < t1; t += THREADS) w.dg[(tok0 + t) * w.HK + hk] = 0.f;
}

// ---------------------------------------------------------------- one token
// S' = exp(g) S + k v^T in place, o = scale S'^T q.  Bound by the state's bytes: read and
// written once.  A workgroup has EB value columns of one (row, kv head): a thread four
// columns of every RG-th key row, sixteen bytes a load, the whole state's share in registers,
// so that every byte is asked for before the first is needed.  240 rows of 12 heads of 128,
// 377 MB: 80 us, 4.7 TB/s (the same pool over and over, from the last-level cache: 56 us); one row
// of 6 heads of 64: 3.3 us.
// Rows that name the same slot are that sequence's next tokens, in the order of the rows:
// the first of them does them all, the others leave.
template <typename E, int D, int EB>
__global__ void __launch_bounds__(THREADS) gated_step(GatedStep w) {
    constexpr int CL = EB / 4, RG = THREADS / CL, R = D / RG;   // lanes of a row, row groups, rows of a thread
    static_assert(CL <= 64 && R >= 1, "a row of columns lies in one wave");
    __shared__ float part[4][EB];
    __shared__ int s_next[4];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, cl = tid % CL, rg = tid / CL;
    constexpr int NB = D / EB;
    int id = blockIdx.x;
    const int eb = id % NB;
    id /= NB;
    const int hk = id % w.HK, row0 = id / w.HK;
    const int G = w.H / w.HK, e0 = eb * EB + 4 * cl;
    const E* const q = static_cast<const E*>(w.q);
    const E* const k = static_cast<const E*>(w.k);
    const E* const v = static_cast<const E*>(w.v);
    E* const out = static_cast<E*>(w.out);

    const int slot = w.slots ? w.slots[row0] : row0;
    if (slot < 0 || slot >= w.nslots) {       // no sequence: the output is zero
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        for (int p = tid; p < G * CL; p += THREADS)
            store4(out + ((int64_t)row0 * w.H + hk * G + p / CL) * D + eb * EB + 4 * (p % CL), zero);
        return;
    }
    float* const st = w.state + ((int64_t)slot * w.HK + hk) * D * D + e0;
    f32x4 S[R];
#pragma unroll
    for (int n = 0; n < R; ++n) S[n] = *reinterpret_cast<const f32x4*>(st + (int64_t)(rg + n * RG) * D);

    // the next row after `row` of the same slot (B if there is none); a row before row0 gives -1
    auto next_row = [&](int row, bool look_back) {
        int found = w.B;
        for (int i0 = look_back ? 0 : (row + 1) / THREADS * THREADS; i0 < w.B; i0 += THREADS) {
            const int i = i0 + tid;
            const bool same = i < w.B && i != row && (look_back || i > row) && w.slots[i] == slot;
            const unsigned long long m = __ballot(same);
            __syncthreads();
            if (lane == 0) s_next[wave] = m ? i0 + 64 * wave + __ffsll(m) - 1 : w.B;
            __syncthreads();
            found = min(min(s_next[0], s_next[1]), min(s_next[2], s_next[3]));
            if (found < w.B) break;
        }
        return found;
    };
    int next = w.B;
    if (w.slots) {
        next = next_row(row0, true);
        if (next < row0) return;              // an earlier row does this one
    }
    for (int row = row0; row < w.B; row = next, next = w.slots && row < w.B ? next_row(row, false) : w.B) {
        const E* kr = k + row * w.ks + (int64_t)hk * D;
        const f32x4 vv = load4(v + row * w.vs + (int64_t)hk * D + e0);
        const float g = w.g[(int64_t)row * w.HK + hk];
        const float a = expf(g);
#pragma unroll
        for (int n = 0; n < R; ++n) {
            float kc;
            if constexpr (sizeof(E) == 2) kc = bf_lo(kr[rg + n * RG]); else kc = kr[rg + n * RG];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[n][j] = fmaf(kc, vv[j], a * S[n][j]);
        }
        for (int h = 0; h < G; ++h) {
            const E* qr = q + row * w.qs + (int64_t)(hk * G + h) * D;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < R; ++n) {
                float qc;
                if constexpr (sizeof(E) == 2) qc = bf_lo(qr[rg + n * RG]); else qc = qr[rg + n * RG];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = fmaf(qc, S[n][j], o[j]);
            }
#pragma unroll
            for (int m = CL; m < 64; m <<= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += shfl_xor(o[j], m);
            __syncthreads();
            if (lane < CL) *reinterpret_cast<f32x4*>(&part[wave][4 * lane]) = o;
            __syncthreads();
            if (tid < CL) {
                f32x4 s;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[j] = w.scale * ((part[0][4 * tid + j] + part[1][4 * tid + j]) + (part[2][4 * tid + j] + part[3][4 * tid + j]));
                store4(out + ((int64_t)row * w.H + hk * G + h) * D + eb * EB + 4 * tid, s);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < R; ++n) *reinterpret_cast<f32x4*>(st + (int64_t)(rg + n * RG) * D) = S[n];
}

// ---------------------------------------------------------------- launches
template <typename E, int D>
hipError_t launch_local(const Local& w, hipStream_t stream) {
    constexpr int EB = gated_value_block(D);
    const int64_t n = (int64_t)w.B * w.HK * w.nseg * w.roles * (D / EB);
    gated_local<E, D, EB><<<dim3((unsigned)n), THREADS, 0, stream>>>(w);
    return hipGetLastError();
}

hipError_t launch_join(float* fst, const float* s0, float* rst, const float* ds1, const float* dec, int pairs, int nseg,
                       int DD, hipStream_t stream) {
    const int n = DD * (rst ? 2 : 1) / 64, waves = nseg <= 8 ? 1 : nseg < 8 * JOIN_WAVES ? (nseg + 7) / 8 : JOIN_WAVES;
    // grid.y is at most 65535: pairs are taken in runs
    for (int p = 0; p < pairs; p += 65535) {
        const int64_t o = p;
        const int m = pairs - p < 65535 ? pairs - p : 65535;
        gated_join<<<dim3(n, m), 64 * waves, 0, stream>>>(
            fst + o * (nseg + 1) * DD, s0 ? s0 + o * DD : nullptr, rst ? rst + o * nseg * DD : nullptr,
            ds1 ? ds1 + o * DD : nullptr, dec + o * nseg, nseg, DD);
    }
    return hipGetLastError();
}

template <typename E, int D>
hipError_t forward(const GatedForward& f) {
    const GatedProblem& p = f.p;
    hipError_t err = hipSuccess;
    if (p.nseg > 1) {
        // the walks need the state before each segment: nobody that of the last one alone
        const int before = p.nseg - 1;
        Local l = {};
        l.roles = 1;
        l.y[0] = {p.k, p.ks};
        l.z[0] = {p.v, p.vs};
        l.ny[0] = 1;
        l.st[0] = f.fst;
        l.pair[0] = (int64_t)p.nseg * D * D;
        l.first[0] = D * D;
        l.key_scale[0] = 1.f;
        l.dec = f.fdec;
        l.g = p.g;
        l.lens = p.lens;
        l.B = p.B; l.T = p.T; l.HK = p.HK; l.nseg = before; l.seg_chunks = p.seg_chunks;
        if ((err = launch_local<E, D>(l, p.stream)) != hipSuccess) return err;
        if ((err = launch_join(f.fst, p.s0, nullptr, nullptr, f.fdec, p.B * p.HK, before, D * D, p.stream)) != hipSuccess)
            return err;
    }
    Walk w = {};
    w.x = {p.q, p.qs};
    w.y = {p.k, p.ks};
    w.z = {p.v, p.vs};
    w.out = f.out;
    w.g = p.g;
    w.lens = p.lens;
    w.start = p.nseg > 1 ? f.fst : p.s0;
    w.start_pair = (int64_t)p.nseg * D * D;
    w.start_seg = D * D;
    w.end = f.s1;
    w.sc = D; w.se = 1;
    w.B = p.B; w.T = p.T; w.HK = p.HK; w.nx = p.H / p.HK; w.ny = 1; w.nseg = p.nseg; w.seg_chunks = p.seg_chunks;
    w.pair_scale = w.row_scale = p.scale;
    w.key_scale = 1.f;
    constexpr int EB = gated_value_block(D);
    gated_walk<E, D, EB><<<dim3((unsigned)((int64_t)p.B * p.HK * p.nseg * (D / EB))), (walk_threads<E, D>()), 0, p.stream>>>(w);
    return hipGetLastError();
}

template <typename E, int D>
hipError_t backward(const GatedBackward& f) {
    const GatedProblem& p = f.p;
    const int G = p.H / p.HK, DD = D * D;
    const int64_t hs = (int64_t)p.H * D;
    hipError_t err;
    if (p.nseg > 1) {
        Local l = {};
        l.roles = 2;
        l.y[0] = {p.k, p.ks};
        l.z[0] = {p.v, p.vs};
        l.y[1] = {p.q, p.qs};
        l.z[1] = {f.dout, hs};
        l.ny[0] = 1;
        l.ny[1] = G;
        l.st[0] = f.fst;
        l.st[1] = f.rst;
        l.pair[0] = (int64_t)(p.nseg + 1) * DD;
        l.pair[1] = (int64_t)p.nseg * DD;
        l.first[0] = DD;
        l.key_scale[0] = 1.f;
        l.key_scale[1] = p.scale;
        l.dec = f.fdec;
        l.g = p.g;
        l.lens = p.lens;
        l.B = p.B; l.T = p.T; l.HK = p.HK; l.nseg = p.nseg; l.seg_chunks = p.seg_chunks;
        if ((err = launch_local<E, D>(l, p.stream)) != hipSuccess) return err;
        if ((err = launch_join(f.fst, p.s0, f.rst, f.ds1, f.fdec, p.B * p.HK, p.nseg, DD, p.stream)) != hipSuccess) return err;
    }

    Grads gr = {};
    Walk& w = gr.q;       // dq and q . dq
    w.g = p.g;
    w.lens = p.lens;
    w.B = p.B; w.T = p.T; w.HK = p.HK; w.nseg = p.nseg; w.seg_chunks = p.seg_chunks;
    w.start_seg = DD;
    w.x = {f.dout, hs};
    w.y = {p.v, p.vs};
    w.z = {p.k, p.ks};
    w.x2 = {p.q, p.qs};
    w.out = f.dq;
    w.r = f.rq;
    w.start = p.nseg > 1 ? f.fst : p.s0;
    w.start_pair = p.nseg > 1 ? (int64_t)(p.nseg + 1) * DD : DD;
    // one segment: the state after it, for its product with its gradient
    w.end = p.nseg > 1 || !f.ds1 ? nullptr : f.fst;
    w.sc = 1; w.se = D;
    w.nx = G; w.ny = 1;
    w.pair_scale = w.row_scale = p.scale;
    w.key_scale = 1.f;
    if constexpr (D <= 64) {
        Back& k = gr.kv;
        k.q = {p.q, p.qs};
        k.k = {p.k, p.ks};
        k.v = {p.v, p.vs};
        k.dout = {f.dout, hs};
        k.dk = f.dk;
        k.dv = f.dv;
        k.r = f.rk;
        k.g = p.g;
        k.lens = p.lens;
        k.start = p.nseg > 1 ? f.rst : f.ds1;
        k.end = f.ds0;
        k.B = p.B; k.T = p.T; k.HK = p.HK; k.G = G; k.nseg = p.nseg; k.seg_chunks = p.seg_chunks;
        k.scale = p.scale;
    } else {
        Walk& v = gr.v;   // dv, and the initial state's gradient
        v = w;
        v.x = {p.k, p.ks};
        v.y = {p.q, p.qs};
        v.z = {f.dout, hs};
        v.x2 = {nullptr, 0};
        v.out = f.dv;
        v.r = nullptr;
        v.start = p.nseg > 1 ? f.rst : f.ds1;
        v.start_pair = (int64_t)p.nseg * DD;
        v.end = f.ds0;
        v.sc = D; v.se = 1;
        v.nx = 1; v.ny = G;
        v.row_scale = 1.f;
        v.key_scale = p.scale;
        Walk& k = gr.k;   // dk and k . dk
        k = v;
        k.x = {p.v, p.vs};
        k.y = {f.dout, hs};
        k.z = {p.q, p.qs};
        k.x2 = {p.k, p.ks};
        k.out = f.dk;
        k.r = f.rk;
        k.end = nullptr;
        k.sc = 1; k.se = D;
    }
    constexpr int EB = gated_value_block(D);
    gated_grads<E, D, EB><<<dim3((unsigned)((int64_t)p.B * p.HK * p.nseg * (D / EB) * (D <= 64 ? 2 : 3))),
                            (walk_threads<E, D>()), 0,
                            p.stream>>>(gr);
    if ((err = hipGetLastError()) != hipSuccess) return err;

    GateGrad d;
    d.rq = f.rq; d.rk = f.rk; d.g = p.g;
    // one segment: <S, dS> of the final state, or none
    d.fst = p.nseg > 1 ? f.fst + DD : f.fst;
    d.fst_pair = p.nseg > 1 ? (int64_t)(p.nseg + 1) * DD : DD;
    d.rst = p.nseg > 1 ? f.rst : f.ds1;
    d.lens = p.lens; d.dg = f.dg;
    d.B = p.B; d.T = p.T; d.HK = p.HK; d.nx = G; d.nb = gated_value_blocks(D); d.nseg = p.nseg;
    d.seg_chunks = p.seg_chunks;
    gated_gate_grad<D><<<dim3((unsigned)((int64_t)p.B * p.HK * p.nseg)), THREADS, 0, p.stream>>>(d);
    return hipGetLastError();
}

template <typename E, int D>
hipError_t step(const GatedStep& s) {
    constexpr int EB = gated_value_block(D);
    gated_step<E, D, EB><<<dim3((unsigned)((int64_t)s.B * s.HK * (D / EB))), THREADS, 0, s.stream>>>(s);
    return hipGetLastError();
}

}  // namespace

hipError_t run_gated_forward(const GatedForward& f) {
    if (f.p.bf16)
        return f.p.D == 32 ? forward<uint16_t, 32>(f) : f.p.D == 64 ? forward<uint16_t, 64>(f) : forward<uint16_t, 128>(f);
    return f.p.D == 32 ? forward<float, 32>(f) : f.p.D == 64 ? forward<float, 64>(f) : forward<float, 128>(f);
}

hipError_t run_gated_backward(const GatedBackward& f) {
    if (f.p.bf16)
        return f.p.D == 32 ? backward<uint16_t, 32>(f) : f.p.D == 64 ? backward<uint16_t, 64>(f) : backward<uint16_t, 128>(f);
    return f.p.D == 32 ? backward<float, 32>(f) : f.p.D == 64 ? backward<float, 64>(f) : backward<float, 128>(f);
}

hipError_t run_gated_step(const GatedStep& s) {
    if (s.bf16) return s.D == 32 ? step<uint16_t, 32>(s) : s.D == 64 ? step<uint16_t, 64>(s) : step<uint16_t, 128>(s);
    return s.D == 32 ? step<float, 32>(s) : s.D == 64 ? step<float, 64>(s) : step<float, 128>(s);
}

}  // namespace mhla
