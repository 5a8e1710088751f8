// gated.h -- internal launchers of the gated linear attention kernels and of
// the query/key norm with rotation (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mhla {

// Tokens of a chunk (one wave holds a chunk's gates, a token a lane).
constexpr int GATED_CHUNK = 64;
// Chunks of a segment at most, backwards (the gates' gradients hold a segment's tokens).
constexpr int GATED_MAX_CHUNKS = 16;

// One sequence problem with the caller's device pointers.  Strides are in
// elements between a token and the next; a batch item is T tokens.
struct GatedProblem {
    int B, T, H, HK, D;
    bool bf16;
    float scale;
    const void* q;
    const void* k;
    const void* v;
    int64_t qs, ks, vs;
    const float* g;       // [B, T, HK]
    const int32_t* lens;  // [B] or nullptr
    const float* s0;      // [B, HK, D, D] or nullptr
    int nseg, seg_chunks; // segments of a sequence and their chunks
    hipStream_t stream;
};

// Workspace regions of a split sequence (nseg > 1): for every (b, kv head) states of D x D
// fp32, before each segment (backwards also after the last) and, backwards, their gradients
// after each segment, and the segments' decays.  Backwards with one segment fst holds the
// state after the sequence alone (where the final state's gradient is given).
struct GatedForward {
    GatedProblem p;
    void* out;
    float* s1;     // [B, HK, D, D] or nullptr
    float* fst;    // [B*HK][nseg][D*D] (nseg > 1)
    float* fdec;   // [B*HK][nseg - 1]
};
hipError_t run_gated_forward(const GatedForward& f);

struct GatedBackward {
    GatedProblem p;
    const void* dout;
    const float* ds1;   // [B, HK, D, D] or nullptr
    void* dq;
    void* dk;
    void* dv;
    float* dg;          // [B, T, HK]
    float* ds0;         // [B, HK, D, D] or nullptr
    float* fst;         // [B*HK][nseg + 1][D*D]
    float* rst;         // [B*HK][nseg][D*D]
    float* fdec;        // [B*HK][nseg]
    float* rq;          // [blocks][B, T, H]:  q . dq, without a token's own term
    float* rk;          // [blocks][B, T, HK]: k . dk, likewise
};
hipError_t run_gated_backward(const GatedBackward& f);

// Value columns that one workgroup of the walk holds, and their blocks.
constexpr int gated_value_block(int D) { return D < 64 ? D : 64; }
inline int gated_value_blocks(int D) { return D / gated_value_block(D); }

struct GatedStep {
    int B, H, HK, D;
    bool bf16;
    float scale;
    const void* q;
    const void* k;
    const void* v;
    int64_t qs, ks, vs;
    const float* g;        // [B, HK]
    const int32_t* slots;  // [B] or nullptr
    float* state;          // [nslots, HK, D, D]
    int nslots;
    void* out;             // [B, H, D]
    hipStream_t stream;
};
hipError_t run_gated_step(const GatedStep& s);

struct QkRope {
    int B, T, H, HK, D;
    bool bf16;
    int style, axes, sec[3], rot;   // rot: rotated values of a head, 2 (sec[0] + sec[1] + sec[2])
    float eps;
    const void* q;
    const void* k;
    int64_t qs, ks;
    const float* wq;        // [D] or nullptr (ones)
    const float* wk;
    const int32_t* pos;     // [B, T, axes]
    const float* freq;      // [rot / 2]
    void* qo;               // forward: outputs; backward: dq, dk
    void* ko;
    const void* dqo;        // backward: gradients of the outputs
    const void* dko;
    float* dwq;             // [D] or nullptr
    float* dwk;
    float* part;            // [groups][2][D] fp32 partial sums of dwq, dwk
    int groups;
    hipStream_t stream;
};
// Workgroups of the backward pass (each leaves one partial sum of the weights' gradients).
int qk_rope_groups(int64_t tokens);
hipError_t run_qk_rope(const QkRope& r, bool backward);

}  // namespace mhla
