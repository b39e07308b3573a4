// What the attention kernels and their host side share.
#ifndef SSH_ATTEND_H
#define SSH_ATTEND_H

#include <hip/hip_runtime.h>

#include "tokens.h"

// One call, as the kernels read it.
struct AttArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* g;        // grad_out (backward)
    const void* o;        // out (backward: read)
    void* out;            // out (forward)
    float* lse;           // forward: written (may be null); backward: read
    void* gq;
    void* gk;
    void* gv;
    float* delta;         // [tq, heads]: sum of grad_out * out
    float* part_o;        // split partials, f32: [nsplit, tq * heads, width] (forward), or of
                          // grad_k, then of grad_v, [nsplit, tk * kv_heads, width]
    float* part_ml;       // [nsplit, tq * heads, 2]: running maximum (base 2) and sum
    const int* q_offsets;
    const int* k_offsets;
    const int* prefix;
    const float* slopes;
    const int* q_pos;
    const int* k_pos;
    long long q_st, q_sh, k_st, k_sh, v_st, v_sh, g_st, g_sh;
    long long qp_st, qp_sa, kp_st, kp_sa;
    int tq, tk, docs, heads, kv_heads, group, width, mask, axes;
    int nsplit;           // ranges a document's keys (forward) or queries (dK dV) are split into
    int tiles;            // row tiles (forward, dQ) or key tiles (dK dV) over all documents
    unsigned first_block; // of this launch, among all the pass's blocks
    float scale;          // > 0
    float scale2;         // scale * log2(e)
    float unscale2;       // 1 / scale2
    float cap_in;         // scale / cap
    float cap2;           // cap * log2(e); 0: no cap
};

enum AttPass { kAttForward = 0, kAttGradQ = 1, kAttGradKV = 2 };

// One pass with these elements and padded width; waves: wavefronts of a block
// (1 or 4). Defined once per (type, padded width).
typedef hipError_t (*AttLaunch)(AttPass pass, const AttArgs& a, int waves, hipStream_t stream);
hipError_t att_launch_bf16_32(AttPass, const AttArgs&, int, hipStream_t);
hipError_t att_launch_bf16_64(AttPass, const AttArgs&, int, hipStream_t);
hipError_t att_launch_bf16_128(AttPass, const AttArgs&, int, hipStream_t);
hipError_t att_launch_f16_32(AttPass, const AttArgs&, int, hipStream_t);
hipError_t att_launch_f16_64(AttPass, const AttArgs&, int, hipStream_t);
hipError_t att_launch_f16_128(AttPass, const AttArgs&, int, hipStream_t);

constexpr int kAttRows = 32;  // query rows (or keys) of a wavefront

#endif  // SSH_ATTEND_H
