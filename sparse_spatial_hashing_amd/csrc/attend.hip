// Host side of the attention operator (tokens.h): argument checks, workspace
// layout, and how a call is cut into blocks. The kernels and their layouts
// are in attend_kernels.hip.

#include <hip/hip_runtime.h>

#include <math.h>

#include "attend.h"
#include "token_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

// Rows and keys are counted in 32 bits, and so is the end of a tile of up to
// 128 that starts under the last.
constexpr long long kMaxElems = (1ll << 31) - 2048;
constexpr int kMaxDocs = 1 << 20;
// Documents times key heads: every document may start a tile, and 2^26 more may
// be full, which leaves the blocks of a pass under 2^31.
constexpr long long kMaxStarts = 1ll << 30;
constexpr long long kMaxStride = 1ll << 25;

// 16-byte pieces; a tile of 64 tokens spans less than 2^32 bytes.
bool stride_ok(const int64_t s[2]) {
    return s[0] % 8 == 0 && s[1] % 8 == 0 && s[0] >= 0 && s[1] >= 0 && s[0] < kMaxStride;
}

bool check(const tok_attention* t) {
    if (!t || (t->dtype != TOK_BF16 && t->dtype != TOK_F16)) return false;
    if (t->heads < 1 || t->kv_heads < 1 || t->heads % t->kv_heads || t->heads > 65536) return false;
    if (t->width < 8 || t->width > 128 || t->width % 8) return false;
    if (t->tq < 0 || t->tk < 0 || t->tq > kMaxElems || t->tk > kMaxElems ||
        t->tq * t->heads > kMaxElems || t->tk * t->kv_heads > kMaxElems)
        return false;
    if ((t->docs + 2ll) * t->kv_heads > kMaxStarts) return false;
    if (t->docs < 1 || t->docs > kMaxDocs || (t->mask != 0 && t->mask != 1)) return false;
    if ((!t->q_offsets || !t->k_offsets) && t->docs != 1) return false;
    if (t->prefix && !t->mask) return false;
    // a scale that is used as a divisor too
    if (!(t->scale >= 1e-30f) || !(t->scale <= 1e30f)) return false;
    // a cap whose product with log2(e) is finite
    if (t->cap != 0.0f && (!(t->cap >= 0x1p-126f) || !(t->cap <= 0x1p127f))) return false;
    if (t->axes < 0 || t->axes > 3 || t->reserved) return false;
    if (t->axes && (!t->slopes || (t->tq && !t->q_pos) || (t->tk && !t->k_pos))) return false;
    const int64_t* strides[3] = {t->q_stride, t->k_stride, t->v_stride};
    for (const int64_t* s : strides)
        if (!stride_ok(s)) return false;
    return true;
}

bool aligned16(const void* p) { return ((size_t)p & 15) == 0; }

struct Cut {
    int waves;       // wavefronts of a block
    int q_tiles, k_tiles;
    int nsplit;      // key ranges (forward)
    int row_splits;  // query ranges (grad_k and grad_v)
};

// Wavefronts per block: four share the key tiles when a document has rows for
// more than two of them on average, else one wavefront per block (windows of a
// few dozen tokens, single queries), so that short documents do not leave
// wavefronts without rows. 500 windows of up to 36 tokens train in 54 us with
// one and 144 with four; four frames of 4,096 in 1,343 us with four and 3,056
// with one.
// Key splits: as many as fill the card (two blocks of four wavefronts, or four
// of one, on each of 256 CUs) while a split keeps at least 512 keys; twice as
// many of half the keys changed nothing for one token of 16 scenes (71 us).
Cut cut(const tok_attention& t) {
    Cut c;
    const long long group = t.heads / t.kv_heads;
    const long long rows = t.tq * group;
    c.waves = rows > 64ll * t.docs ? 4 : 1;
    const int per = kAttRows * c.waves;
    c.q_tiles = (int)(rows / per + t.docs + 2);
    c.k_tiles = (int)(t.tk / per + t.docs + 2);
    const long long blocks = (rows / per + t.docs) * t.kv_heads;
    const long long want = c.waves == 4 ? 512 : 1024;
    const long long most = t.tk / t.docs / 512;
    long long n = want / (blocks > 0 ? blocks : 1);
    if (n > most) n = most;
    if (n > 64) n = 64;
    c.nsplit = n < 1 ? 1 : (int)n;
    // Query splits: two blocks on each CU while a split keeps 16 tiles of 32
    // queries. Four frames of up to 4,096 pillars, 8 heads on 2: 240 blocks
    // take 841 us, two splits 578 and their join 12.
    const long long key_blocks = (t.tk / per + t.docs) * t.kv_heads;
    long long r = c.waves == 4 ? 512 / (key_blocks > 0 ? key_blocks : 1) : 1;
    if (r > rows / t.docs / 512) r = rows / t.docs / 512;
    if (r > 16) r = 16;
    c.row_splits = r < 1 ? 1 : (int)r;
    return c;
}

long long round256(long long n) { return (n + 255) / 256 * 256; }

AttArgs make_args(const tok_attention& t, const Cut& c) {
    AttArgs a = {};
    a.q_offsets = t.q_offsets;
    a.k_offsets = t.k_offsets;
    a.prefix = t.prefix;
    a.slopes = t.slopes;
    a.q_pos = t.q_pos;
    a.k_pos = t.k_pos;
    a.q_st = t.q_stride[0], a.q_sh = t.q_stride[1];
    a.k_st = t.k_stride[0], a.k_sh = t.k_stride[1];
    a.v_st = t.v_stride[0], a.v_sh = t.v_stride[1];
    a.g_st = t.g_stride[0], a.g_sh = t.g_stride[1];
    a.qp_st = t.q_pos_stride[0], a.qp_sa = t.q_pos_stride[1];
    a.kp_st = t.k_pos_stride[0], a.kp_sa = t.k_pos_stride[1];
    a.tq = (int)t.tq, a.tk = (int)t.tk, a.docs = t.docs;
    a.heads = t.heads, a.kv_heads = t.kv_heads, a.group = t.heads / t.kv_heads;
    a.width = t.width, a.mask = t.mask, a.axes = t.axes;
    a.nsplit = c.nsplit;
    const double log2e = 1.4426950408889634;
    a.scale = t.scale;
    a.scale2 = (float)(t.scale * log2e);
    a.unscale2 = (float)(1.0 / (t.scale * log2e));
    // at most the largest float: a score of 0 stays 0, all others come to +-cap
    a.cap_in = t.cap > 0.0f ? (float)fmin((double)t.scale / t.cap, 3.4e38) : 0.0f;
    a.cap2 = (float)(t.cap * log2e);
    return a;
}

int run(const tok_attention& t, AttPass pass, const AttArgs& a, int waves, hipStream_t stream) {
    const int wide = t.width <= 32 ? 0 : t.width <= 64 ? 1 : 2;
    static const AttLaunch launches[2][3] = {
        {att_launch_bf16_32, att_launch_bf16_64, att_launch_bf16_128},
        {att_launch_f16_32, att_launch_f16_64, att_launch_f16_128}};
    const hipError_t e = launches[t.dtype == TOK_F16][wide](pass, a, waves, stream);
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

}  // namespace

extern "C" {

int64_t tok_attend_workspace_bytes(const tok_attention* t) {
    if (!check(t)) return VOX_EINVAL;
    const Cut c = cut(*t);
    if (c.nsplit == 1) return 0;
    const long long rows = t->tq * t->heads;
    return round256(c.nsplit * rows * t->width * 4) + round256(c.nsplit * rows * 8);
}

int64_t tok_attend_grad_workspace_bytes(const tok_attention* t) {
    if (!check(t)) return VOX_EINVAL;
    const Cut c = cut(*t);
    const long long parts = c.row_splits > 1 ? 2 * c.row_splits * t->tk * t->kv_heads * t->width * 4 : 0;
    return round256(t->tq * t->heads * 4) + round256(parts);
}

int tok_attend(const tok_attention* t, const void* q, const void* k, const void* v, void* out,
               float* lse, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!check(t)) return VOX_EINVAL;
    if (t->tq == 0) return VOX_OK;
    if (!q || !out || (t->tk && (!k || !v))) return VOX_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, tok_attend_workspace_bytes(t))) return VOX_EWORKSPACE;
    const Cut c = cut(*t);
    AttArgs a = make_args(*t, c);
    a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse;
    a.tiles = c.q_tiles;
    a.part_o = (float*)workspace;
    a.part_ml = (float*)((char*)workspace + round256(c.nsplit * t->tq * t->heads * t->width * 4));
    return run(*t, kAttForward, a, c.waves, stream);
}

int tok_attend_grad(const tok_attention* t, const void* q, const void* k, const void* v,
                    const void* out, const float* lse, const void* grad_out, void* grad_q,
                    void* grad_k, void* grad_v, void* workspace, int64_t workspace_bytes,
                    hipStream_t stream) {
    if (!check(t)) return VOX_EINVAL;
    if (!stride_ok(t->g_stride)) return VOX_EINVAL;
    if (t->tq == 0 && t->tk == 0) return VOX_OK;
    if (t->tq && (!q || !out || !lse || !grad_out || !grad_q)) return VOX_EINVAL;
    if (t->tk && (!k || !v || !grad_k || !grad_v)) return VOX_EINVAL;
    const void* all[] = {q, k, v, out, grad_out, grad_q, grad_k, grad_v};
    for (const void* p : all)
        if (!aligned16(p)) return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, tok_attend_grad_workspace_bytes(t))) return VOX_EWORKSPACE;
    const Cut c = cut(*t);
    AttArgs a = make_args(*t, c);
    a.q = q, a.k = k, a.v = v, a.o = out, a.lse = const_cast<float*>(lse), a.g = grad_out;
    a.gq = grad_q, a.gk = grad_k, a.gv = grad_v;
    a.delta = (float*)workspace;
    if (t->tq) {  // also leaves delta for the other pass
        a.tiles = c.q_tiles;
        const int rc = run(*t, kAttGradQ, a, c.waves, stream);
        if (rc != VOX_OK) return rc;
    }
    if (t->tk) {
        a.tiles = c.k_tiles;
        a.nsplit = c.row_splits;
        a.part_o = (float*)((char*)workspace + round256(t->tq * t->heads * 4));
        return run(*t, kAttGradKV, a, c.waves, stream);
    }
    return VOX_OK;
}

}  // extern "C"
