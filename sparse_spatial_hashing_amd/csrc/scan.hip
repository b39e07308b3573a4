// Gated linear recurrence over packed documents (tokens.h), forward and
// backward.

#include <hip/hip_runtime.h>

#include "token_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr int kRun = TOK_SCAN_RUN;
constexpr long long kMaxTokens = 0x7fffffffll;
constexpr long long kMaxWidth = 65536;
constexpr int kMaxDocs = 1 << 20;

struct ScanArgs {
    const void* gate;
    const void* x;
    const void* gy;           // backward
    const int* offsets;
    const float* state;       // may be null
    void* y;
    float* last;              // forward: last_state (may be null)
    float* carry;             // state before each run (forward: may be null)
    const float* grad_last;   // may be null
    void* ggate;
    void* gx;
    float* grad_state;        // may be null
    int t, width, docs, reverse;
};

// a = sigmoid(f) and 1 - a, each to a few units in its last place: the smaller
// one is a quotient, the larger its difference from one.
__device__ __forceinline__ void gates(float f, float& a, float& keep) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(f) * 1.4426950408889634f);
    const float lo = e * __builtin_amdgcn_rcpf(1.0f + e);
    const float hi = 1.0f - lo;
    a = f >= 0.0f ? hi : lo;   // NaN: lo, NaN itself
    keep = f >= 0.0f ? lo : hi;
}

// One thread per document and channel, along the document. Step s of the scan
// over all tokens is token s, or t - 1 - s in reverse.
template <typename T>
__global__ __launch_bounds__(256) void k_scan_doc(ScanArgs a) {
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const int range = blockIdx.x;
    if (c >= a.width) return;
    const int lo = tok_boundary(a.offsets, a.docs, a.t, range);
    const int hi = max(lo, tok_boundary(a.offsets, a.docs, a.t, range + 1));
    const bool doc = range >= 1 && range <= a.docs;
    float h = doc && a.state ? a.state[(long long)(range - 1) * a.width + c] : 0.0f;
    for (int k = 0; k < hi - lo; ++k) {
        const int token = a.reverse ? hi - 1 - k : lo + k;
        const long long at = (long long)token * a.width + c;
        if (a.carry) {
            const int s = a.reverse ? a.t - 1 - token : token;
            if (s % kRun == 0) a.carry[(long long)(s / kRun) * a.width + c] = h;
        }
        if (doc) {
            float g, keep;
            gates((float)((const T*)a.gate)[at], g, keep);
            h = __builtin_fmaf(g, h, keep * (float)((const T*)a.x)[at]);
        }
        ((T*)a.y)[at] = (T)h;
    }
    if (doc && a.last) a.last[(long long)(range - 1) * a.width + c] = h;
}

// The same backward, run by run from the document's end: the states inside a
// run are computed again from the state before it.
template <typename T>
__global__ __launch_bounds__(256) void k_scan_doc_grad(ScanArgs a) {
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const int range = blockIdx.x;
    if (c >= a.width) return;
    const int lo = tok_boundary(a.offsets, a.docs, a.t, range);
    const int hi = max(lo, tok_boundary(a.offsets, a.docs, a.t, range + 1));
    const bool doc = range >= 1 && range <= a.docs;
    if (!doc) {
        for (int token = lo; token < hi; ++token) {
            const long long at = (long long)token * a.width + c;
            ((T*)a.ggate)[at] = (T)0.0f;
            ((T*)a.gx)[at] = (T)0.0f;
        }
        return;
    }
    const long long own = (long long)(range - 1) * a.width + c;
    const float h0 = a.state ? a.state[own] : 0.0f;
    float back = a.grad_last ? a.grad_last[own] : 0.0f;
    const int s0 = a.reverse ? a.t - hi : lo;      // the document's steps
    const int s1 = a.reverse ? a.t - lo : hi;
    for (int end = s1; end > s0;) {
        const int run = (end - 1) / kRun;
        const int begin = max(run * kRun, s0);
        float h = begin == s0 ? h0 : a.carry[(long long)run * a.width + c];
        float before[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            before[k] = h;
            const int s = begin + k;
            if (s < end) {
                const int token = a.reverse ? a.t - 1 - s : s;
                const long long at = (long long)token * a.width + c;
                float g, keep;
                gates((float)((const T*)a.gate)[at], g, keep);
                h = __builtin_fmaf(g, h, keep * (float)((const T*)a.x)[at]);
            }
        }
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            const int s = begin + k;
            if (s < end) {
                const int token = a.reverse ? a.t - 1 - s : s;
                const long long at = (long long)token * a.width + c;
                float g, keep;
                gates((float)((const T*)a.gate)[at], g, keep);
                const float d = back + (float)((const T*)a.gy)[at];
                ((T*)a.ggate)[at] = (T)(d * (before[k] - (float)((const T*)a.x)[at]) * (g * keep));
                ((T*)a.gx)[at] = (T)(d * keep);
                back = d * g;
            }
        }
        end = begin;
    }
    if (a.grad_state) a.grad_state[own] = back;
}

bool check(int dtype, long long t, long long width, const int32_t* offsets, int32_t docs,
           int32_t reverse) {
    return tok_dtype_ok(dtype) && t >= 0 && t <= kMaxTokens && width >= 1 && width <= kMaxWidth &&
           docs >= 1 && docs <= kMaxDocs && (offsets || docs == 1) &&
           (reverse == 0 || reverse == 1);
}

template <typename T>
int run(const ScanArgs& a, bool grad, hipStream_t stream) {
    const dim3 block(a.width >= 256 ? 256 : (a.width + 63) / 64 * 64);
    const dim3 grid((unsigned)(a.docs + 2), (unsigned)((a.width + block.x - 1) / block.x));
    if (grad)
        k_scan_doc_grad<T><<<grid, block, 0, stream>>>(a);
    else
        k_scan_doc<T><<<grid, block, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

int dispatch(int dtype, const ScanArgs& a, bool grad, hipStream_t stream) {
    if (dtype == TOK_F32) return run<float>(a, grad, stream);
    if (dtype == TOK_BF16) return run<bf16_t>(a, grad, stream);
    return run<f16_t>(a, grad, stream);
}

}  // namespace

extern "C" {

int64_t tok_scan_runs(int64_t t) {
    return t < 0 || t > kMaxTokens ? VOX_EINVAL : (t + kRun - 1) / kRun;
}

int64_t tok_scan_workspace_bytes(int64_t t, int64_t width) {
    if (t < 0 || t > kMaxTokens || width < 1 || width > kMaxWidth) return VOX_EINVAL;
    return 256;
}

int tok_scan(const void* gate, const void* x, int32_t dtype, int64_t t, int64_t width,
             const int32_t* offsets, int32_t docs, int32_t reverse, const float* state, void* y,
             float* last_state, float* carry, void* workspace, int64_t workspace_bytes,
             hipStream_t stream) {
    if (!check(dtype, t, width, offsets, docs, reverse)) return VOX_EINVAL;
    if (t && (!gate || !x || !y)) return VOX_EINVAL;
    if (!workspace || ((size_t)workspace & 255) ||
        workspace_bytes < tok_scan_workspace_bytes(t, width))
        return VOX_EWORKSPACE;
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.offsets = offsets, a.state = state, a.y = y, a.last = last_state;
    a.carry = carry;
    a.t = (int)t, a.width = (int)width, a.docs = docs, a.reverse = reverse;
    return dispatch(dtype, a, false, stream);
}

int tok_scan_grad(const void* grad_y, const void* gate, const void* x, const float* carry,
                  int32_t dtype, int64_t t, int64_t width, const int32_t* offsets, int32_t docs,
                  int32_t reverse, const float* state, const float* grad_last, void* grad_gate,
                  void* grad_x, float* grad_state, void* workspace, int64_t workspace_bytes,
                  hipStream_t stream) {
    if (!check(dtype, t, width, offsets, docs, reverse)) return VOX_EINVAL;
    if (t && (!grad_y || !gate || !x || !carry || !grad_gate || !grad_x)) return VOX_EINVAL;
    if (!workspace || ((size_t)workspace & 255) ||
        workspace_bytes < tok_scan_workspace_bytes(t, width))
        return VOX_EWORKSPACE;
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.gy = grad_y, a.offsets = offsets, a.state = state;
    a.carry = const_cast<float*>(carry);
    a.grad_last = grad_last, a.ggate = grad_gate, a.gx = grad_x, a.grad_state = grad_state;
    a.t = (int)t, a.width = (int)width, a.docs = docs, a.reverse = reverse;
    return dispatch(dtype, a, true, stream);
}

}  // extern "C"
