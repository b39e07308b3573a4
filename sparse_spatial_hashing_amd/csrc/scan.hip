// Gated linear recurrence over packed documents (tokens.h), forward and
// backward.
//
// A step maps a state to a h + b, and so does any run of steps, so a chunk's
// effect is two numbers a channel: k_scan_sum computes them, k_scan_join turns
// them into the state that enters each chunk, k_scan_run walks the chunks from
// there. The backward is the same recurrence from the other end; its states
// inside a run of kRun steps are computed again from the one saved before it.
// Memory bounds all but k_scan_join, whose loads are all under way at once.
// Sixteen frames, 163,000 pillars of 256 bf16 channels: sums 35 us (167 MB at
// 4.8 TB/s), join 10, run 47 (250 MB at 5.3). 122,880 points of 128 fp32
// channels: 21.5, 9, 32 and backward 21.5, 9, 55.

#include <hip/hip_runtime.h>

#include "token_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr int kRun = TOK_SCAN_RUN;
constexpr int kMaxChunk = 1024;
// Steps are counted in 32 bits: the end of a chunk that starts under t, and the
// step after a batch that does, have to stay under 2^31.
constexpr long long kMaxTokens = (1ll << 31) - 2 * kMaxChunk;
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
    float* mul;               // sum_at(): what each chunk does to a state, then (add)
    float* add;               // the state that enters it
    int t, width, docs, reverse;
    int chunk, chunks;        // steps of a chunk (a multiple of kRun)
    int by_doc;               // a block walks a document, not a chunk
};

// a = sigmoid(f) and 1 - a: the smaller one is a quotient, the larger its
// difference from one. The smaller's relative error is that of the exponent's
// rounded argument and a few more roundings, at most (|f| + 8) 2^-24 while it is
// a normal number (the argument's part: 15 of 2^-24 up to |f| = 20, 64 up to 87);
// the larger's is a few roundings.
__device__ __forceinline__ void gates(float f, float& a, float& keep) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(f) * 1.4426950408889634f);
    const float lo = e * __builtin_amdgcn_rcpf(1.0f + e);
    const float hi = 1.0f - lo;
    a = f >= 0.0f ? hi : lo;   // NaN: lo, NaN itself
    keep = f >= 0.0f ? lo : hi;
}

// Steps: step s of the scan over all tokens is token s, or t - 1 - s in
// reverse. `Doc` is the range of steps [begin, end) of the document (or of the
// tokens of no document: doc < 0) that holds a step.
struct Doc {
    int begin, end, doc;
};

// Walks the documents of a chunk: lane i holds boundary base + i, so going to
// the next document reads no memory. Every lane of the wavefront calls at().
struct Walk {
    int range = -1, base = 0, bound = 0;

    __device__ __forceinline__ Doc of(const ScanArgs& a, int next, int r) {
        if (range < 0 || r < base || r + 1 >= base + kWave) {
            base = next > 0 ? r : r + 2 - kWave;
            bound = tok_boundary(a.offsets, a.docs, a.t, base + (int)__lane_id());
        }
        const int lo = __builtin_amdgcn_readlane(bound, r - base);
        const int hi = max(lo, __builtin_amdgcn_readlane(bound, r - base + 1));
        Doc d;
        d.begin = a.reverse ? a.t - hi : lo;
        d.end = a.reverse ? a.t - lo : hi;
        d.doc = r >= 1 && r <= a.docs ? r - 1 : -1;
        return d;
    }
    // The document of a step; next: where the following one lies (+1 or -1).
    __device__ __forceinline__ Doc at(const ScanArgs& a, int step, int next) {
        if (range >= 0) {
            // the neighbours first: empty documents are passed over
            for (int r = range + next; r >= 0 && r <= a.docs + 1 && r >= range - 64 && r <= range + 64;
                 r += next) {
                const Doc d = of(a, next, r);
                if (d.begin <= step && step < d.end) {
                    range = r;
                    return d;
                }
            }
        }
        const int r = tok_range(a.offsets, a.docs, a.t, a.reverse ? a.t - 1 - step : step);
        Doc d = of(a, next, r);
        range = r;
        // only offsets that decrease end here: one step at a time
        if (step < d.begin || step >= d.end) d.begin = step, d.end = step + 1, d.doc = -1;
        return d;
    }
};

template <int V>
__device__ __forceinline__ void state_of(const float* state, const Doc& d, int width, int c,
                                         float (&h)[V]) {
    if (d.doc >= 0 && state) {
        Pack<float, V>::load(state + (long long)d.doc * width + c, h);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = 0.0f;
    }
}

// Elements of V channels of one step.
template <typename T, int V>
struct Steps {
    const T* base;      // step 0, this thread's channels
    long long stride;   // to the next step
    __device__ __forceinline__ Steps(const ScanArgs& a, const void* p, int c)
        : base((const T*)p + (a.reverse ? (long long)(a.t - 1) * a.width : 0) + c),
          stride(a.reverse ? -(long long)a.width : a.width) {}
    __device__ __forceinline__ const T* at(int s) const { return base + s * stride; }
};

// What a chunk of steps does to the state that enters it: h -> mul h + add.
// A document that starts in the chunk forgets what came before: mul = -0, which
// no product of gates gives and which stays under them, so that not even a NaN
// passes.
constexpr float kForget = -0.0f;

// (mul, add) of chunk k, channel c: 8 channels of all chunks together, which
// is what a block of k_scan_join reads.
__device__ __forceinline__ long long sum_at(const ScanArgs& a, int k, int c) {
    return ((long long)(c >> 3) * a.chunks + k) * 8 + (c & 7);
}

__device__ __forceinline__ bool forgets(float mul) { return __float_as_uint(mul) == 0x80000000u; }

__device__ __forceinline__ float enter(float mul, float add, float h) {
    return forgets(mul) ? add : __builtin_fmaf(mul, h, add);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_sum(ScanArgs a) {
    constexpr int kBatch = 8;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int begin = blockIdx.x * a.chunk, end = min(a.t, begin + a.chunk);
    const bool on = c < a.width;
    const Steps<T, V> gate(a, a.gate, on ? c : 0), x(a, a.x, on ? c : 0);
    float mul[V], add[V];
#pragma unroll
    for (int j = 0; j < V; ++j) mul[j] = 1.0f, add[j] = 0.0f;
    Walk walk;
    for (int s = begin; s < end;) {
        const Doc d = walk.at(a, s, a.reverse ? -1 : 1);
        if (s == d.begin) {
            state_of<V>(a.state, d, a.width, on ? c : 0, add);
#pragma unroll
            for (int j = 0; j < V; ++j) mul[j] = kForget;
        }
        const int e = min(d.end, end);
        if (d.doc < 0) {
            s = e;
            continue;
        }
        for (; s < e; s += kBatch) {
            const int m = min(kBatch, e - s);
            float g[kBatch][V], y[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(gate.at(s + min(k, m - 1)), g[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(x.at(s + min(k, m - 1)), y[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool in = k < m;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float f, keep;
                    gates(g[k][j], f, keep);
                    add[j] = in ? __builtin_fmaf(f, add[j], keep * y[k][j]) : add[j];
                    mul[j] = in ? mul[j] * f : mul[j];
                }
            }
        }
        s = e;
    }
    if (on) {
        const long long at = sum_at(a, blockIdx.x, c);
        Pack<float, V>::store(a.mul + at, mul);
        Pack<float, V>::store(a.add + at, add);
    }
}

// The same for the gradient, which runs from the last step to the first:
// back -> mul back + add, with d = back + grad_y and back = a d at each step.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_sum_grad(ScanArgs a) {
    constexpr int kBatch = 8;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int begin = blockIdx.x * a.chunk, end = min(a.t, begin + a.chunk);
    const bool on = c < a.width;
    const Steps<T, V> gate(a, a.gate, on ? c : 0), grad(a, a.gy, on ? c : 0);
    float mul[V], add[V];
#pragma unroll
    for (int j = 0; j < V; ++j) mul[j] = 1.0f, add[j] = 0.0f;
    Walk walk;
    for (int s = end; s > begin;) {
        const Doc d = walk.at(a, s - 1, a.reverse ? 1 : -1);
        if (s == d.end) {
            state_of<V>(a.grad_last, d, a.width, on ? c : 0, add);
#pragma unroll
            for (int j = 0; j < V; ++j) mul[j] = kForget;
        }
        const int b = max(d.begin, begin);
        if (d.doc < 0) {
            s = b;
            continue;
        }
        for (; s > b; s -= kBatch) {
            const int m = min(kBatch, s - b);
            float g[kBatch][V], y[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(gate.at(s - 1 - min(k, m - 1)), g[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(grad.at(s - 1 - min(k, m - 1)), y[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool in = k < m;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float f, keep;
                    gates(g[k][j], f, keep);
                    add[j] = in ? (add[j] + y[k][j]) * f : add[j];
                    mul[j] = in ? mul[j] * f : mul[j];
                }
            }
        }
        s = b;
    }
    if (on) {
        const long long at = sum_at(a, blockIdx.x, c);
        Pack<float, V>::store(a.mul + at, mul);
        Pack<float, V>::store(a.add + at, add);
    }
}

// The state that enters each chunk, over the chunks' (mul, add), in place of
// add: 8 channels of a block, 128 threads along the chunks, each first over its
// own share, then over the shares before it, then over its own again. Up to
// kHeld chunks of a share stay in registers, all loaded at once: with the
// 3000 chunks at most that chunk_of() makes of up to 3 M tokens, none is read twice.
// grad: from the last chunk to the first.
constexpr int kParts = 128, kHeld = 32;

template <bool GRAD>
__global__ __launch_bounds__(1024) void k_scan_join(ScanArgs a) {
    __shared__ float muls[kParts][8], adds[kParts][8];
    __shared__ float group_mul[kParts / 8][8], group_add[kParts / 8][8];
    const int lane = threadIdx.x & 7, part = threadIdx.x >> 3;
    const int c = blockIdx.x * 8 + lane;
    const bool on = c < a.width;
    const int per = (a.chunks + kParts - 1) / kParts;
    const int k0 = min(a.chunks, part * per), k1 = min(a.chunks, k0 + per);
    auto at = [&](int k) {
        return sum_at(a, GRAD ? a.chunks - 1 - k : k, on ? c : 0);
    };
    float u[kHeld], v[kHeld];
    auto load = [&](int k) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            u[j] = 1.0f, v[j] = 0.0f;
            if (k + j < k1) u[j] = a.mul[at(k + j)], v[j] = a.add[at(k + j)];
        }
    };
    float mul = 1.0f, add = 0.0f;
    for (int k = k0; k < k1; k += kHeld) {
        load(k);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            add = enter(u[j], v[j], add);
            mul = forgets(u[j]) ? u[j] : mul * u[j];
        }
    }
    muls[part][lane] = mul;
    adds[part][lane] = add;
    __syncthreads();
    // over the shares before it, in groups of 8 whose last folds the group
    const int group = part & ~7;
    float before_mul = 1.0f, before_add = 0.0f;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        if (group + j < part) {
            const float u1 = muls[group + j][lane];
            before_add = enter(u1, adds[group + j][lane], before_add);
            before_mul = forgets(u1) ? u1 : before_mul * u1;
        }
    }
    if ((part & 7) == 7) {
        group_mul[part >> 3][lane] = forgets(mul) ? mul : before_mul * mul;
        group_add[part >> 3][lane] = enter(mul, add, before_add);
    }
    __syncthreads();
    float h = 0.0f;  // nothing enters the first chunk: it starts a range
#pragma unroll
    for (int g = 0; g < kParts / 8 - 1; ++g)
        if (g < part >> 3) h = enter(group_mul[g][lane], group_add[g][lane], h);
    h = enter(before_mul, before_add, h);
    for (int k = k0; k < k1; k += kHeld) {
        if (k1 - k0 > kHeld) load(k);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            if (on && k + j < k1) a.add[at(k + j)] = h;
            h = enter(u[j], v[j], h);
        }
    }
}

// Documents of no tokens pass their state through.
template <int V>
__device__ __forceinline__ void pass_empty(const ScanArgs& a, const float* from, float* to, int doc,
                                           int c) {
    float h[V];
    const Doc d = {0, 0, doc};
    state_of<V>(from, d, a.width, c, h);
    Pack<float, V>::store(to + (long long)doc * a.width + c, h);
}

// The steps of a block: a chunk, whose documents are found as it is walked, or
// (by_doc) one document, or the tokens of none. Empty documents are dealt with
// here, kEmpty of them in each block past the chunks' own; false: no steps.
constexpr int kEmpty = 64;

template <int V>
__device__ __forceinline__ bool block_steps(const ScanArgs& a, const float* from, float* to, int c,
                                            Doc* d, int* begin, int* end) {
    const int block = blockIdx.x;
    const bool writes = to && c < a.width;
    if (a.by_doc) {
        const int lo = tok_boundary(a.offsets, a.docs, a.t, block);
        const int hi = max(lo, tok_boundary(a.offsets, a.docs, a.t, block + 1));
        d->begin = *begin = a.reverse ? a.t - hi : lo;
        d->end = *end = a.reverse ? a.t - lo : hi;
        d->doc = block >= 1 && block <= a.docs ? block - 1 : -1;
        if (hi == lo && d->doc >= 0 && writes) pass_empty<V>(a, from, to, d->doc, c);
        return hi > lo;
    }
    if (block < a.chunks) {
        *begin = block * a.chunk;
        *end = min(a.t, *begin + a.chunk);
        return true;
    }
    const int first = (block - a.chunks) * kEmpty;
    for (int doc = first; doc < min(a.docs, first + kEmpty) && writes; ++doc) {
        const int lo = tok_boundary(a.offsets, a.docs, a.t, doc + 1);
        if (tok_boundary(a.offsets, a.docs, a.t, doc + 2) <= lo) pass_empty<V>(a, from, to, doc, c);
    }
    return false;
}

// The recurrence over a chunk of steps, from the state that enters it.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_run(ScanArgs a) {
    constexpr int kBatch = 8;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    Doc d = {0, 0, -1};
    int begin, end;
    if (!block_steps<V>(a, a.state, a.last, c, &d, &begin, &end)) return;
    const bool on = c < a.width;
    const Steps<T, V> gate(a, a.gate, on ? c : 0), x(a, a.x, on ? c : 0), y(a, a.y, on ? c : 0);
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = 0.0f;
    if (a.chunks > 1 && !a.by_doc && on) Pack<float, V>::load(a.add + sum_at(a, blockIdx.x, c), h);
    Walk walk;
    for (int s = begin; s < end;) {
        if (s == begin || s == d.end) {
            if (!a.by_doc) d = walk.at(a, s, a.reverse ? -1 : 1);
            if (s == d.begin) state_of<V>(a.state, d, a.width, on ? c : 0, h);
        }
        if (a.carry && s % kRun == 0 && on)
            Pack<float, V>::store(a.carry + (long long)(s / kRun) * a.width + c, h);
        const int e = min(min(d.end, end), (s / kRun + 1) * kRun);
        if (d.doc < 0) {
            float zero[V];
#pragma unroll
            for (int j = 0; j < V; ++j) zero[j] = 0.0f;
            for (; s < e; ++s)
                if (on) Pack<T, V>::store((T*)y.at(s), zero);
            continue;
        }
        for (; s < e; s += kBatch) {
            const int m = min(kBatch, e - s);
            float g[kBatch][V], z[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(gate.at(s + min(k, m - 1)), g[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Pack<T, V>::load(x.at(s + min(k, m - 1)), z[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const bool in = k < m;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float f, keep;
                    gates(g[k][j], f, keep);
                    h[j] = in ? __builtin_fmaf(f, h[j], keep * z[k][j]) : h[j];
                }
                if (on && in) Pack<T, V>::store((T*)y.at(s + k), h);
            }
        }
        s = e;
        if (s == d.end && a.last && on)
            Pack<float, V>::store(a.last + (long long)d.doc * a.width + c, h);
    }
}

// The gradient over a chunk of steps, a run of kRun at a time from its last:
// the states inside a run are computed again from the state before it.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_run_grad(ScanArgs a) {
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    Doc d = {0, 0, -1};
    int begin, end;
    if (!block_steps<V>(a, a.grad_last, a.grad_state, c, &d, &begin, &end)) return;
    const bool on = c < a.width;
    const int cc = on ? c : 0;
    const Steps<T, V> gate(a, a.gate, cc), x(a, a.x, cc), grad(a, a.gy, cc);
    const Steps<T, V> ggate(a, a.ggate, cc), gx(a, a.gx, cc);
    float back[V];
#pragma unroll
    for (int j = 0; j < V; ++j) back[j] = 0.0f;
    if (a.chunks > 1 && !a.by_doc && on) Pack<float, V>::load(a.add + sum_at(a, blockIdx.x, c), back);
    Walk walk;
    for (int s = end; s > begin;) {
        if (s == end || s == d.begin) {
            if (!a.by_doc) d = walk.at(a, s - 1, a.reverse ? 1 : -1);
            if (s == d.end) state_of<V>(a.grad_last, d, a.width, cc, back);
        }
        const int b = max(max(d.begin, begin), (s - 1) / kRun * kRun);
        if (d.doc < 0) {
            float zero[V];
#pragma unroll
            for (int j = 0; j < V; ++j) zero[j] = 0.0f;
            for (; s > b; --s)
                if (on) {
                    Pack<T, V>::store((T*)ggate.at(s - 1), zero);
                    Pack<T, V>::store((T*)gx.at(s - 1), zero);
                }
            continue;
        }
        const int m = s - b;
        typename Pack<T, V>::vec g[kRun], z[kRun], w[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) g[k] = Pack<T, V>::raw(gate.at(b + min(k, m - 1)));
#pragma unroll
        for (int k = 0; k < kRun; ++k) z[k] = Pack<T, V>::raw(x.at(b + min(k, m - 1)));
#pragma unroll
        for (int k = 0; k < kRun; ++k) w[k] = Pack<T, V>::raw(grad.at(b + min(k, m - 1)));
        float h[V], before[kRun][V];
        if (b == d.begin)
            state_of<V>(a.state, d, a.width, cc, h);
        else
            Pack<float, V>::load(a.carry + (long long)(b / kRun) * a.width + cc, h);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            float f[V], y[V];
            Pack<T, V>::wide(g[k], f);
            Pack<T, V>::wide(z[k], y);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                before[k][j] = h[j];
                float fa, keep;
                gates(f[j], fa, keep);
                h[j] = __builtin_fmaf(fa, h[j], keep * y[j]);
            }
        }
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (k >= m) continue;
            float f[V], y[V], q[V], p[V], r[V];
            Pack<T, V>::wide(g[k], f);
            Pack<T, V>::wide(z[k], y);
            Pack<T, V>::wide(w[k], q);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float fa, keep;
                // computed again, not kept for the whole run since the sweep above
                asm("" : "+v"(f[j]));
                gates(f[j], fa, keep);
                const float dh = back[j] + q[j];
                p[j] = dh * (before[k][j] - y[j]) * (fa * keep);
                r[j] = dh * keep;
                back[j] = dh * fa;
            }
            if (on) {
                Pack<T, V>::store((T*)ggate.at(b + k), p);
                Pack<T, V>::store((T*)gx.at(b + k), r);
            }
        }
        s = b;
        if (s == d.begin && a.grad_state && on)
            Pack<float, V>::store(a.grad_state + (long long)d.doc * a.width + c, back);
    }
}

bool check(int dtype, long long t, long long width, const int32_t* offsets, int32_t docs,
           int32_t reverse) {
    return tok_dtype_ok(dtype) && t >= 0 && t <= kMaxTokens && width >= 1 && width <= kMaxWidth &&
           docs >= 1 && docs <= kMaxDocs && (offsets || docs == 1) &&
           (reverse == 0 || reverse == 1);
}

// Steps per chunk: 32, doubled while there are more than 3000 chunks. Short
// chunks fill the card (a wavefront walks a chunk of 64 lanes of channels),
// long ones keep the chunks' sums few: 122,880 points of 128 channels train in
// 167 us with 3840 chunks of 32 and in 162 with 1920 of 64; 163,000 pillars of
// 256 channels take 114 us with 5100 chunks of 32, 103 with 2550 of 64 and 116
// with 1280 of 128.
// Up to 64 steps are one chunk: its walk takes less than two more launches.
int chunk_of(long long t) {
    int chunk = t <= 64 ? 64 : 32;
    while (chunk < kMaxChunk && (t + chunk - 1) / chunk > 3000) chunk *= 2;
    return chunk;
}

template <typename T, int V, bool GRAD>
int run(ScanArgs a, hipStream_t stream) {
    const int lanes = (a.width / V + kWave - 1) / kWave * kWave;
    const dim3 block(lanes < 256 ? lanes : 256);
    const unsigned slabs = (unsigned)((a.width / V + block.x - 1) / block.x);
    // Documents of a few tokens on average (a decoding step): a block each, in
    // one launch. 64 sequences of one token, 512 channels: 3.4 us; walked one
    // after another as a chunk, 89. (At worst one document holds all 4096
    // tokens: 850 us.)
    a.by_doc = a.t <= 4096 && a.t <= 8ll * a.docs;
    if (a.chunks > 1 && !a.by_doc) {
        const dim3 grid((unsigned)a.chunks, slabs), join((unsigned)((a.width + 7) / 8));
        if constexpr (GRAD) {
            k_scan_sum_grad<T, V><<<grid, block, 0, stream>>>(a);
            k_scan_join<true><<<join, dim3(1024), 0, stream>>>(a);
        } else {
            k_scan_sum<T, V><<<grid, block, 0, stream>>>(a);
            k_scan_join<false><<<join, dim3(1024), 0, stream>>>(a);
        }
    }
    const unsigned blocks = a.by_doc ? a.docs + 2 : a.chunks + (a.docs + kEmpty - 1) / kEmpty;
    if constexpr (GRAD)
        k_scan_run_grad<T, V><<<dim3(blocks, slabs), block, 0, stream>>>(a);
    else
        k_scan_run<T, V><<<dim3(blocks, slabs), block, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

// Two channels per thread where every array is aligned for pairs and a
// wavefront's lanes stay in use. (Four of 16 bits: sixteen frames of 256
// channels took 105 us, with two 103: more wavefronts hide more.)
template <typename T>
int dispatch_type(const ScanArgs& a, bool grad, hipStream_t stream) {
    const void* elems[] = {a.gate, a.x, a.gy, a.y, a.ggate, a.gx};
    const void* floats[] = {a.state, a.last, a.carry, a.grad_last, a.grad_state};
    int v = 2;
    auto fits = [&](int n) {
        if (a.width % n || (n > 1 && a.width / n < kWave)) return false;
        for (const void* p : elems)
            if ((size_t)p % (n * sizeof(T))) return false;
        for (const void* p : floats)
            if ((size_t)p % (n * 4)) return false;
        return true;
    };
    while (v > 1 && !fits(v)) v /= 2;
    if (grad) return v == 2 ? run<T, 2, true>(a, stream) : run<T, 1, true>(a, stream);
    return v == 2 ? run<T, 2, false>(a, stream) : run<T, 1, false>(a, stream);
}

int dispatch(int dtype, ScanArgs& a, bool grad, void* workspace, hipStream_t stream) {
    a.chunk = chunk_of(a.t);
    a.chunks = (int)((a.t + (long long)a.chunk - 1) / a.chunk);
    a.mul = (float*)workspace;
    a.add = a.mul + a.chunks * ((a.width + 7ll) / 8 * 8);
    if (dtype == TOK_F32) return dispatch_type<float>(a, grad, stream);
    if (dtype == TOK_BF16) return dispatch_type<bf16_t>(a, grad, stream);
    return dispatch_type<f16_t>(a, grad, stream);
}

}  // namespace

extern "C" {

int64_t tok_scan_runs(int64_t t) {
    return t < 0 || t > kMaxTokens ? VOX_EINVAL : (t + kRun - 1) / kRun;
}

int64_t tok_scan_workspace_bytes(int64_t t, int64_t width) {
    if (t < 0 || t > kMaxTokens || width < 1 || width > kMaxWidth) return VOX_EINVAL;
    const long long chunk = chunk_of(t), chunks = (t + chunk - 1) / chunk;
    return chunks <= 1 ? 0 : (chunks * ((width + 7) / 8 * 64) + 255) / 256 * 256;
}

int tok_scan(const void* gate, const void* x, int32_t dtype, int64_t t, int64_t width,
             const int32_t* offsets, int32_t docs, int32_t reverse, const float* state, void* y,
             float* last_state, float* carry, void* workspace, int64_t workspace_bytes,
             hipStream_t stream) {
    if (!check(dtype, t, width, offsets, docs, reverse)) return VOX_EINVAL;
    if (t && (!gate || !x || !y)) return VOX_EINVAL;
    if (((size_t)gate | (size_t)x | (size_t)y) % tok_elem_bytes(dtype)) return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, tok_scan_workspace_bytes(t, width)))
        return VOX_EWORKSPACE;
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.offsets = offsets, a.state = state, a.y = y, a.last = last_state;
    a.carry = carry;
    a.t = (int)t, a.width = (int)width, a.docs = docs, a.reverse = reverse;
    return dispatch(dtype, a, false, workspace, stream);
}

int tok_scan_grad(const void* grad_y, const void* gate, const void* x, const float* carry,
                  int32_t dtype, int64_t t, int64_t width, const int32_t* offsets, int32_t docs,
                  int32_t reverse, const float* state, const float* grad_last, void* grad_gate,
                  void* grad_x, float* grad_state, void* workspace, int64_t workspace_bytes,
                  hipStream_t stream) {
    if (!check(dtype, t, width, offsets, docs, reverse)) return VOX_EINVAL;
    if (t && (!grad_y || !gate || !x || !carry || !grad_gate || !grad_x)) return VOX_EINVAL;
    if (((size_t)grad_y | (size_t)gate | (size_t)x | (size_t)grad_gate | (size_t)grad_x) %
        tok_elem_bytes(dtype))
        return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, tok_scan_workspace_bytes(t, width)))
        return VOX_EWORKSPACE;
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.gy = grad_y, a.offsets = offsets, a.state = state;
    a.carry = const_cast<float*>(carry);
    a.grad_last = grad_last, a.ggate = grad_gate, a.gx = grad_x, a.grad_state = grad_state;
    a.t = (int)t, a.width = (int)width, a.docs = docs, a.reverse = reverse;
    return dispatch(dtype, a, true, workspace, stream);
}

}  // extern "C"
