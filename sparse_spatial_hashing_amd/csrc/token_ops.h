// Device pieces shared by the token operators: element types and packed
// documents.
#ifndef SSH_TOKEN_OPS_H
#define SSH_TOKEN_OPS_H

#include <hip/hip_runtime.h>

#include "tokens.h"
#include "wave_ops.h"

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

inline int tok_elem_bytes(int dtype) { return dtype == TOK_F32 ? 4 : 2; }
inline bool tok_dtype_ok(int dtype) {
    return dtype == TOK_F32 || dtype == TOK_BF16 || dtype == TOK_F16;
}

// Blocks of one launch: of 2^32 threads or more along a dimension HIP leaves some
// out, without an error.
constexpr long long most_blocks(int threads) { return 0xffffffffll / threads; }

// NULL will do where nothing is needed.
inline bool workspace_ok(const void* p, long long bytes, long long need) {
    return need == 0 || (p && ((size_t)p & 255) == 0 && bytes >= need);
}

// N elements moved at once.
template <typename T, int N>
struct Pack {
    typedef T vec __attribute__((ext_vector_type(N)));
    static __device__ __forceinline__ vec raw(const T* p) { return *(const vec*)p; }
    static __device__ __forceinline__ void wide(vec v, float (&x)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = (float)v[j];
    }
    static __device__ __forceinline__ void load(const T* p, float (&x)[N]) {
        const vec v = *(const vec*)p;
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = (float)v[j];
    }
    static __device__ __forceinline__ void store(T* p, const float (&x)[N]) {
        vec v;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (T)x[j];
        *(vec*)p = v;
    }
};
template <typename T>
struct Pack<T, 1> {
    typedef T vec;
    static __device__ __forceinline__ vec raw(const T* p) { return *p; }
    static __device__ __forceinline__ void wide(vec v, float (&x)[1]) { x[0] = (float)v; }
    static __device__ __forceinline__ void load(const T* p, float (&x)[1]) { x[0] = (float)*p; }
    static __device__ __forceinline__ void store(T* p, const float (&x)[1]) { *p = (T)x[0]; }
};

// Boundary b of the tokens' ranges: 0, offsets[0 .. docs], total. Range 0 and
// range docs + 1 hold the tokens of no document, range b the document b - 1.
__device__ __forceinline__ int tok_boundary(const int* offsets, int docs, int total, int b) {
    if (b <= 0) return 0;
    if (b > docs + 1) return total;
    if (!offsets) return b == 1 ? 0 : total;
    return min(max(offsets[b - 1], 0), total);
}

// The range of a token in [0, total): the last one that starts at or before
// it. 64 boundaries are tried at once; every lane of the wavefront calls.
__device__ __forceinline__ int tok_range(const int* offsets, int docs, int total, int token) {
    int lo = 0, n = docs + 2;
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave;
        const int at = (int)__lane_id() * step;
        const bool hit = at < n && tok_boundary(offsets, docs, total, lo + at) <= token;
        const int last = max(1, (int)__popcll(__ballot(hit))) - 1;
        lo += last * step;
        n = min(step, n - last * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

#endif  // SSH_TOKEN_OPS_H
