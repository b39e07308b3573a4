// Device pieces of the kernels that multiply tiles: 32x32x16 matrix
// instructions, and tiles brought from HBM straight into LDS.
//
// Operand A of a lane: row lane % 32, elements 8 h .. 8 h + 7 of the inner index
// with h = lane / 32; operand B the same of a column; the result has column
// lane % 32 and, in register r, row 8 (r / 4) + 4 h + r % 4.
#ifndef SSH_MMA_OPS_H
#define SSH_MMA_OPS_H

#include <hip/hip_runtime.h>

#include "token_ops.h"

typedef float acc16 __attribute__((ext_vector_type(16)));

template <typename T>
struct Mma {
    typedef T vec8 __attribute__((ext_vector_type(8)));
    typedef T vec2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ acc16 mul(vec8 a, vec8 b, acc16 c);
    // Two floats rounded to the type, in one register.
    static __device__ __forceinline__ unsigned pair(float x, float y) {
        const vec2 v = {(T)x, (T)y};
        return __builtin_bit_cast(unsigned, v);
    }
};
template <>
__device__ __forceinline__ acc16 Mma<bf16_t>::mul(vec8 a, vec8 b, acc16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ acc16 Mma<f16_t>::mul(vec8 a, vec8 b, acc16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ acc16 zero16() {
    acc16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.0f;
    return z;
}

// Row of a result's register r in a lane of half h.
__device__ __forceinline__ constexpr int acc_row(int r, int half) { return 8 * (r / 4) + 4 * half + r % 4; }

template <typename P>
__device__ __forceinline__ unsigned lds_address(const P* p) {
    return (unsigned)(size_t)(__attribute__((address_space(3))) const char*)p;
}

// 16 bytes of LDS as an operand.
template <typename V>
__device__ __forceinline__ V lds_read(unsigned at) {
    static_assert(sizeof(V) == 16, "an operand of 8");
    typedef const __attribute__((address_space(3))) V* P;
    return *(P)(size_t)at;
}

// Two transposing reads of 8 bytes: every group of 16 lanes takes four rows of 16
// elements, and a lane receives its column's four.
template <typename V>
__device__ __forceinline__ V lds_read_columns(unsigned first, unsigned second) {
    typedef short short4v __attribute__((ext_vector_type(4)));
    typedef short short8v __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) short4v* P;
    const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(size_t)first);
    const short4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(size_t)second);
    const short8v z = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(V, z);
}

// 16 bytes per lane from memory to LDS, a wavefront's 64 pieces one after another
// from `to` on. Written out: the compiler would wait for the load before the next
// read of any LDS. load_wait() and a barrier come before a read. m0 is a reserved register: the
// compiler keeps nothing there from one instruction that needs it to another, and warns of a clobber
// that names it; in these kernels nothing else uses it.
__device__ __forceinline__ void load_to_lds(unsigned to, const void* base, unsigned offset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_to_lds(unsigned to, const void* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(to), "v"(from) : "memory");
}
// At most LEFT of this wavefront's loads are still under way.
template <int LEFT>
__device__ __forceinline__ void load_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LEFT) : "memory");
}

// What is read in place of rows and elements that do not exist.
__device__ const uint4 kNothing = {0, 0, 0, 0};

// Nothing moves across.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// The two halves of the wavefront trade: lanes 0 .. 31 end with x of both halves,
// their own and then the other's, lanes 32 .. 63 with y of both, the lower half's
// first.
__device__ __forceinline__ void trade_halves(unsigned& x, unsigned& y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0], y = r[1];
}

// A block of 32 x 32 results, rounded and traded in halves, is two pieces of 16 bytes per lane:
// lane % 32's, pieces half and 2 + half of its four. Traded here between groups of 16
// lanes: x is that of lane % 16, y of 16 + lane % 16, both piece quarter_piece(lane), so
// that a store writes 64 bytes in a row.
__device__ __forceinline__ void trade_quarters(uint4& x, uint4& y) {
    auto swap = [](unsigned& a, unsigned& b) {
        const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = r[0], b = r[1];
    };
    swap(x.x, y.x);
    swap(x.y, y.y);
    swap(x.z, y.z);
    swap(x.w, y.w);
}
__device__ __forceinline__ int quarter_piece(int lane) { return ((lane >> 4) & 1) * 2 + (lane >> 5); }

// Consecutive logical blocks run on one XCD.
__device__ __forceinline__ unsigned xcd_block(unsigned bid, unsigned n) {
    return (unsigned)xcd_tile(bid, n);
}

#endif  // SSH_MMA_OPS_H
