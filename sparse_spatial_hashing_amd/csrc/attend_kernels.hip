// Attention kernels for one element type (ATT_F16 0: bf16, 1: fp16) and one
// padded head width (ATT_WIDTH 32, 64 or 128); compiled once for each.
//
// Rows. A document's query rows are its (query, head of the group) pairs of
// one key head, r = i * group + g, so heads that share keys fill a tile
// together. A wavefront owns 32 rows (forward, grad_q) or 32 keys (grad_k and
// grad_v).
//
// Products, on 32x32x16 matrix instructions. Operand A of a lane: row
// lane % 32, elements 8 h .. 8 h + 7 with h = lane / 32; operand B the same
// of a column; the result has column lane % 32 and, in register r, row
// 8 (r / 4) + 4 h + r % 4. The first product is taken transposed,
// S^T = K Q^T, so that a lane holds scores of one query: the softmax's maximum
// and sum run inside the lane and across one pair of lanes. Registers
// 8 c .. 8 c + 7 of S^T are then, rounded, operand B of the second product
// O^T = V^T P^T over the 16 keys of chunk c, its inner index running over the
// keys in the order 4 h + (0..3), 8 + 4 h + (0..3); V^T is read with the same
// order (two transposing LDS reads of four keys each). Nothing is shuffled.
//
// Roundings. What enters the second products (weights forward, weights and
// score gradients backward) is rounded to the tensors' type, as the matrix
// units of 16 bits take it: in 32 bits those products run at a sixteenth of the
// rate, and a second product with what the rounding left would add half of the
// forward's to it. It costs, against 64 bits, 2.0e-3 to 2.4e-3 of the output's
// norm in bf16 where the output's own rounding costs 1.7e-3 (fp16 2.9e-4 and
// 2.1e-4). Scores, maxima, sums and accumulators are in 32 bits.
//
// LDS tiles are rows of 2 * WIDTH bytes with the 16-byte chunks of a row
// permuted by XOR with swz(row), so that both a read of one chunk of 16
// consecutive rows and a transposing read of four consecutive rows times 64
// bytes touch every bank group once.

#include <hip/hip_runtime.h>

#include "attend.h"
#include "token_ops.h"

#ifndef ATT_WIDTH
#error "ATT_WIDTH: 32, 64 or 128"
#endif

namespace {

constexpr int W = ATT_WIDTH;
constexpr int kChunks = W / 8;    // 16-byte chunks of a row
constexpr int kSteps = W / 16;    // inner steps of a product over the width
constexpr int kBlocks = W / 32;   // 32-wide blocks of the width

#if ATT_F16
typedef _Float16 elem;
#else
typedef __bf16 elem;
#endif
typedef elem vec8 __attribute__((ext_vector_type(8)));
typedef elem vec4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float acc16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e+38f;
// The backward's weights are computed 2^kLift too large and the sums put right
// at the end, so that they keep all their bits down to 2^-150 (bf16; exp2 ends
// at 2^-126) and 2^-28 (fp16, which ends at 2^16 and has them from 2^-14 on).
constexpr float kLift = ATT_F16 ? 14.0f : 24.0f;
constexpr float kUnlift = ATT_F16 ? 0x1p-14f : 0x1p-24f;
constexpr float kRescale = 8.0f;  // running maximum may lag by this much (base 2)
// The forward's weights are computed less a number 2^kTop under the running
// maximum: fp16 then holds them from 2^15 on down, with all their bits to 2^-21
// of the largest (2^-14 without, and nothing under 2^-25: a dominant key hid
// what 20,000 others of e^-17.5 its weight add up to).
constexpr float kTop = ATT_F16 ? 7.0f : 0.0f;

__device__ __forceinline__ acc16 mma(vec8 a, vec8 b, acc16 c) {
#if ATT_F16
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
#else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
#endif
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int swz(int row) {
    if (W == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
    if (W == 64) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    return (row >> 2) & 3;
}

// LDS as byte addresses. Tiles start at multiples of 256 bytes, so the chunk's
// XOR works on the sum of a tile's address and a lane's place in it: from one
// sum per lane, an operand's chunk is one XOR and its 16 or 32 rows are in the
// instruction's offset.
template <typename T>
__device__ __forceinline__ unsigned lds_address(const T* p) {
    return (unsigned)(size_t)(__attribute__((address_space(3))) const char*)p;
}

// Operand A of a product over the width, rows lane % 32: where in a tile.
__device__ __forceinline__ unsigned rows_place(int lane) {
    const int row = lane & 31;
    return row * 2 * W + (((lane >> 5) ^ swz(row)) << 4);
}
// at: tile address + rows_place
__device__ __forceinline__ vec8 lds_rows(unsigned at, int row0, int k) {
    typedef const __attribute__((address_space(3))) vec8* P;
    return *(P)(size_t)((at ^ (k << 5)) + row0 * 2 * W);
}

// Operand A of a transposed product: rows are elements 32 b + lane % 32 of
// the width, inner index 16 tile rows in the order above; where in a tile
// the first four of eight rows are, and the others.
__device__ __forceinline__ uint2 columns_place(int lane) {
    const int row = 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), in = (lane & 1) << 3;
    return make_uint2(row * 2 * W + ((c ^ swz(row)) << 4) + in,
                      (row + 8) * 2 * W + ((c ^ swz(row + 8)) << 4) + in);
}
// row0: a multiple of 16, which swz() does not see
__device__ __forceinline__ vec8 lds_columns(uint2 at, int row0, int b) {
    typedef __attribute__((address_space(3))) short4v* P;
    const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(size_t)((at.x ^ (b << 6)) + row0 * 2 * W));
    const short4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(size_t)((at.y ^ (b << 6)) + row0 * 2 * W));
    typedef short short8v __attribute__((ext_vector_type(8)));
    const short8v z = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(vec8, z);
}

__device__ __forceinline__ vec8 round8(const acc16& s, int c) {
    vec8 p;
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (elem)s[8 * c + j];
    return p;
}

__device__ __forceinline__ vec8 zero8() {
    vec8 z;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = (elem)0.0f;
    return z;
}

// The other half's value (lane ^ 32).
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Tile t belongs to the last range whose first tile, floor(start * per / size)
// + range, is <= t: that leaves every range at least ceil(length * per / size)
// tiles without anyone knowing the lengths on the host. 64 ranges are tried
// at once.
template <int SIZE>
__device__ __forceinline__ int find_range(const int* offsets, int docs, int total, int per, int t,
                                          int* first_tile) {
    int lo = 0, n = docs + 2;
    const int lane = __lane_id();
    int first = 0;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int b = lo + lane * step;
        const bool in = lane * step < n;
        const int f = in ? (int)((unsigned long long)tok_boundary(offsets, docs, total, b) * per / SIZE) + b
                         : 0x7fffffff;
        const unsigned long long hit = __ballot(in && f <= t);
        const int cnt = max(1, (int)__popcll(hit));
        first = __shfl(f, cnt - 1);
        lo += (cnt - 1) * step;
        n = min(step, n - (cnt - 1) * step);
    }
    *first_tile = __builtin_amdgcn_readfirstlane(first);
    return __builtin_amdgcn_readfirstlane(lo);
}

// Score gradients have the size of grad_out times a weight, which fp16 cannot
// hold at a loss's usual size and 12,000 keys, nor where grad_out . v is large.
// There each column carries a power of two that its score gradients are
// multiplied with before they are rounded, and its sums until the end: from
// the first that are not zero on, chosen so that the largest comes to
// 2^kAim, and again when one passes 2^kMost. bf16 has the range (by is 1).
// Four frames of up to 4,096 in fp16, 8 heads on 2 of 128: 1,515 us forward and
// backward, without 1,450; a grad_out of 1e-6 then left nothing of grad_q.
struct Lift {
    static constexpr int kAim = 8;
    static constexpr float kMost = 0x1p15f;
    float by = ATT_F16 ? 0x1p100f : 1.0f;

    __device__ __forceinline__ void apply(acc16& ds, acc16 (&sums)[kBlocks]) {
        if (!ATT_F16) return;
        float top = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(ds[r]));
        if (__any(top * by > kMost)) {
            top = fmaxf(top, other_half(top));
            const float was = by;
            if (top * by > kMost) by = ldexpf(1.0f, kAim - __builtin_amdgcn_frexp_expf(top));
            const float w = by / was;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) sums[b][r] *= w;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) ds[r] *= by;
    }
    __device__ __forceinline__ float undo() const { return ATT_F16 ? 1.0f / by : 1.0f; }
};

struct Range {
    int qlo, lq, klo, lk, prefix;
};

__device__ __forceinline__ Range get_range(const AttArgs& a, int b) {
    Range r;
    r.qlo = tok_boundary(a.q_offsets, a.docs, a.tq, b);
    r.lq = max(0, tok_boundary(a.q_offsets, a.docs, a.tq, b + 1) - r.qlo);
    r.klo = tok_boundary(a.k_offsets, a.docs, a.tk, b);
    r.lk = max(0, tok_boundary(a.k_offsets, a.docs, a.tk, b + 1) - r.klo);
    r.prefix = 0;
    if (b == 0 || b == a.docs + 1) {
        r.lk = 0;  // rows of no document see nothing
    } else if (a.mask && a.prefix) {
        r.prefix = a.prefix[b - 1];
    }
    return r;
}

// Keys [0, limit) of the document are visible to its query i.
__device__ __forceinline__ int key_limit(const AttArgs& a, const Range& d, int i) {
    if (!a.mask) return d.lk;
    return clampi(max(d.prefix, min(d.lk, i - d.lq + d.lk + 1)), 0, d.lk);
}

// A token's position as it is in memory, and packed for sad_u16: .x the last
// two axes, .y the first of three. Apart, so that a position fetched ahead is
// first waited for where it is packed.
template <int AX>
__device__ __forceinline__ int3 load_pos(const int* pos, long long st, long long sa, int axes,
                                         long long token) {
    int3 r = make_int3(0, 0, 0);
    if (AX) {
        const int* p = pos + token * st;
        r.x = p[0];
        if (axes >= 2) r.y = p[sa];
        if (AX == 3) r.z = p[2 * sa];
    }
    return r;
}
__device__ __forceinline__ uint2 pack_pos(int3 p) {
    return make_uint2((unsigned)clampi(p.x, 0, 65535) | (unsigned)clampi(p.y, 0, 65535) << 16,
                      (unsigned)clampi(p.z, 0, 65535));
}

// -slope2 |a - b|, the distance summed over the axes. The sums of absolute
// differences (below 2^23) are added to the bits of 1.0, so f = 1 + d 2^-23
// exactly, and with steep = slope2 2^23 one product-sum gives the bias rounded
// once: no conversion.
template <int AX>
__device__ __forceinline__ float bias(uint2 p, unsigned x, unsigned y, float steep) {
    unsigned d = __builtin_amdgcn_sad_u16(p.x, x, 0x3f800000u);
    if (AX == 3) d = __builtin_amdgcn_sad_u16(p.y, y, d);
    return __builtin_fmaf(__uint_as_float(d), -steep, steep);
}

// Scores are wanted less a number of the row. With a bias and no cap it goes
// into the product's first summand; else into scores().
template <int AX, bool CAP>
__device__ __forceinline__ float first_summand(const AttArgs& a, float sub) {
    return AX && !CAP ? -sub * a.unscale2 : 0.0f;
}

// tanh(u), u = score / cap, for a block's scores at once: where all are small,
// u times a polynomial in u^2 (on |u| <= 0.5, found by the exchange method; with
// the coefficients rounded its relative error is 2.9e-8, half a step of a float,
// and 8.4e-8 as computed here) in 6 instructions a score; else
// 1 - 2 / (exp(2 u) + 1), right at both ends (exp = 0 and inf), whose two
// transcendentals alone take the time of 8.
constexpr float kSmallTanh = 0.5f;

__device__ __forceinline__ float tanh_small(float u) {
    const float w = u * u;
    float r = __builtin_fmaf(0.017135007f, w, -0.052986074f);
    r = __builtin_fmaf(r, w, 0.13324779f);
    r = __builtin_fmaf(r, w, -0.33333069f);
    return __builtin_fmaf(u * w, r, u);
}

__device__ __forceinline__ void cap_block(const AttArgs& a, acc16& s) {
    float far = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] *= a.cap_in;
#pragma unroll
    for (int r = 0; r < 16; ++r) far = fmaxf(far, fabsf(s[r]));
    if (!__any(!(far <= kSmallTanh))) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = tanh_small(s[r]);
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            s[r] = __builtin_fmaf(
                -2.0f, __builtin_amdgcn_rcpf(exp2_(s[r] * (2.0f * kLog2e)) + 1.0f), 1.0f);
    }
}

// A lane or thread number again, as a value that places in LDS and memory are
// computed from where they are used: kept over a loop, at a width of 128 they
// push what the products need out of the registers.
__device__ __forceinline__ int fresh(int x) {
    if (W == 128) asm volatile("" : "+v"(x));
    return x;
}

// A tile of ROWS rows of k or v (or q, grad_out), brought from HBM into LDS
// without passing registers: a wavefront's load puts 64 consecutive 16-byte
// chunks of LDS, so the XOR of swz() is on the side of the source. Rows past
// the last are copies of it; chunks past the width keep the zeros of clear().
// load() only starts the loads: landed() and a barrier come before a read.
template <int ROWS, int NT>
struct Tile {
    static constexpr int kPer = (ROWS * kChunks + NT - 1) / NT;
    static_assert(ROWS * kChunks % 64 == 0 && NT % kChunks == 0, "whole wavefronts and rows");

    static __device__ __forceinline__ void clear(uint4* tile, int width) {
        if (width == W) return;
        for (int p = threadIdx.x; p < ROWS * kChunks; p += NT) tile[p] = make_uint4(0, 0, 0, 0);
    }
    // rows: that exist from `base` on (>= 1), stride in elements
    static __device__ __forceinline__ void load(uint4* tile, const elem* base, long long stride,
                                                int rows, int width) {
        const int tid = fresh(threadIdx.x), r0 = tid / kChunks, at = tid % kChunks;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        constexpr int kStep = NT / kChunks;  // rows from one load to the next
        const unsigned to = lds_address(tile) + 1024u * wave;
        if (rows >= ROWS && width == W) {
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                if (p * NT + wave * 64 < ROWS * kChunks)
                    start(to + 16u * NT * p, base + (long long)p * kStep * stride,
                          (unsigned)r0 * (unsigned)(2 * stride) + 16u * (at ^ swz(p * kStep + r0)));
            return;
        }
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int r = p * kStep + r0, c = at ^ swz(r);
            if (p * NT + wave * 64 < ROWS * kChunks && c * 8 < width)
                start(to + 16u * NT * p, base, (unsigned)min(r, rows - 1) * (unsigned)(2 * stride) + 16u * c);
        }
    }
    // 64 chunks to LDS from `to` on. Written out: the compiler would wait for
    // the load before the next read of any LDS. Offsets inside a tile fit 32
    // bits: the host bounds the stride.
    static __device__ __forceinline__ void start(unsigned to, const elem* base, unsigned offset) {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :: "s"(to), "v"(offset), "s"(base) : "memory");
    }
};

// Nothing moves across: reads of LDS written above it are under way before
// what is below, however few registers the compiler would rather use.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// The operands A of the transposed product over 16 rows of a tile.
__device__ __forceinline__ void read_columns(uint2 at, int row0, vec8 (&x)[kBlocks]) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) x[b] = lds_columns(at, row0, b);
}

// s += 32 rows of a tile times an operand in registers. At a width of 128 two
// steps are read ahead, else all at once: the backward has no registers left.
__device__ __forceinline__ void product(acc16& s, unsigned at, int row0, const vec8 (&f)[kSteps]) {
    constexpr int kAhead = W == 128 ? 2 : kSteps;
    vec8 x[2][kAhead];
    auto read = [&](int j) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[j & 1][i] = lds_rows(at, row0, kAhead * j + i);
    };
    read(0);
#pragma unroll
    for (int j = 0; j < kSteps / kAhead; ++j) {
        if (j + 1 < kSteps / kAhead) read(j + 1);
        fence();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s = mma(x[j & 1][i], f[kAhead * j + i], s);
    }
}

// Operands B that a wavefront keeps in LDS instead of registers, each lane its
// own: at a width of 128 the backward's four sets and its sums do not fit the
// 256 registers that let two wavefronts share a SIMD.
// FROM, COUNT: the steps kept.
template <int FROM, int COUNT>
__device__ __forceinline__ void keep(uint4* kept, int lane, const vec8 (&x)[kSteps]) {
#pragma unroll
    for (int k = 0; k < COUNT; ++k) kept[64 * k + lane] = __builtin_bit_cast(uint4, x[FROM + k]);
}
// s += rows of the tile times an operand whose first COUNT steps are kept and
// whose others are in f; a step read ahead.
template <int COUNT>
__device__ __forceinline__ void product_kept(acc16& s, unsigned at, int row0, const uint4* kept, int lane,
                                             const vec8 (&f)[kSteps]) {
    vec8 x[2], y[2];
    auto read = [&](int k) {
        x[k & 1] = lds_rows(at, row0, k);
        if (k < COUNT) y[k & 1] = __builtin_bit_cast(vec8, kept[64 * k + lane]);
    };
    read(0);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        if (k + 1 < kSteps) read(k + 1);
        fence();
        s = mma(x[k & 1], k < COUNT ? y[k & 1] : f[k], s);
    }
}

__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Values loaded before a loop are waited for before it: inside, the wait would
// be for the tile under way as well, each time round.
template <int N>
__device__ __forceinline__ void settle(vec8 (&x)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+v"(x[k]));
}

__device__ __forceinline__ vec8 load_chunk(const elem* row, int c, int width) {
    return c * 8 < width ? *(const vec8*)(row + c * 8) : zero8();
}

// The lane's query row of a row tile.
struct Row {
    int i, head;         // query of the document, head
    bool real;
    long long token;     // of a row that exists (clamped)
    int limit;           // visible keys
    float steep;         // slope log2(e) 2^23
    uint2 pos;
};

template <int AX>
__device__ __forceinline__ Row get_row(const AttArgs& a, const Range& d, int kvh, int r) {
    Row w;
    const int rows = d.lq * a.group;
    w.real = r < rows;
    const int rr = min(r, rows - 1);
    w.i = rr / a.group;
    w.head = kvh * a.group + rr % a.group;
    w.token = d.qlo + w.i;
    w.limit = w.real ? key_limit(a, d, w.i) : 0;
    w.steep = 0.0f;
    w.pos = make_uint2(0, 0);
    if (AX) {
        w.steep = a.slopes[w.head] * kLog2e * 0x1p23f;
        w.pos = pack_pos(load_pos<AX>(a.q_pos, a.qp_st, a.qp_sa, a.axes, w.token));
    }
    return w;
}

// Base-2 scores less `sub` of a 32-key block, in place, from products that
// started with first_summand(sub). AX: 0 no bias, 2 one or two axes, 3 three.
// kpx, kpy: the block's packed key positions. CAP: bent receives
// tanh(score / cap).
template <int AX, bool CAP>
__device__ __forceinline__ void scores(const AttArgs& a, acc16& s, acc16& bent, const Row& row,
                                       float sub, const unsigned* kpx, const unsigned* kpy, int half) {
    if (CAP) {
        cap_block(a, s);
        bent = s;
    }
    const float by = CAP ? a.cap2 : a.scale2;
    if (!AX) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], by, -sub);
        return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 x = *(const uint4*)(kpx + 8 * q + 4 * half);
        uint4 y = make_uint4(0, 0, 0, 0);
        if (AX == 3) y = *(const uint4*)(kpy + 8 * q + 4 * half);
        const float t[4] = {bias<AX>(row.pos, x.x, y.x, row.steep), bias<AX>(row.pos, x.y, y.y, row.steep),
                            bias<AX>(row.pos, x.z, y.z, row.steep), bias<AX>(row.pos, x.w, y.w, row.steep)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s[4 * q + j] = __builtin_fmaf(s[4 * q + j], by, CAP ? t[j] - sub : t[j]);
    }
}

// Scores of keys from `limit` on become -inf; key0: the block's first key.
__device__ __forceinline__ void hide(acc16& s, int key0, int limit, int half) {
    const int left = limit - key0 - 4 * half;
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if (8 * (r / 4) + r % 4 >= left) s[r] = -__builtin_inff();
}

// Logical block: which (split, row tile, key head); consecutive ones share
// keys and run on one XCD.
__device__ __forceinline__ unsigned xcd_block(unsigned bid, unsigned n) {
    const unsigned q = n / 8, r = n % 8;
    const unsigned x = bid % 8, y = bid / 8;
    return x * q + (x < r ? x : r) + y;
}

// ---- forward ---------------------------------------------------------------
// Scores are computed less m, kTop under the maximum of the tiles before, so
// the largest of a tile says how far m lags; up to 2^kRescale nothing is
// rescaled.
// Key tiles are loaded one ahead into the other half of LDS.
// Bound by vector instructions: with a bias a score takes 6 and an exp2 (the
// bias 2, scale, half a max, sum, half a conversion), 1312 cycles per 32 x 64
// scores against 512 of the matrix units at a width of 64. 12,000 tokens, 8
// heads of 64, two axes: 403 us a call, 732 TFLOP/s; six prefixes of 2,300, 16
// on 4 heads of 128, cap: 242, 745 (of a card whose clock has settled; the first
// tens of calls after a pause take up to 510 and 310). One token of 16 scenes
// against 12,000 keys at most is bound by memory: 65 us, 4.8 TB/s, and 4.6 for
// the join.
// Three wavefronts share a SIMD where they fit without spilling.

template <int AX, bool CAP, int NW, int BN>
__global__ __launch_bounds__(64 * NW, NW == 4 && (W < 128 || AX == 0) ? 3 : NW == 4 || W < 128 || AX == 0 ? 2 : 1) void k_att_forward(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int NB = BN / 32;
    typedef Tile<BN, NT> KeyTile;
    __shared__ __align__(256) uint4 tk[2][BN * kChunks];
    __shared__ __align__(256) uint4 tv[2][BN * kChunks];
    __shared__ __align__(16) unsigned kpx[2][AX ? BN : 4], kpy[2][AX == 3 ? BN : 4];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    unsigned id = a.first_block + xcd_block(blockIdx.x, gridDim.x);
    const int split = (int)(id % a.nsplit);
    id /= a.nsplit;
    const int tile = a.tiles - 1 - (int)(id % a.tiles);  // long causal rows first
    const int kvh = (int)(id / a.tiles);

    int first;
    const int range = find_range<kAttRows * NW>(a.q_offsets, a.docs, a.tq, a.group, tile, &first);
    const Range d = get_range(a, range);
    const int rows = d.lq * a.group;
    const long long row0l = (long long)(tile - first) * kAttRows * NW;
    if (row0l < 0 || row0l >= rows) return;
    const int row0 = (int)row0l;
    const Row row = get_row<AX>(a, d, kvh, row0 + wave * kAttRows + (lane & 31));

    // the block's keys: up to its last row's limit, this split's share of the tiles
    const int last = min(row0 + kAttRows * NW, rows) - 1;
    const int tiles = (key_limit(a, d, last / a.group) + BN - 1) / BN;
    const int t0 = (int)((long long)tiles * split / a.nsplit);
    const int t1 = (int)((long long)tiles * (split + 1) / a.nsplit);
    // keys every row of the block sees (rows past the end hold nothing that is kept)
    const int common = key_limit(a, d, row0 / a.group);

    const elem* k0 = (const elem*)a.k + (long long)kvh * a.k_sh + d.klo * a.k_st;
    const elem* v0 = (const elem*)a.v + (long long)kvh * a.v_sh + d.klo * a.v_st;
    int3 ahead = make_int3(0, 0, 0);
    auto fetch = [&](int t) {
        KeyTile::load(tk[t & 1], k0 + (long long)t * BN * a.k_st, a.k_st, d.lk - t * BN, a.width);
        KeyTile::load(tv[t & 1], v0 + (long long)t * BN * a.v_st, a.v_st, d.lk - t * BN, a.width);
        if (AX && threadIdx.x < BN)
            ahead = load_pos<AX>(a.k_pos, a.kp_st, a.kp_sa, a.axes,
                                 d.klo + min(t * BN + (int)threadIdx.x, d.lk - 1));
    };
    for (int b = 0; b < 2; ++b) {
        KeyTile::clear(tk[b], a.width);
        KeyTile::clear(tv[b], a.width);
    }
    if (a.width < W) __syncthreads();
    if (t0 < t1) fetch(t0);

    vec8 qf[kSteps];
    const elem* qrow = (const elem*)a.q + row.token * a.q_st + row.head * a.q_sh;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) qf[k] = load_chunk(qrow, 2 * k + half, a.width);
    settle(qf);

    acc16 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] = 0.0f;
    float m = 0.0f, l = 0.0f;

    for (int t = t0; t < t1; ++t) {
        const int buf = t & 1;
        if (AX && threadIdx.x < BN) {
            const uint2 pos = pack_pos(ahead);
            kpx[buf][threadIdx.x] = pos.x;
            if (AX == 3) kpy[buf][threadIdx.x] = pos.y;
        }
        landed();
        __syncthreads();  // this tile is there, and all are done with the one before
        if (t + 1 < t1) fetch(t + 1);

        const int ln = fresh(lane);
        const unsigned k_at = lds_address(tk[0]) + rows_place(ln) + buf * sizeof(tk[0]);
        uint2 v_at = columns_place(ln);
        v_at.x += lds_address(tv[0]) + buf * sizeof(tv[0]), v_at.y += lds_address(tv[0]) + buf * sizeof(tv[0]);
        acc16 s[NB];
        vec8 vf[2][kBlocks];
        const float start = first_summand<AX, CAP>(a, m);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[nb][r] = start;
            product(s[nb], k_at, 32 * nb, qf);
        }
        read_columns(v_at, 0, vf[0]);
        fence();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            acc16 none;
            scores<AX, CAP>(a, s[nb], none, row, m, kpx[buf] + (AX ? 32 * nb : 0),
                            kpy[buf] + (AX == 3 ? 32 * nb : 0), half);
        }
        if ((t + 1) * BN > common) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) hide(s[nb], t * BN + 32 * nb, row.limit, half);
        }
        float top = s[0][0];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[nb][r]);
        if (t == t0 || __any(top > kTop + kRescale)) {
            top = fmaxf(top, other_half(top));
            // a row's visible keys are its document's first ones: it sees some
            // in the first tile or none at all
            const float up = t == t0 ? (top > -__builtin_inff() ? top - kTop : 0.0f) : fmaxf(top - kTop, 0.0f);
            m += up;
            if (t > t0) {
                const float w = exp2_(-up);
                l *= w;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[b][r] *= w;
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[nb][r] -= up;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[nb][r] = exp2_(s[nb][r]);
                l += s[nb][r];
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // the next 16 keys' values while these are worked on
                if (2 * nb + c + 1 < 2 * NB) read_columns(v_at, 32 * nb + 16 * (c + 1), vf[(c + 1) & 1]);
                const vec8 p = round8(s[nb], c);
                fence();
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) o[b] = mma(vf[c][b], p, o[b]);
            }
        }
    }
    l += other_half(l);
    if (!row.real) return;
    const bool none = l == 0.0f;  // sees no key: zeros, whatever the tiles held
    const long long at = row.token * a.heads + row.head;
    if (a.nsplit > 1) {
        const long long n = (long long)a.tq * a.heads;
        float* part = a.part_o + ((long long)split * n + at) * a.width;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = 32 * b + 8 * q + 4 * half;
                if (c < a.width)
                    *(float4*)(part + c) =
                        none ? make_float4(0, 0, 0, 0)
                             : make_float4(o[b][4 * q], o[b][4 * q + 1], o[b][4 * q + 2], o[b][4 * q + 3]);
            }
        if (half == 0) {
            a.part_ml[2 * ((long long)split * n + at)] = none ? kLowest : m;
            a.part_ml[2 * ((long long)split * n + at) + 1] = l;
        }
        return;
    }
    const float inv = 1.0f / l;
    elem* out = (elem*)a.out + at * a.width;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * b + 8 * q + 4 * half;
            if (c >= a.width) continue;
            vec4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = none ? (elem)0.0f : (elem)(o[b][4 * q + j] * inv);
            *(vec4*)(out + c) = x;
        }
    if (a.lse && half == 0)
        a.lse[at] = none ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Splits of a row joined in order: one wavefront per row, lanes over the width.
__global__ __launch_bounds__(256) void k_att_join(AttArgs a) {
    const long long n = (long long)a.tq * a.heads;
    const long long at = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (at >= n) return;
    const int lane = threadIdx.x & 63;
    // lane s holds split s (there are at most 64)
    float m = kLowest, l = 0.0f;
    if (lane < a.nsplit) {
        m = a.part_ml[2 * (lane * n + at)];
        l = a.part_ml[2 * (lane * n + at) + 1];
    }
    float top = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float weight = exp2_(m - top);
    m = top;
    l *= weight;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) l += __shfl_xor(l, off);
    float x = 0.0f, y = 0.0f;
    for (int s0 = 0; s0 < a.nsplit; s0 += 8) {
        float2 p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = min(s0 + j, a.nsplit - 1);
            p[j] = make_float2(0.0f, 0.0f);
            if (2 * lane < a.width) p[j] = *(const float2*)(a.part_o + (s * n + at) * a.width + 2 * lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), min(s0 + j, 63)));
            if (s0 + j < a.nsplit) {
                x = __builtin_fmaf(w, p[j].x, x);
                y = __builtin_fmaf(w, p[j].y, y);
            }
        }
    }
    const float inv = 1.0f / l;
    const bool none = l == 0.0f;
    typedef elem vec2 __attribute__((ext_vector_type(2)));
    if (2 * lane < a.width) {
        vec2 r;
        r[0] = none ? (elem)0.0f : (elem)(x * inv);
        r[1] = none ? (elem)0.0f : (elem)(y * inv);
        *(vec2*)((elem*)a.out + at * a.width + 2 * lane) = r;
    }
    if (a.lse && lane == 0)
        a.lse[at] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---- grad_q ----------------------------------------------------------------
// With P = exp2(score - lse), delta = sum(grad_out * out) and dP = grad_out V^T:
// dS = P (dP - delta) (times 1 - tanh^2 under a cap), grad_q = scale dS K. The
// same transposed products as the forward's, one more for dP, and one for P K:
// out is rounded, so its delta is off by up to half a step of |grad_out|.|out|,
// and where one key has nearly all the weight dP - delta is smaller than that.
// The error is r = sum P (dP - delta), known at the end of the row; there
// grad_q loses r P K, and grad_k and grad_v get the delta that is right in
// 32 bits.
// Bound by the waits between one product's result and the next's operand, with
// two wavefronts a SIMD to fill them: four frames of up to 4,096, 8 heads on 2
// of 128, in 530 us (the first ten calls 555), the matrix units busy for a third
// of it.

template <int AX, bool CAP, int NW, int BN>
__global__ __launch_bounds__(64 * NW, NW == 1 && W == 32 ? 3 : NW == 4 || W < 128 ? 2 : 1) void k_att_grad_q(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int NB = BN / 32;
    typedef Tile<BN, NT> KeyTile;
    __shared__ __align__(256) uint4 tk[2][BN * kChunks];
    __shared__ __align__(256) uint4 tv[2][BN * kChunks];
    __shared__ __align__(16) unsigned kpx[2][AX ? BN : 4], kpy[2][AX == 3 ? BN : 4];

    constexpr bool kKeep = W == 128 && NW == 4;
    constexpr int kKeepQ = kKeep ? 3 : 0;  // of q's steps, what LDS has left for two blocks a CU
    __shared__ uint4 kept[kKeep ? NW : 1][kKeep ? 64 * kSteps : 1];
    __shared__ uint4 kept_q[kKeep ? NW : 1][kKeep ? 64 * kKeepQ : 1];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const unsigned id = a.first_block + xcd_block(blockIdx.x, gridDim.x);
    const int tile = a.tiles - 1 - (int)(id % a.tiles);
    const int kvh = (int)(id / a.tiles);
    int first;
    const int range = find_range<kAttRows * NW>(a.q_offsets, a.docs, a.tq, a.group, tile, &first);
    const Range d = get_range(a, range);
    const int rows = d.lq * a.group;
    const long long row0l = (long long)(tile - first) * kAttRows * NW;
    if (row0l < 0 || row0l >= rows) return;
    const int row0 = (int)row0l;
    const Row row = get_row<AX>(a, d, kvh, row0 + wave * kAttRows + (lane & 31));
    const int last = min(row0 + kAttRows * NW, rows) - 1;
    const int t1 = (key_limit(a, d, last / a.group) + BN - 1) / BN;
    const int common = row0 + kAttRows * NW <= rows ? key_limit(a, d, row0 / a.group) : 0;

    const elem* k0 = (const elem*)a.k + (long long)kvh * a.k_sh + d.klo * a.k_st;
    const elem* v0 = (const elem*)a.v + (long long)kvh * a.v_sh + d.klo * a.v_st;
    int3 ahead = make_int3(0, 0, 0);
    auto fetch = [&](int t) {
        KeyTile::load(tk[t & 1], k0 + (long long)t * BN * a.k_st, a.k_st, d.lk - t * BN, a.width);
        KeyTile::load(tv[t & 1], v0 + (long long)t * BN * a.v_st, a.v_st, d.lk - t * BN, a.width);
        const int tid = fresh(threadIdx.x);
        if (AX && tid < BN)
            ahead = load_pos<AX>(a.k_pos, a.kp_st, a.kp_sa, a.axes,
                                 d.klo + min(t * BN + tid, d.lk - 1));
    };
    for (int b = 0; b < 2; ++b) {
        KeyTile::clear(tk[b], a.width);
        KeyTile::clear(tv[b], a.width);
    }
    if (a.width < W) __syncthreads();
    if (t1 > 0) fetch(0);

    const long long at = row.token * a.heads + row.head;
    vec8 qf[kSteps], gf[kSteps];
    const elem* qrow = (const elem*)a.q + row.token * a.q_st + row.head * a.q_sh;
    const elem* grow = (const elem*)a.g + row.token * a.g_st + row.head * a.g_sh;
    const elem* orow = (const elem*)a.o + at * a.width;
    float delta = 0.0f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        qf[k] = load_chunk(qrow, 2 * k + half, a.width);
        gf[k] = load_chunk(grow, 2 * k + half, a.width);
        const vec8 of = load_chunk(orow, 2 * k + half, a.width);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta = __builtin_fmaf((float)gf[k][j], (float)of[j], delta);
    }
    delta += other_half(delta);
    float lse2 = a.lse[at] * kLog2e - kLift;
    settle(qf);
    if constexpr (kKeep) {
        keep<0, kSteps>(kept[wave], lane, gf);
        keep<0, kKeepQ>(kept_q[wave], lane, qf);
    } else {
        settle(gf);
    }
    asm volatile("" : "+v"(lse2));

    const float start = first_summand<AX, CAP>(a, lse2);
    acc16 o[kBlocks], pk[kBlocks];
    float rest = 0.0f;
    Lift lift;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] = pk[b][r] = 0.0f;

    for (int t = 0; t < t1; ++t) {
        const int buf = t & 1;
        const int tid = fresh(threadIdx.x);
        if (AX && tid < BN) {
            const uint2 pos = pack_pos(ahead);
            kpx[buf][tid] = pos.x;
            if (AX == 3) kpy[buf][tid] = pos.y;
        }
        landed();
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);
        const bool masked = (t + 1) * BN > common;
        const int ln = fresh(lane);
        const unsigned k_at = lds_address(tk[0]) + rows_place(ln) + buf * sizeof(tk[0]);
        const unsigned v_at = lds_address(tv[0]) + rows_place(ln) + buf * sizeof(tv[0]);
        uint2 kt_at = columns_place(ln);
        kt_at.x += lds_address(tk[0]) + buf * sizeof(tk[0]), kt_at.y += lds_address(tk[0]) + buf * sizeof(tk[0]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            acc16 s, dp, bent;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = start;
            if constexpr (kKeep)
                product_kept<kKeepQ>(s, k_at, 32 * nb, kept_q[wave], ln, qf);
            else
                product(s, k_at, 32 * nb, qf);
            scores<AX, CAP>(a, s, bent, row, lse2, kpx[buf] + (AX ? 32 * nb : 0),
                            kpy[buf] + (AX == 3 ? 32 * nb : 0), half);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = exp2_(s[r]);
            const int left = masked ? row.limit - (t * BN + 32 * nb) - 4 * half : 32;
            if (masked) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r / 4) + r % 4 >= left) s[r] = 0.0f;
            }
            if (CAP) {
#pragma unroll
                for (int r = 0; r < 16; ++r) bent[r] = __builtin_fmaf(-bent[r], bent[r], 1.0f);
            }
            vec8 kt[2][kBlocks];
            if (!kKeep) {
                read_columns(kt_at, 32 * nb, kt[0]);
                read_columns(kt_at, 32 * nb + 16, kt[1]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (kKeep) {  // read when used, and again below: registers for one set
                    fence();
                    read_columns(kt_at, 32 * nb + 16 * c, kt[c]);
                }
                acc16 flat = s;
                if (CAP) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) flat[r] *= bent[r];
                }
                const vec8 p = round8(flat, c);
                fence();
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) pk[b] = mma(kt[c][b], p, pk[b]);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) dp[r] = -delta;
            if constexpr (kKeep)
                product_kept<kSteps>(dp, v_at, 32 * nb, kept[wave], ln, gf);
            else
                product(dp, v_at, 32 * nb, gf);
            fence();
            if (masked) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r / 4) + r % 4 >= left) dp[r] = 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                dp[r] *= s[r];
                rest += dp[r];
            }
            if (CAP) {
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] *= bent[r];
            }
            lift.apply(dp, o);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (kKeep) {
                    fence();
                    read_columns(kt_at, 32 * nb + 16 * c, kt[c]);
                }
                const vec8 ds = round8(dp, c);
                fence();
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) o[b] = mma(kt[c][b], ds, o[b]);
            }
        }
    }
    rest = (rest + other_half(rest)) * kUnlift;
    const float undo = lift.undo();
    if (!row.real) return;
    // saw no key, or one, whose weight is 1 whatever its score: no gradient
    const bool none = row.limit <= 1;
    if (half == 0) a.delta[at] = delta + rest;
    elem* out = (elem*)a.gq + at * a.width;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * b + 8 * q + 4 * half;
            if (c >= a.width) continue;
            vec4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = none ? (elem)0.0f
                            : (elem)(__builtin_fmaf(-rest, pk[b][4 * q + j], o[b][4 * q + j] * undo) * (a.scale * kUnlift));
            *(vec4*)(out + c) = x;
        }
}

// ---- grad_k and grad_v -------------------------------------------------------
// A wavefront owns 32 keys and runs over the document's queries, one head of
// the group after another: S = Q K^T and dP = grad_out V^T with a lane's column
// one key, so P and dS are operand B of grad_v^T = grad_out^T P and
// grad_k^T = Q^T dS. The weights' product goes before dP, so that fewer values
// are alive at once. Bound as grad_q; the same frames in 511 us
// (the first ten calls 541).

template <int AX, bool CAP, int NW>
__global__ __launch_bounds__(64 * NW, NW == 1 && W == 32 ? 3 : NW == 4 || W < 128 ? 2 : 1) void k_att_grad_kv(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int BM = 32;
    typedef Tile<BM, NT> RowTile;
    __shared__ __align__(256) uint4 tq[2][BM * kChunks];
    __shared__ __align__(256) uint4 tg[2][BM * kChunks];
    __shared__ __align__(16) float rlse[2][BM], rdelta[2][BM];
    __shared__ __align__(16) unsigned rpx[2][BM], rpy[2][BM];

    constexpr bool kKeep = W == 128 && NW == 4;
    __shared__ uint4 kept[kKeep ? NW : 1][kKeep ? 64 * kSteps : 1];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    unsigned id = a.first_block + xcd_block(blockIdx.x, gridDim.x);
    const int split = (int)(id % a.nsplit);
    id /= a.nsplit;
    const int tile = (int)(id % a.tiles);  // causal: the first keys have the most rows
    const int kvh = (int)(id / a.tiles);
    int first;
    const int range = find_range<kAttRows * NW>(a.k_offsets, a.docs, a.tk, 1, tile, &first);
    Range d = get_range(a, range);
    const int lk = max(0, tok_boundary(a.k_offsets, a.docs, a.tk, range + 1) - d.klo);
    const long long key0l = (long long)(tile - first) * kAttRows * NW;
    if (key0l < 0 || key0l >= lk) return;
    const int key0 = (int)key0l;
    const int key = key0 + wave * kAttRows + (lane & 31);
    const long long token = d.klo + min(key, lk - 1);
    if (d.lk == 0) d.lq = 0;  // keys of no document are read by nobody: no rows

    // the first query that sees the block's first key (limits grow with the query)
    int i0 = 0;
    if (a.mask && d.prefix <= key0) i0 = max(0, key0 - (d.lk - d.lq));
    const int first_tile = i0 / BM, per_head = max(0, (d.lq + BM - 1) / BM - first_tile);
    // this split's share of the tiles
    const long long tiles = (long long)per_head * a.group;
    const int t0 = (int)(tiles * split / a.nsplit), t1 = (int)(tiles * (split + 1) / a.nsplit);
    int g = per_head > 0 ? t0 / per_head : 0;
    int i = (first_tile + t0 - g * per_head) * BM;

    float s_lse = 0.0f, s_delta = 0.0f;
    int3 s_pos = make_int3(0, 0, 0);
    auto fetch = [&](int t, int g, int i) {
        const int head = kvh * a.group + g;
        RowTile::load(tq[t & 1], (const elem*)a.q + (long long)head * a.q_sh + (long long)(d.qlo + i) * a.q_st,
                      a.q_st, d.lq - i, a.width);
        RowTile::load(tg[t & 1], (const elem*)a.g + (long long)head * a.g_sh + (long long)(d.qlo + i) * a.g_st,
                      a.g_st, d.lq - i, a.width);
        const int tid = fresh(threadIdx.x);
        if (tid < BM) {
            const long long q = d.qlo + min(i + tid, d.lq - 1);
            s_lse = a.lse[q * a.heads + head];
            s_delta = a.delta[q * a.heads + head];
            s_pos = load_pos<AX>(a.q_pos, a.qp_st, a.qp_sa, a.axes, q);
        }
    };
    for (int b = 0; b < 2; ++b) {
        RowTile::clear(tq[b], a.width);
        RowTile::clear(tg[b], a.width);
    }
    if (a.width < W) __syncthreads();
    if (t0 < t1) fetch(t0, g, i);

    vec8 kf[kSteps], vf[kSteps];
    const elem* krow = (const elem*)a.k + token * a.k_st + kvh * a.k_sh;
    const elem* vrow = (const elem*)a.v + token * a.v_st + kvh * a.v_sh;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        kf[k] = load_chunk(krow, 2 * k + half, a.width);
        vf[k] = load_chunk(vrow, 2 * k + half, a.width);
    }
    uint2 kpos = make_uint2(0, 0);
    if (AX && t0 < t1) kpos = pack_pos(load_pos<AX>(a.k_pos, a.kp_st, a.kp_sa, a.axes, token));
    float steep = AX && t0 < t1 ? a.slopes[kvh * a.group + g] * kLog2e * 0x1p23f : 0.0f;
    if constexpr (kKeep)
        keep<0, kSteps>(kept[wave], lane, kf);
    else
        settle(kf);
    settle(vf);
    asm volatile("" : "+v"(kpos.x), "+v"(kpos.y), "+v"(steep));

    acc16 gk[kBlocks], gv[kBlocks];
    Lift lift;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) gk[b][r] = gv[b][r] = 0.0f;

    for (int t = t0; t < t1; ++t) {
        const int buf = t & 1;
        const int tid = fresh(threadIdx.x);
        if (tid < BM) {
            const float lse2 = s_lse * kLog2e - kLift;
            rlse[buf][tid] = AX && !CAP ? first_summand<AX, CAP>(a, lse2) : -lse2;
            rdelta[buf][tid] = -s_delta;
            const uint2 pos = pack_pos(s_pos);
            if (AX) rpx[buf][tid] = pos.x;
            if (AX == 3) rpy[buf][tid] = pos.y;
        }
        landed();
        __syncthreads();
        const bool turn = i + BM >= d.lq;  // the head's last tile
        if (t + 1 < t1) fetch(t + 1, turn ? g + 1 : g, turn ? first_tile * BM : i + BM);

        const int ln = fresh(lane);
        const unsigned q_at = lds_address(tq[0]) + rows_place(ln) + buf * sizeof(tq[0]);
        const unsigned g_at = lds_address(tg[0]) + rows_place(ln) + buf * sizeof(tg[0]);
        uint2 qt_at = columns_place(ln), gt_at = qt_at;
        qt_at.x += lds_address(tq[0]) + buf * sizeof(tq[0]), qt_at.y += lds_address(tq[0]) + buf * sizeof(tq[0]);
        gt_at.x += lds_address(tg[0]) + buf * sizeof(tg[0]), gt_at.y += lds_address(tg[0]) + buf * sizeof(tg[0]);
        acc16 s, dp, bent;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float4 ls = make_float4(0, 0, 0, 0);
            if (AX && !CAP) ls = *(const float4*)(rlse[buf] + 8 * q + 4 * half);
            s[4 * q + 0] = ls.x, s[4 * q + 1] = ls.y, s[4 * q + 2] = ls.z, s[4 * q + 3] = ls.w;
        }
        if constexpr (kKeep)
            product_kept<kSteps>(s, q_at, 0, kept[wave], ln, kf);
        else
            product(s, q_at, 0, kf);
        if (CAP) {
            cap_block(a, s);
            bent = s;
        }
        const float by = CAP ? a.cap2 : a.scale2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (!AX || CAP) {
                const float4 ls = *(const float4*)(rlse[buf] + 8 * q + 4 * half);
                t[0] = ls.x, t[1] = ls.y, t[2] = ls.z, t[3] = ls.w;
            }
            if (AX) {
                const uint4 x = *(const uint4*)(rpx[buf] + 8 * q + 4 * half);
                uint4 y = make_uint4(0, 0, 0, 0);
                if (AX == 3) y = *(const uint4*)(rpy[buf] + 8 * q + 4 * half);
                const float u[4] = {bias<AX>(kpos, x.x, y.x, steep), bias<AX>(kpos, x.y, y.y, steep),
                                    bias<AX>(kpos, x.z, y.z, steep), bias<AX>(kpos, x.w, y.w, steep)};
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = CAP ? t[j] + u[j] : u[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[4 * q + j] = exp2_(__builtin_fmaf(s[4 * q + j], by, t[j]));
        }
        // every row of the tile sees every key of the block, and two or more?
        const int least = key_limit(a, d, i);
        const bool masked = i + BM > d.lq || least < min(key0 + kAttRows * NW, lk) || least <= 1;
        unsigned seen = 0xffffu, moved = 0xffffu;  // weights, and those that a score can change
        if (masked) {
            seen = moved = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int q = i + 8 * (r / 4) + 4 * half + r % 4;
                const int limit = key_limit(a, d, q);
                if (q < d.lq && key < limit) seen |= 1u << r;
                if (q < d.lq && key < limit && limit > 1) moved |= 1u << r;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!(seen >> r & 1)) s[r] = 0.0f;
        }
        vec8 col[2][kBlocks];
        read_columns(gt_at, 0, col[0]);
        read_columns(gt_at, 16, col[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const vec8 p = round8(s, c);
            fence();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) gv[b] = mma(col[c][b], p, gv[b]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 de = *(const float4*)(rdelta[buf] + 8 * q + 4 * half);
            dp[4 * q + 0] = de.x, dp[4 * q + 1] = de.y, dp[4 * q + 2] = de.z, dp[4 * q + 3] = de.w;
        }
        product(dp, g_at, 0, vf);
        read_columns(qt_at, 0, col[0]);
        fence();
        if (masked) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!(moved >> r & 1)) dp[r] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] *= s[r];
        if (CAP) {
#pragma unroll
            for (int r = 0; r < 16; ++r) dp[r] *= __builtin_fmaf(-bent[r], bent[r], 1.0f);
        }
        lift.apply(dp, gk);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (c == 0) read_columns(qt_at, 16, col[1]);
            const vec8 ds = round8(dp, c);
            fence();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) gk[b] = mma(col[c][b], ds, gk[b]);
        }
        i += BM;
        if (turn) {
            i = first_tile * BM;
            ++g;
            if (AX && t + 1 < t1) steep = a.slopes[kvh * a.group + g] * kLog2e * 0x1p23f;
        }
    }
    if (key >= lk) return;
    const float undo = lift.undo();
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) gk[b][r] *= undo;
    const long long at = token * a.kv_heads + kvh;
    if (a.nsplit > 1) {
        const long long n = (long long)a.tk * a.kv_heads;
        float* pk = a.part_o + ((long long)split * n + at) * a.width;
        float* pv = pk + (long long)a.nsplit * n * a.width;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = 32 * b + 8 * q + 4 * half;
                if (c >= a.width) continue;
                *(float4*)(pk + c) = make_float4(gk[b][4 * q], gk[b][4 * q + 1], gk[b][4 * q + 2], gk[b][4 * q + 3]);
                *(float4*)(pv + c) = make_float4(gv[b][4 * q], gv[b][4 * q + 1], gv[b][4 * q + 2], gv[b][4 * q + 3]);
            }
        return;
    }
    elem* outk = (elem*)a.gk + at * a.width;
    elem* outv = (elem*)a.gv + at * a.width;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * b + 8 * q + 4 * half;
            if (c >= a.width) continue;
            vec4 x, y;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = (elem)(gk[b][4 * q + j] * (a.scale * kUnlift));
                y[j] = (elem)(gv[b][4 * q + j] * kUnlift);
            }
            *(vec4*)(outk + c) = x;
            *(vec4*)(outv + c) = y;
        }
}

// Splits of grad_k and grad_v added in order, four elements per thread.
__global__ __launch_bounds__(256) void k_att_join_kv(AttArgs a) {
    const long long n = (long long)a.tk * a.kv_heads * a.width;
    const long long at = 4 * ((long long)blockIdx.x * 256 + threadIdx.x);
    if (at >= n) return;
    const float* parts[2] = {a.part_o + at, a.part_o + a.nsplit * n + at};
    elem* outs[2] = {(elem*)a.gk + at, (elem*)a.gv + at};
    const float by[2] = {a.scale * kUnlift, kUnlift};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float4 sum = *(const float4*)parts[w];
        for (int s = 1; s < a.nsplit; ++s) {
            const float4 x = *(const float4*)(parts[w] + s * n);
            sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
        }
        vec4 r;
        r[0] = (elem)(sum.x * by[w]), r[1] = (elem)(sum.y * by[w]);
        r[2] = (elem)(sum.z * by[w]), r[3] = (elem)(sum.w * by[w]);
        *(vec4*)outs[w] = r;
    }
}

template <int AX, bool CAP, int NW>
hipError_t launch(AttPass pass, const AttArgs& a, hipStream_t stream) {
    // keys of a tile: 64 where two tiles of k and v, twice, leave LDS for two blocks
    constexpr int BN = NW == 4 && W <= 64 ? 64 : 32, BF = NW == 4 && (W <= 64 || AX) ? 64 : 32;
    const unsigned blocks = (unsigned)a.tiles * a.kv_heads * (pass == kAttGradQ ? 1 : a.nsplit);
    constexpr unsigned kMost = (unsigned)most_blocks(64 * NW);
    for (unsigned first = 0; first < blocks; first += kMost) {
        const dim3 grid(blocks - first < kMost ? blocks - first : kMost), block(64 * NW);
        AttArgs slice = a;
        slice.first_block = first;
        if (pass == kAttForward)
            k_att_forward<AX, CAP, NW, BF><<<grid, block, 0, stream>>>(slice);
        else if (pass == kAttGradQ)
            k_att_grad_q<AX, CAP, NW, BN><<<grid, block, 0, stream>>>(slice);
        else
            k_att_grad_kv<AX, CAP, NW><<<grid, block, 0, stream>>>(slice);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // joins: few rows and keys, or nothing is split
    if (pass == kAttForward && a.nsplit > 1) {
        const long long n = (long long)a.tq * a.heads;
        k_att_join<<<dim3((unsigned)((n + 3) / 4)), dim3(256), 0, stream>>>(a);
    } else if (pass == kAttGradKV && a.nsplit > 1) {
        const long long n = (long long)a.tk * a.kv_heads * a.width / 4;
        k_att_join_kv<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <int AX, bool CAP>
hipError_t launch_waves(AttPass pass, const AttArgs& a, int waves, hipStream_t stream) {
    return waves == 4 ? launch<AX, CAP, 4>(pass, a, stream) : launch<AX, CAP, 1>(pass, a, stream);
}

}  // namespace

#define ATT_JOIN2(a, b, c) att_launch_##a##_##b
#define ATT_JOIN(a, b) ATT_JOIN2(a, b, )
#if ATT_F16
#define ATT_NAME ATT_JOIN(f16, ATT_WIDTH)
#else
#define ATT_NAME ATT_JOIN(bf16, ATT_WIDTH)
#endif

__attribute__((visibility("hidden"))) hipError_t ATT_NAME(AttPass pass, const AttArgs& a, int waves,
                                                          hipStream_t stream) {
    const bool cap = a.cap2 > 0.0f;
    if (a.axes == 0)
        return cap ? launch_waves<0, true>(pass, a, waves, stream)
                   : launch_waves<0, false>(pass, a, waves, stream);
    if (a.axes < 3)
        return cap ? launch_waves<2, true>(pass, a, waves, stream)
                   : launch_waves<2, false>(pass, a, waves, stream);
    return cap ? launch_waves<3, true>(pass, a, waves, stream)
               : launch_waves<3, false>(pass, a, waves, stream);
}
