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
// LDS tiles are rows of 2 * WIDTH bytes with the 16-byte chunks of a row
// permuted by XOR with swz(row), so that both a read of one chunk of 16
// consecutive rows and a transposing read of four consecutive rows times 64
// bytes touch every bank group once.

#include <hip/hip_runtime.h>

#include "attend.h"

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
// at the end: bf16 has the range, and weights that exp2 would flush to zero
// keep their gradient. fp16's largest weights times a gradient would overflow.
constexpr float kLift = ATT_F16 ? 0.0f : 24.0f;
constexpr float kUnlift = ATT_F16 ? 1.0f : 0x1p-24f;
constexpr float kRescale = 8.0f;  // running maximum may lag by this much (base 2)

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

// 16-byte chunk c of a tile row.
__device__ __forceinline__ vec8 lds_chunk(const uint4* tile, int row, int c) {
    return __builtin_bit_cast(vec8, tile[row * kChunks + (c ^ swz(row))]);
}

// Operand A of a transposed product: rows are elements 32 b + lane % 32 of
// the width, inner index the 16 tile rows from row0 in the order above.
__device__ __forceinline__ vec8 lds_transposed(const uint4* tile, int row0, int b, int lane) {
    typedef __attribute__((address_space(3))) short4v lds4;
    const int row = row0 + 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const char* base = (const char*)tile;
    const char* p0 = base + row * (2 * W) + ((c ^ swz(row)) << 4) + ((lane & 1) << 3);
    const char* p1 = base + (row + 8) * (2 * W) + ((c ^ swz(row + 8)) << 4) + ((lane & 1) << 3);
    const short4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p0);
    const short4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p1);
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

// Boundary b of the tokens' ranges: 0, offsets[0 .. docs], total. Range 0 and
// range docs + 1 are the tokens of no document.
__device__ __forceinline__ int boundary(const int* offsets, int docs, int total, int b) {
    if (b <= 0) return 0;
    if (b > docs + 1) return total;
    if (!offsets) return b == 1 ? 0 : total;
    return clampi(offsets[b - 1], 0, total);
}

// Tile t belongs to the last range whose first tile, floor(start * per / size)
// + range, is <= t: that leaves every range at least ceil(length * per / size)
// tiles without anyone knowing the lengths on the host. 64 ranges are tried
// at once.
__device__ __forceinline__ int find_range(const int* offsets, int docs, int total, int per,
                                          int size, int t, int* first_tile) {
    int lo = 0, n = docs + 2;
    const int lane = __lane_id();
    int first = 0;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int b = lo + lane * step;
        const bool in = lane * step < n;
        const int f = in ? (int)((long long)boundary(offsets, docs, total, b) * per / size) + b
                         : 0x7fffffff;
        const unsigned long long hit = __ballot(in && f <= t);
        const int cnt = max(1, (int)__popcll(hit));
        first = __shfl(f, cnt - 1);
        lo += (cnt - 1) * step;
        n = min(step, n - (cnt - 1) * step);
    }
    *first_tile = first;
    return __builtin_amdgcn_readfirstlane(lo);
}

struct Range {
    int qlo, lq, klo, lk, prefix;
};

__device__ __forceinline__ Range get_range(const AttArgs& a, int b) {
    Range r;
    r.qlo = boundary(a.q_offsets, a.docs, a.tq, b);
    r.lq = max(0, boundary(a.q_offsets, a.docs, a.tq, b + 1) - r.qlo);
    r.klo = boundary(a.k_offsets, a.docs, a.tk, b);
    r.lk = max(0, boundary(a.k_offsets, a.docs, a.tk, b + 1) - r.klo);
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
    return clampi(max(d.prefix, min(d.lk, i + d.lk - d.lq + 1)), 0, d.lk);
}

// Positions packed for sad_u16: .x the last two axes, .y the first of three.
__device__ __forceinline__ uint2 pack_pos(const int* pos, long long st, long long sa, int axes,
                                          long long token) {
    const int* p = pos + token * st;
    uint2 r = make_uint2((unsigned)clampi(p[0], 0, 65535), 0u);
    if (axes >= 2) r.x |= (unsigned)clampi(p[sa], 0, 65535) << 16;
    if (axes >= 3) r.y = (unsigned)clampi(p[2 * sa], 0, 65535);
    return r;
}

// |a - b| summed over the axes, as a float: the sums of absolute differences
// are added to the bits of 2^23, whose last place is one.
__device__ __forceinline__ float distance(unsigned ax, unsigned ay, unsigned bx, unsigned by,
                                          bool three) {
    unsigned d = __builtin_amdgcn_sad_u16(ax, bx, 0x4b000000u);
    if (three) d = __builtin_amdgcn_sad_u16(ay, by, d);
    return __uint_as_float(d) - 8388608.0f;
}

// cap tanh(z / cap) in base 2, from e = exp(2 z / cap): tanh = 1 - 2 / (e + 1)
// (e = inf and e = 0 give 1 and -1).
__device__ __forceinline__ float bend(float s, float cap_in) {
    return __builtin_amdgcn_rcpf(exp2_(s * cap_in) + 1.0f);
}

// A tile of ROWS rows of k or v (or q, grad_out) on its way from HBM to LDS:
// NT threads, each some 16-byte chunks, held in registers while the tile
// before it is worked on.
template <int ROWS, int NT>
struct Stage {
    static constexpr int kPer = (ROWS * kChunks + NT - 1) / NT;
    static constexpr bool kEven = ROWS * kChunks % NT == 0;
    uint4 x[kPer];

    // row(r): element offset of tile row r (always a row that may be read)
    template <typename Row>
    __device__ __forceinline__ void load(const void* base, int width, Row row) {
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int at = p * NT + threadIdx.x;
            const int r = at / kChunks, c = at % kChunks;
            x[p] = make_uint4(0, 0, 0, 0);
            if (c * 8 < width && (kEven || r < ROWS)) x[p] = *(const uint4*)((const elem*)base + row(r) + c * 8);
        }
    }
    __device__ __forceinline__ void store(uint4* tile) const {
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int at = p * NT + threadIdx.x;
            const int r = at / kChunks, c = at % kChunks;
            if (kEven || r < ROWS) tile[r * kChunks + (c ^ swz(r))] = x[p];
        }
    }
};

__device__ __forceinline__ vec8 load_chunk(const elem* row, int c, int width) {
    return c * 8 < width ? *(const vec8*)(row + c * 8) : zero8();
}

// The lane's query row of a row tile.
struct Row {
    int i, head;         // query of the document, head
    bool real;
    long long token;     // of a row that exists (clamped)
    int limit;           // visible keys
    float slope2;
    uint2 pos;
};

template <bool GENERAL>
__device__ __forceinline__ Row get_row(const AttArgs& a, const Range& d, int kvh, int r) {
    Row w;
    const int rows = d.lq * a.group;
    w.real = r < rows;
    const int rr = min(r, rows - 1);
    w.i = rr / a.group;
    w.head = kvh * a.group + rr % a.group;
    w.token = d.qlo + w.i;
    w.limit = w.real ? key_limit(a, d, w.i) : 0;
    w.slope2 = 0.0f;
    w.pos = make_uint2(0, 0);
    if (GENERAL && a.axes) {
        w.slope2 = a.slopes[w.head] * kLog2e;
        w.pos = pack_pos(a.q_pos, a.qp_st, a.qp_sa, a.axes, w.token);
    }
    return w;
}

// Base-2 scores of a 32-key block in place. GENERAL: cap and distance.
// kpx, kpy: the block's packed key positions. bent (or null) receives 1 / (e + 1).
template <bool GENERAL, bool KEEP>
__device__ __forceinline__ void scores(const AttArgs& a, acc16& s, acc16& bent, const Row& row,
                                       const unsigned* kpx, const unsigned* kpy, int half) {
    if (!GENERAL) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] *= a.scale2;
        return;
    }
    if (a.cap2 > 0.0f) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float b = bend(s[r], a.cap_in);
            if (KEEP) bent[r] = b;
            s[r] = __builtin_fmaf(-2.0f * a.cap2, b, a.cap2);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] *= a.scale2;
    }
    if (a.axes) {
        if (a.axes < 3) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 x = *(const uint4*)(kpx + 8 * q + 4 * half);
                s[4 * q + 0] = __builtin_fmaf(-row.slope2, distance(row.pos.x, 0, x.x, 0, false), s[4 * q + 0]);
                s[4 * q + 1] = __builtin_fmaf(-row.slope2, distance(row.pos.x, 0, x.y, 0, false), s[4 * q + 1]);
                s[4 * q + 2] = __builtin_fmaf(-row.slope2, distance(row.pos.x, 0, x.z, 0, false), s[4 * q + 2]);
                s[4 * q + 3] = __builtin_fmaf(-row.slope2, distance(row.pos.x, 0, x.w, 0, false), s[4 * q + 3]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 x = *(const uint4*)(kpx + 8 * q + 4 * half);
                const uint4 y = *(const uint4*)(kpy + 8 * q + 4 * half);
                s[4 * q + 0] = __builtin_fmaf(-row.slope2, distance(row.pos.x, row.pos.y, x.x, y.x, true), s[4 * q + 0]);
                s[4 * q + 1] = __builtin_fmaf(-row.slope2, distance(row.pos.x, row.pos.y, x.y, y.y, true), s[4 * q + 1]);
                s[4 * q + 2] = __builtin_fmaf(-row.slope2, distance(row.pos.x, row.pos.y, x.z, y.z, true), s[4 * q + 2]);
                s[4 * q + 3] = __builtin_fmaf(-row.slope2, distance(row.pos.x, row.pos.y, x.w, y.w, true), s[4 * q + 3]);
            }
        }
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
__device__ __forceinline__ long long xcd_block(long long bid, long long n) {
    const long long q = n / 8, r = n % 8;
    const long long x = bid % 8, y = bid / 8;
    return x * q + (x < r ? x : r) + y;
}

// ---- forward ---------------------------------------------------------------

template <bool GENERAL, int NW, int BN>
__global__ __launch_bounds__(64 * NW, NW == 4 ? 2 : 1) void k_att_forward(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int NB = BN / 32;
    __shared__ __align__(16) uint4 tk[BN * kChunks];
    __shared__ __align__(16) uint4 tv[BN * kChunks];
    __shared__ __align__(16) unsigned kpx[GENERAL ? BN : 4], kpy[GENERAL ? BN : 4];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    long long id = xcd_block(blockIdx.x, gridDim.x);
    const int split = (int)(id % a.nsplit);
    id /= a.nsplit;
    const int tile = a.tiles - 1 - (int)(id % a.tiles);  // long causal rows first
    const int kvh = (int)(id / a.tiles);

    int first;
    const int range = find_range(a.q_offsets, a.docs, a.tq, a.group, kAttRows * NW, tile, &first);
    const Range d = get_range(a, range);
    const int rows = d.lq * a.group;
    const long long row0l = (long long)(tile - first) * kAttRows * NW;
    if (row0l < 0 || row0l >= rows) return;
    const int row0 = (int)row0l;
    const Row row = get_row<GENERAL>(a, d, kvh, row0 + wave * kAttRows + (lane & 31));

    // the block's keys: up to its last row's limit, this split's share of the tiles
    const int last = min(row0 + kAttRows * NW, rows) - 1;
    const int tiles = (key_limit(a, d, last / a.group) + BN - 1) / BN;
    const int t0 = (int)((long long)tiles * split / a.nsplit);
    const int t1 = (int)((long long)tiles * (split + 1) / a.nsplit);
    // keys every row of the block sees (rows past the end hold nothing that is kept)
    const int common = key_limit(a, d, row0 / a.group);

    vec8 qf[kSteps];
    const elem* qrow = (const elem*)a.q + row.token * a.q_st + row.head * a.q_sh;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) qf[k] = load_chunk(qrow, 2 * k + half, a.width);

    acc16 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] = 0.0f;
    float m = kLowest, l = 0.0f;

    Stage<BN, NT> sk, sv;
    uint2 sp = make_uint2(0, 0);
    auto fetch = [&](int t) {
        const long long k0 = (long long)kvh * a.k_sh, v0 = (long long)kvh * a.v_sh;
        sk.load(a.k, a.width, [&](int r) {
            return k0 + (long long)(d.klo + min(t * BN + r, d.lk - 1)) * a.k_st;
        });
        sv.load(a.v, a.width, [&](int r) {
            return v0 + (long long)(d.klo + min(t * BN + r, d.lk - 1)) * a.v_st;
        });
        if (GENERAL && a.axes && threadIdx.x < BN)
            sp = pack_pos(a.k_pos, a.kp_st, a.kp_sa, a.axes,
                          d.klo + min(t * BN + (int)threadIdx.x, d.lk - 1));
    };
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; ++t) {
        __syncthreads();
        sk.store(tk);
        sv.store(tv);
        if (GENERAL && threadIdx.x < BN) {
            kpx[threadIdx.x] = sp.x;
            kpy[threadIdx.x] = sp.y;
        }
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);

        acc16 s[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[nb][r] = 0.0f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
                s[nb] = mma(lds_chunk(tk, 32 * nb + (lane & 31), 2 * k + half), qf[k], s[nb]);
            acc16 none;
            scores<GENERAL, false>(a, s[nb], none, row, kpx + 32 * nb, kpy + 32 * nb, half);
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
        top = fmaxf(top, other_half(top));
        if (__any(top > m + kRescale)) {
            const float mn = fmaxf(m, top);
            const float w = exp2_(m - mn);
            m = mn;
            l *= w;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[b][r] *= w;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[nb][r] = exp2_(s[nb][r] - m);
                l += s[nb][r];
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const vec8 p = round8(s[nb], c);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    o[b] = mma(lds_transposed(tv, 32 * nb + 16 * c, b, lane), p, o[b]);
            }
        }
    }
    l += other_half(l);
    if (!row.real) return;
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
                    *(float4*)(part + c) = make_float4(o[b][4 * q], o[b][4 * q + 1],
                                                       o[b][4 * q + 2], o[b][4 * q + 3]);
            }
        if (half == 0) {
            a.part_ml[2 * ((long long)split * n + at)] = m;
            a.part_ml[2 * ((long long)split * n + at) + 1] = l;
        }
        return;
    }
    const float inv = 1.0f / l;
    const bool none = l == 0.0f;  // sees no key: zeros, whatever the tiles held
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
        a.lse[at] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Splits of a row joined in order: one wavefront per row, lanes over the width.
__global__ __launch_bounds__(256) void k_att_join(AttArgs a) {
    const long long n = (long long)a.tq * a.heads;
    const long long at = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (at >= n) return;
    const int lane = threadIdx.x & 63;
    float m = kLowest;
    for (int s = 0; s < a.nsplit; ++s) m = fmaxf(m, a.part_ml[2 * (s * n + at)]);
    float l = 0.0f, x = 0.0f, y = 0.0f;
    for (int s = 0; s < a.nsplit; ++s) {
        const float w = exp2_(a.part_ml[2 * (s * n + at)] - m);
        const float* part = a.part_o + (s * n + at) * a.width;
        l = __builtin_fmaf(w, a.part_ml[2 * (s * n + at) + 1], l);
        if (2 * lane < a.width) {
            const float2 p = *(const float2*)(part + 2 * lane);
            x = __builtin_fmaf(w, p.x, x);
            y = __builtin_fmaf(w, p.y, y);
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

template <bool GENERAL, int NW, int BN>
__global__ __launch_bounds__(64 * NW, NW == 4 ? 2 : 1) void k_att_grad_q(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int NB = BN / 32;
    __shared__ __align__(16) uint4 tk[BN * kChunks];
    __shared__ __align__(16) uint4 tv[BN * kChunks];
    __shared__ __align__(16) unsigned kpx[GENERAL ? BN : 4], kpy[GENERAL ? BN : 4];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const long long id = xcd_block(blockIdx.x, gridDim.x);
    const int tile = a.tiles - 1 - (int)(id % a.tiles);
    const int kvh = (int)(id / a.tiles);
    int first;
    const int range = find_range(a.q_offsets, a.docs, a.tq, a.group, kAttRows * NW, tile, &first);
    const Range d = get_range(a, range);
    const int rows = d.lq * a.group;
    const long long row0l = (long long)(tile - first) * kAttRows * NW;
    if (row0l < 0 || row0l >= rows) return;
    const int row0 = (int)row0l;
    const Row row = get_row<GENERAL>(a, d, kvh, row0 + wave * kAttRows + (lane & 31));
    const int last = min(row0 + kAttRows * NW, rows) - 1;
    const int t1 = (key_limit(a, d, last / a.group) + BN - 1) / BN;
    const int common = row0 + kAttRows * NW <= rows ? key_limit(a, d, row0 / a.group) : 0;

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
    const float lse2 = a.lse[at] * kLog2e - kLift;

    acc16 o[kBlocks], pk[kBlocks];
    float rest = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] = pk[b][r] = 0.0f;

    Stage<BN, NT> sk, sv;
    uint2 sp = make_uint2(0, 0);
    auto fetch = [&](int t) {
        const long long k0 = (long long)kvh * a.k_sh, v0 = (long long)kvh * a.v_sh;
        sk.load(a.k, a.width, [&](int r) {
            return k0 + (long long)(d.klo + min(t * BN + r, d.lk - 1)) * a.k_st;
        });
        sv.load(a.v, a.width, [&](int r) {
            return v0 + (long long)(d.klo + min(t * BN + r, d.lk - 1)) * a.v_st;
        });
        if (GENERAL && a.axes && threadIdx.x < BN)
            sp = pack_pos(a.k_pos, a.kp_st, a.kp_sa, a.axes,
                          d.klo + min(t * BN + (int)threadIdx.x, d.lk - 1));
    };
    if (t1 > 0) fetch(0);
    for (int t = 0; t < t1; ++t) {
        __syncthreads();
        sk.store(tk);
        sv.store(tv);
        if (GENERAL && threadIdx.x < BN) {
            kpx[threadIdx.x] = sp.x;
            kpy[threadIdx.x] = sp.y;
        }
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);
        const bool masked = (t + 1) * BN > common;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            acc16 s, dp, bent;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                s = mma(lds_chunk(tk, 32 * nb + (lane & 31), 2 * k + half), qf[k], s);
                dp = mma(lds_chunk(tv, 32 * nb + (lane & 31), 2 * k + half), gf[k], dp);
            }
            scores<GENERAL, true>(a, s, bent, row, kpx + 32 * nb, kpy + 32 * nb, half);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = exp2_(s[r] - lse2);
            if (masked) {
                const int left = row.limit - (t * BN + 32 * nb) - 4 * half;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r / 4) + r % 4 >= left) s[r] = dp[r] = 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                dp[r] = s[r] * (dp[r] - delta);
                rest += dp[r];
            }
            if (GENERAL && a.cap2 > 0.0f) {
                // 1 - tanh^2 = 4 b (1 - b) with b = 1 / (e + 1)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float flat = 4.0f * bent[r] * (1.0f - bent[r]);
                    dp[r] *= flat;
                    s[r] *= flat;
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const vec8 ds = round8(dp, c), p = round8(s, c);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const vec8 kt = lds_transposed(tk, 32 * nb + 16 * c, b, lane);
                    o[b] = mma(kt, ds, o[b]);
                    pk[b] = mma(kt, p, pk[b]);
                }
            }
        }
    }
    rest = (rest + other_half(rest)) * kUnlift;
    if (!row.real) return;
    const bool none = a.lse[at] == -__builtin_inff();  // saw no key: no gradient
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
            for (int j = 0; j < 4; ++j) x[j] = none ? (elem)0.0f
                            : (elem)(__builtin_fmaf(-rest, pk[b][4 * q + j], o[b][4 * q + j]) * (a.scale * kUnlift));
            *(vec4*)(out + c) = x;
        }
}

// ---- grad_k and grad_v -------------------------------------------------------
// A wavefront owns 32 keys and runs over the document's query rows, all heads
// of the group: S = Q K^T and dP = grad_out V^T with a lane's column one key,
// so P and dS are operand B of grad_v^T = grad_out^T P and grad_k^T = Q^T dS.

template <bool GENERAL, int NW>
__global__ __launch_bounds__(64 * NW, 1) void k_att_grad_kv(AttArgs a) {
    constexpr int NT = 64 * NW;
    constexpr int BM = 32;
    __shared__ __align__(16) uint4 tq[BM * kChunks];
    __shared__ __align__(16) uint4 tg[BM * kChunks];
    __shared__ __align__(16) float rlse[BM], rdelta[BM], rslope[BM];
    __shared__ __align__(16) int rlimit[BM];
    __shared__ __align__(16) unsigned rpx[BM], rpy[BM];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const long long id = xcd_block(blockIdx.x, gridDim.x);
    const int tile = (int)(id % a.tiles);  // causal: the first keys have the most rows
    const int kvh = (int)(id / a.tiles);
    int first;
    const int range = find_range(a.k_offsets, a.docs, a.tk, 1, kAttRows * NW, tile, &first);
    Range d = get_range(a, range);
    const int lk = max(0, boundary(a.k_offsets, a.docs, a.tk, range + 1) - d.klo);
    const long long key0l = (long long)(tile - first) * kAttRows * NW;
    if (key0l < 0 || key0l >= lk) return;
    const int key0 = (int)key0l;
    const int key = key0 + wave * kAttRows + (lane & 31);
    const long long token = d.klo + min(key, lk - 1);
    // keys of no document are read by nobody: no rows
    const int rows = d.lk > 0 ? d.lq * a.group : 0;

    vec8 kf[kSteps], vf[kSteps];
    const elem* krow = (const elem*)a.k + token * a.k_st + kvh * a.k_sh;
    const elem* vrow = (const elem*)a.v + token * a.v_st + kvh * a.v_sh;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        kf[k] = load_chunk(krow, 2 * k + half, a.width);
        vf[k] = load_chunk(vrow, 2 * k + half, a.width);
    }
    uint2 kpos = make_uint2(0, 0);
    if (GENERAL && a.axes && rows) kpos = pack_pos(a.k_pos, a.kp_st, a.kp_sa, a.axes, token);

    acc16 gk[kBlocks], gv[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) gk[b][r] = gv[b][r] = 0.0f;

    // the first query that sees the block's first key (limits grow with the query)
    int i0 = 0;
    if (a.mask && d.prefix <= key0) i0 = max(0, key0 - (d.lk - d.lq));
    const int t0 = i0 * a.group / BM, t1 = (rows + BM - 1) / BM;

    Stage<BM, NT> sq, sg;
    float s_lse = 0.0f, s_delta = 0.0f, s_slope = 0.0f;
    int s_limit = 0;
    uint2 s_pos = make_uint2(0, 0);
    auto fetch = [&](int t) {
        sq.load(a.q, a.width, [&](int r) {
            const int rr = min(t * BM + r, rows - 1);
            return (long long)(d.qlo + rr / a.group) * a.q_st +
                   (long long)(kvh * a.group + rr % a.group) * a.q_sh;
        });
        sg.load(a.g, a.width, [&](int r) {
            const int rr = min(t * BM + r, rows - 1);
            return (long long)(d.qlo + rr / a.group) * a.g_st +
                   (long long)(kvh * a.group + rr % a.group) * a.g_sh;
        });
        if (threadIdx.x < BM) {
            const Row w = get_row<GENERAL>(a, d, kvh, t * BM + threadIdx.x);
            const long long at = w.token * a.heads + w.head;
            s_lse = a.lse[at] * kLog2e - kLift;
            s_delta = a.delta[at];
            s_slope = w.slope2;
            s_limit = w.limit;
            s_pos = w.pos;
        }
    };
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; ++t) {
        __syncthreads();
        sq.store(tq);
        sg.store(tg);
        if (threadIdx.x < BM) {
            rlse[threadIdx.x] = s_lse;
            rdelta[threadIdx.x] = s_delta;
            rlimit[threadIdx.x] = s_limit;
            if (GENERAL) {
                rslope[threadIdx.x] = s_slope;
                rpx[threadIdx.x] = s_pos.x;
                rpy[threadIdx.x] = s_pos.y;
            }
        }
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);

        acc16 s, dp, bent;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            s = mma(lds_chunk(tq, lane & 31, 2 * k + half), kf[k], s);
            dp = mma(lds_chunk(tg, lane & 31, 2 * k + half), vf[k], dp);
        }
        if (GENERAL && a.cap2 > 0.0f) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                bent[r] = bend(s[r], a.cap_in);
                s[r] = __builtin_fmaf(-2.0f * a.cap2, bent[r], a.cap2);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] *= a.scale2;
        }
        if (GENERAL && a.axes) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 sl = *(const float4*)(rslope + 8 * q + 4 * half);
                const uint4 x = *(const uint4*)(rpx + 8 * q + 4 * half);
                const uint4 y = *(const uint4*)(rpy + 8 * q + 4 * half);
                s[4 * q + 0] = __builtin_fmaf(-sl.x, distance(kpos.x, kpos.y, x.x, y.x, true), s[4 * q + 0]);
                s[4 * q + 1] = __builtin_fmaf(-sl.y, distance(kpos.x, kpos.y, x.y, y.y, true), s[4 * q + 1]);
                s[4 * q + 2] = __builtin_fmaf(-sl.z, distance(kpos.x, kpos.y, x.z, y.z, true), s[4 * q + 2]);
                s[4 * q + 3] = __builtin_fmaf(-sl.w, distance(kpos.x, kpos.y, x.w, y.w, true), s[4 * q + 3]);
            }
        }
        // every row of the tile sees every key of the block?
        const bool masked = (t + 1) * BM > rows ||
                            key_limit(a, d, t * BM / a.group) < min(key0 + kAttRows * NW, lk);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 ls = *(const float4*)(rlse + 8 * q + 4 * half);
            s[4 * q + 0] = exp2_(s[4 * q + 0] - ls.x);
            s[4 * q + 1] = exp2_(s[4 * q + 1] - ls.y);
            s[4 * q + 2] = exp2_(s[4 * q + 2] - ls.z);
            s[4 * q + 3] = exp2_(s[4 * q + 3] - ls.w);
        }
        if (masked) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int4 lim = *(const int4*)(rlimit + 8 * q + 4 * half);
                if (key >= lim.x) s[4 * q + 0] = 0.0f;
                if (key >= lim.y) s[4 * q + 1] = 0.0f;
                if (key >= lim.z) s[4 * q + 2] = 0.0f;
                if (key >= lim.w) s[4 * q + 3] = 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const vec8 p = round8(s, c);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                gv[b] = mma(lds_transposed(tg, 16 * c, b, lane), p, gv[b]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 de = *(const float4*)(rdelta + 8 * q + 4 * half);
            dp[4 * q + 0] = s[4 * q + 0] * (dp[4 * q + 0] - de.x);
            dp[4 * q + 1] = s[4 * q + 1] * (dp[4 * q + 1] - de.y);
            dp[4 * q + 2] = s[4 * q + 2] * (dp[4 * q + 2] - de.z);
            dp[4 * q + 3] = s[4 * q + 3] * (dp[4 * q + 3] - de.w);
        }
        if (GENERAL && a.cap2 > 0.0f) {
#pragma unroll
            for (int r = 0; r < 16; ++r) dp[r] *= 4.0f * bent[r] * (1.0f - bent[r]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const vec8 p = round8(dp, c);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                gk[b] = mma(lds_transposed(tq, 16 * c, b, lane), p, gk[b]);
        }
    }
    if (key >= lk) return;
    const long long at = token * a.kv_heads + kvh;
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

template <bool GENERAL, int NW>
hipError_t launch(AttPass pass, const AttArgs& a, hipStream_t stream) {
    constexpr int BN = NW == 4 ? 64 : 32;
    const dim3 block(64 * NW);
    const long long blocks = (long long)a.tiles * a.kv_heads * (pass == kAttForward ? a.nsplit : 1);
    if (blocks <= 0 || blocks > 0x7fffffffll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    if (pass == kAttForward) {
        k_att_forward<GENERAL, NW, BN><<<grid, block, 0, stream>>>(a);
        if (a.nsplit > 1) {
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const long long n = (long long)a.tq * a.heads;
            k_att_join<<<dim3((unsigned)((n + 3) / 4)), dim3(256), 0, stream>>>(a);
        }
    } else if (pass == kAttGradQ) {
        k_att_grad_q<GENERAL, NW, BN><<<grid, block, 0, stream>>>(a);
    } else {
        k_att_grad_kv<GENERAL, NW><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

#define ATT_JOIN2(a, b, c) att_launch_##a##_##b
#define ATT_JOIN(a, b) ATT_JOIN2(a, b, )
#if ATT_F16
#define ATT_NAME ATT_JOIN(f16, ATT_WIDTH)
#else
#define ATT_NAME ATT_JOIN(bf16, ATT_WIDTH)
#endif

__attribute__((visibility("hidden"))) hipError_t ATT_NAME(AttPass pass, const AttArgs& a,
                                                          bool general, int waves,
                                                          hipStream_t stream) {
    if (waves == 4)
        return general ? launch<true, 4>(pass, a, stream) : launch<false, 4>(pass, a, stream);
    return general ? launch<true, 1>(pass, a, stream) : launch<false, 1>(pass, a, stream);
}
