// Attention with decay (tokens.h): forward, backward, and token by token.
//
// S[t] = e^-r S[t-1] + k[t] v[t]^T, out[t] = scale q[t] S[t]. Over a chunk of 32
// tokens, with S the state before it:
//   out[i] = scale (e^-r(i+1) q[i] S + sum over j <= i of e^-r(i-j) (q[i].k[j]) v[j])
//   S'     = e^-rm S + sum over j of e^-r(m-1-j) k[j] v[j]^T   (m tokens)
// which is four small products on matrix instructions. A document is cut into
// segments: k_decay_sum takes what each segment adds to a state, k_decay_join
// turns that into the state that enters each segment, k_decay_run walks the
// segments from there. The gradients are the same walk with other tensors in its
// places: grad_q that of (grad, v, k) with the states transposed, and from the other
// end grad_v that of (k, q, grad) and grad_k that of (v, grad, q).
//
// A block has W / 32 wavefronts, each with 32 columns of the state (all its rows) in
// registers, W the padded width. Everything is taken transposed (out^T = S^T Q^T +
// V^T P^T), so that registers that hold a result are, rounded, the next product's
// operand: a state's column, 8 rows at a time, and a query's weights, 8 keys at a
// time. For that the rows of K, and its columns, are read with bits 2 and 3 of their
// number traded: register 8 c + j of half h then is row 16 c + 8 h + j.
//
// Roundings. The state is in 32 bits, and a result: v e^-r(m-1-j), which enters it, is
// taken in two or three parts of the tensors' type that together hold 22 bits or more. The
// weights (q.k) e^-r(i-j) are taken in two parts: a few tokens' outputs are a few weights'
// and would show each one's rounding. The state's copy for the product with q is rounded
// to the tensors' type, as the 16-bit matrix instructions take it: a sum of `width` such
// roundings, 2.3e-3 of an output in bf16 where the result's own are 1.7e-3. (In two parts it
// would show none: a training step over 122,880 tokens of 8 heads of 128 1,390 us for 1,205, the
// gradients at widths of 64 and less up to 10% more.) In fp16 each of the three is first multiplied
// with a power of two that brings its largest to about 1.
//
// Bounds. k and v are read twice, all else once; the gradients' walks read 7.3 tensors' bytes of
// nine that they ask for and the sums two more, where five would do. 122,880 tokens of 8 heads of
// 128: sums 116 us (530 MB, 4.5 TB/s), their prefix 15, the walk 248 (1.04 GB, 4.2), the gradients'
// three walks 692 (2.6 GB, 3.8). Without its products the walk takes 216 us, without its loads 185:
// with two blocks on a CU, memory and products overlap nearly whole. Sixteen frames of 8 heads of
// 64: 87, 12 and 164 (707 MB, 4.3).
// Windows of a few dozen tokens pay for each block's beginning: 14 us forward, 30 backward.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "decay_parts.h"
#include "mma_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr long long kMaxElems = (1ll << 31) - 4096;
constexpr int kMaxDocs = 1 << 20;
constexpr int kChunk = 32;
constexpr int kAlone = 256;  // tokens of a segment in a call of one launch (of 512: 3,000 next to 300 75 -> 83 us)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLargest = 3.402823466e+38f;

// A tensor in one of the walk's places.
struct Place {
    const void* p;
    long long st, sh;  // token and head stride
    int group;         // query heads that share one of its heads
};

// A walk along the documents: which tensors are in which places, and from which end.
struct Walk {
    Place q, k, v;
    void* out;            // [t, heads, width]; float32 with out_wide
    const float* state;   // [docs, heads, width, width] or null
    float* last;          // or null
    float* carry;         // [rows, heads, width, width]: sums, then the states after them
    int back;             // from a document's last token
    int turned;           // states are read transposed
    int lag;              // 1: a state counts one token on; 0: it is that of the token itself
    int out_wide;
    float near_by, enter_by, leave_by;  // of tokens of a chunk, of the state, of what enters it
};

struct DecayArgs {
    Walk walk[3];
    int walks;
    const int* offsets;
    const float* decay;
    int t, docs, heads, width;
    int segment;          // tokens: a multiple of kChunk
    int segments;
    int more;             // of them, in a call of one launch, those that begin inside a document
    unsigned first_block;
};

// The document, and the part of it, of a segment number: the segments of range b start at
// floor(start / segment) + b, which leaves every range enough without anyone knowing
// the lengths on the host.
struct Part {
    int lo, n;       // the document's first token and its tokens
    int doc;         // -1: of no document
    int from, to;    // tokens of this segment, in the walk's order
    bool none;       // no such segment
    bool last;
    int row;         // of carry, for the state after it
};

__device__ __forceinline__ Part find_part(const DecayArgs& a, int slot) {
    int lo = 0, n = a.docs + 2, first = 0;
    const int lane = __lane_id();
    if (a.segment >= a.t) lo = first = slot, n = 1;  // one segment a range: nothing to search
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave;
        const int b = lo + lane * step;
        const bool in = lane * step < n;
        const int f = in ? tok_boundary(a.offsets, a.docs, a.t, b) / a.segment + b : 0x7fffffff;
        const int cnt = max(1, (int)__popcll(__ballot(in && f <= slot)));
        first = __shfl(f, cnt - 1);
        lo += (cnt - 1) * step;
        n = min(step, n - (cnt - 1) * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    first = __builtin_amdgcn_readfirstlane(first);
    Part p;
    p.lo = tok_boundary(a.offsets, a.docs, a.t, lo);
    p.n = max(0, tok_boundary(a.offsets, a.docs, a.t, lo + 1) - p.lo);
    p.doc = lo >= 1 && lo <= a.docs ? lo - 1 : -1;
    const long long from = (long long)(slot - first) * a.segment;
    p.none = from < 0 || (from > 0 && from >= p.n);
    p.from = p.none ? 0 : (int)from;
    p.to = part_end(p.from, p.n, a.segment);
    p.last = p.to == p.n;
    p.row = slot - lo;
    return p;
}

// A document's segment whose state goes to `row` of carry, if it has one there. Segment p of a
// document, if not its last, has row floor(lo / segment) + p.
__device__ __forceinline__ Part row_of(const DecayArgs& a, int doc, int row) {
    Part p;
    p.doc = doc;
    p.lo = __builtin_amdgcn_readfirstlane(tok_boundary(a.offsets, a.docs, a.t, doc + 1));
    p.n = max(0, __builtin_amdgcn_readfirstlane(tok_boundary(a.offsets, a.docs, a.t, doc + 2)) - p.lo);
    p.row = row < 0 ? p.lo / a.segment : row;  // below zero: its first
    p.from = __builtin_amdgcn_readfirstlane((p.row - p.lo / a.segment) * a.segment);
    p.last = false;
    p.none = doc < 0 || doc >= a.docs || p.from < 0 || p.n - p.from <= a.segment;
    p.to = p.none ? p.from : part_end(p.from, p.n, a.segment);
    return p;
}
// The document that a row is of: the last token of the row's stretch of `segment` tokens is its.
__device__ __forceinline__ int doc_of_row(const DecayArgs& a, int row) {
    return tok_range(a.offsets, a.docs, a.t, (row + 1) * a.segment - 1) - 1;
}

// A document's first tokens, or further ones of a document longer than a segment, where every block
// starts from the document's beginning: the numbers below a.more are those of rows of carry, whose
// segments' successors they are, the longest way first; then one for each range.
__device__ __forceinline__ Part alone_part(const DecayArgs& a, int slot) {
    Part p;
    if (slot < a.more) {
        const int row = a.more - 1 - slot;
        p = row_of(a, doc_of_row(a, row), row);
        if (p.none) return p;
        p.from = p.to;
        p.to = part_end(p.from, p.n, a.segment);
    } else {
        const int range = slot - a.more;
        p.lo = __builtin_amdgcn_readfirstlane(tok_boundary(a.offsets, a.docs, a.t, range));
        p.n = max(0, __builtin_amdgcn_readfirstlane(tok_boundary(a.offsets, a.docs, a.t, range + 1)) - p.lo);
        p.doc = range >= 1 && range <= a.docs ? range - 1 : -1;
        p.from = 0;
        p.to = p.doc < 0 ? p.n : part_end(0, p.n, a.segment);
        p.none = false;
    }
    p.last = p.to == p.n;
    p.row = 0;
    return p;
}

// decay * log2(e) of a head: never negative, and at most what leaves nothing of a token.
__device__ __forceinline__ float rate_of(const DecayArgs& a, int head) {
    return fminf(fmaxf(a.decay[head], 0.0f), 1000.0f) * kLog2e;
}
__device__ __forceinline__ float fall(float rate, int steps) {
    return __builtin_amdgcn_exp2f(-rate * (float)steps);
}

template <typename T, int W>
struct Decay {
    typedef typename Mma<T>::vec8 vec8;
    static constexpr int kWaves = W / 32, NT = 64 * kWaves;
    static constexpr int kPieces = W / 8;           // of 16 bytes in a row
    static constexpr int kTile = kChunk * W * 2;    // bytes
    static constexpr int kBlocks = W / 32;
    // Chunks in LDS at once: at the smallest width, one less lets three wavefronts share a
    // SIMD.
    static constexpr int kBuffers = W == 32 ? 2 : 3;
    static constexpr bool kHalf = __is_same(T, f16_t);

    static __device__ __forceinline__ int swz(int row) {
        if (W == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
        if (W == 64) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
        return (row >> 2) & 3;
    }
    // bits 2 and 3 traded
    static __device__ __forceinline__ int traded(int x) { return (x & ~12) | ((x & 4) << 1) | ((x & 8) >> 1); }

    // The rows of one tensor, chunk by chunk, to LDS.
    struct Rows {
        const T* base;     // the segment's first row in the walk's order
        long long step;    // to the next row
        unsigned offset;   // of this lane's piece, in a whole chunk: from its lowest address on

        __device__ __forceinline__ Rows(const Place& p, int head, const Walk& w, const Part& d) {
            const int first = w.back ? d.lo + d.n - 1 - d.from : d.lo + d.from;
            base = (const T*)p.p + (long long)(head / p.group) * p.sh + first * p.st;
            step = w.back ? -p.st : p.st;
            const int row = threadIdx.x / kPieces, c = (threadIdx.x % kPieces) ^ swz(row);
            offset = (unsigned)(w.back ? kChunk / 2 - 1 - row : row) * (unsigned)(2 * p.st) + 16u * c;
        }
        // Chunk c of `left` rows from there on; zeros past its end and the width.
        __device__ __forceinline__ void load(unsigned to, int chunk, int left, int width) const {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const T* from = base + (long long)chunk * kChunk * step;
            if (left >= kChunk && width == W) {
                const T* low = step < 0 ? from + (kChunk / 2 - 1) * step : from;
                load_to_lds(to + 1024u * wave, low, offset);
                load_to_lds(to + 1024u * wave + 16u * NT, low + kChunk / 2 * step, offset);
                return;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = i * NT + threadIdx.x, row = n / kPieces, c = (n % kPieces) ^ swz(row);
                const bool there = row < left && 8 * c < width;
                load_to_lds(to + 1024u * wave + 16u * NT * i, there ? (const void*)(from + row * step + 8 * c) : &kNothing);
            }
        }
    };
    // Operand of a product over the width: row number `row`, step s of 16.
    static __device__ __forceinline__ unsigned row_place(int row, int half) {
        return row * 2 * W + ((half ^ swz(row)) << 4);
    }
    static __device__ __forceinline__ vec8 read_row(unsigned at, int s) { return lds_read<vec8>(at ^ (s << 5)); }
    // Operand of a product over the tokens: columns of block b, step s of 16 tokens.
    // TRADED: with bits 2 and 3 of the column traded.
    template <bool TRADED>
    static __device__ __forceinline__ uint2 column_place(int lane) {
        const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
        const int four = TRADED ? ((lane & 1) << 1) | ((lane & 2) >> 1) : lane & 3;
        const int c = 2 * ((lane >> 4) & 1) + (four >> 1), in = (four & 1) << 3;
        return make_uint2(row * 2 * W + ((c ^ swz(row)) << 4) + in, (row + 4) * 2 * W + ((c ^ swz(row + 4)) << 4) + in);
    }
    static __device__ __forceinline__ vec8 read_column(uint2 at, int b, int s) {
        const unsigned on = s * 32 * W, flip = b << 6;
        return lds_read_columns<vec8>((at.x ^ flip) + on, (at.y ^ flip) + on);
    }

    // The power of two that brings x to about 1 (1 for 0 and what is not finite).
    static __device__ __forceinline__ float to_one(float x) {
        return x > 0.0f && x <= kLargest
                   ? ldexpf(1.0f, min(max(-__builtin_amdgcn_frexp_expf(x), -120), 120)) : 1.0f;
    }
    static __device__ __forceinline__ float wave_max(float x) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
        return x;
    }

    // This wavefront's columns of a state. Rows 16 c + 8 h + j of block b are
    // registers 8 c + j.
    typedef acc16 State[kBlocks];
    static __device__ __forceinline__ void load_state(State& s, const float* from, int width, bool turned, int column,
                                                      int half) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 32 * b + 16 * c + 8 * half;
                const bool there = from && column < width && row < width;
#pragma unroll
                for (int j = 0; j < 8; ++j) s[b][8 * c + j] = 0.0f;
                if (there && turned) {
                    float x[8];
                    Pack<float, 4>::load(from + column * width + row, *(float(*)[4])x);
                    Pack<float, 4>::load(from + column * width + row + 4, *(float(*)[4])(x + 4));
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[b][8 * c + j] = x[j];
                } else if (there) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[b][8 * c + j] = from[(row + j) * width + column];
                }
            }
    }
    static __device__ __forceinline__ void store_state(const State& s, float* to, int width, int column, int half) {
        if (column >= width) return;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 32 * b + 16 * c + 8 * half;
                if (row >= width) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) to[(row + j) * width + column] = s[b][8 * c + j];
            }
    }

    // What v's rows are multiplied with on their way into the state: e^-r(m - lag - j)
    // (1 for rows that are not there), and leave_by.
    static __device__ __forceinline__ void leaving(float (&w)[16], const Walk& a, float rate, int m, int half) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            w[r] = fall(rate, max(0, m - a.lag - (16 * (r / 8) + 8 * half + r % 8))) * a.leave_by;
    }

    // S <- S + by K^T (w V) over a chunk in LDS, w V in as many parts as hold 22 bits or
    // more of it: 2 of fp16, 3 of bf16.
    static __device__ __forceinline__ void advance(State& s, uint2 k_at, const vec8 (&v)[2], const float (&w)[16], float by) {
        constexpr int kParts = kHalf ? 2 : 3;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = (float)v[r / 8][r % 8] * w[r];
        if (kHalf) {
            float top = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[r]));
            const float up = to_one(wave_max(top));
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] *= up;
            by /= up;
        } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] *= by;
        }
        vec8 y[kParts][2];
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                y[part][r / 8][r % 8] = (T)x[r];
                x[r] -= (float)y[part][r / 8][r % 8];
            }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            acc16 add = zero16();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const vec8 k = read_column(k_at, b, c);
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part) {
                    if (kHalf)
                        add = Mma<T>::mul(k, y[part][c], add);
                    else
                        s[b] = Mma<T>::mul(k, y[part][c], s[b]);
                }
            }
            if (kHalf)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] = __builtin_fmaf(add[r], by, s[b][r]);
        }
    }

    // The state that is kept falls by e^-rm with every chunk. That is applied to its
    // registers only when it comes to 2^-kFall; until then what enters is taken that much
    // larger. (Each further power of two would cost the state a 2^-24 of its precision.)
    struct Fall {
        static constexpr float kFall = 8.0f;
        int tokens = 0;  // since then
        // What the registers are to be multiplied with.
        __device__ __forceinline__ float now(float rate) const { return fall(rate, tokens); }
        // A chunk of m tokens passes; the factor for what enters after it.
        __device__ __forceinline__ float pass(State& s, float rate, int m, bool apply) {
            tokens += m;
            const float exponent = rate * (float)tokens;
            if (!apply && exponent <= kFall) return __builtin_amdgcn_exp2f(exponent);
            const float by = __builtin_amdgcn_exp2f(-exponent);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] *= by;
            tokens = 0;
            return 1.0f;
        }
    };
};

// The segment, head and walk of a block. Walks of one segment run together: the gradients of v and k
// read the same rows of four tensors, from the document's other end than that of q.
__device__ __forceinline__ int block_of(const DecayArgs& a, int* head, int* walk, unsigned apart = 0) {
    // the first `apart` blocks of a launch one by one over the XCDs
    const unsigned bid = blockIdx.x;
    unsigned id = a.first_block + (bid < apart ? bid : apart + xcd_block(bid - apart, gridDim.x - apart));
    *walk = id % a.walks;
    id /= a.walks;
    *head = id % a.heads;
    return id / a.heads;
}

// S <- what it is after the first chunks of a part of a document, all of them whole.
template <typename T, int W>
__device__ __forceinline__ void add_chunks(typename Decay<T, W>::State& s, const DecayArgs& a, const Walk& walk,
                                           const Part& d, int head, int chunks, float rate, unsigned base) {
    typedef Decay<T, W> D;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    float w[16];
    D::leaving(w, walk, rate, kChunk, half);
    const uint2 k_in = D::template column_place<true>(lane), v_in = D::template column_place<false>(lane);
    typename D::Fall fallen;
    const typename D::Rows k(walk.k, head, walk, d), v(walk.v, head, walk, d);
    auto issue = [&](int c, int buf) {
        const unsigned to = base + buf * 2 * D::kTile;
        k.load(to, c, kChunk, a.width);
        v.load(to + D::kTile, c, kChunk, a.width);
    };
    issue(0, 0);
    if (D::kBuffers > 2 && chunks > 1) issue(1, 1);
    int buf = 0;
    for (int c = 0; c < chunks; ++c) {
        if (D::kBuffers > 2 && c + 1 < chunks)
            load_wait<4>();
        else
            load_wait<0>();
        __syncthreads();
        if (c + D::kBuffers - 1 < chunks) issue(c + D::kBuffers - 1, buf == 0 ? D::kBuffers - 1 : buf - 1);
        const unsigned on = base + buf * 2 * D::kTile;
        typename D::vec8 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[i] = D::read_column(make_uint2(v_in.x + on + D::kTile, v_in.y + on + D::kTile), wave, i);
        const float by = fallen.pass(s, rate, kChunk, c + 1 == chunks);
        D::advance(s, make_uint2(k_in.x + on, k_in.y + on), x, w, by);
        buf = buf == D::kBuffers - 1 ? 0 : buf + 1;
    }
}

// What a segment adds to the state that enters it; nothing needs a document's last.
template <typename T, int W>
__global__ __launch_bounds__(2 * W, 2) void k_decay_sum(DecayArgs a) {
    typedef Decay<T, W> D;
    __shared__ __align__(1024) char lds[D::kBuffers * 2 * D::kTile];
    int head, role;
    const int row = block_of(a, &head, &role);
    const Part d = row_of(a, doc_of_row(a, row), row);
    if (d.none) return;
    const Walk& walk = a.walk[0];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    typename D::State s;
#pragma unroll
    for (int b = 0; b < D::kBlocks; ++b) s[b] = zero16();
    // whole chunks: a document goes on after it
    add_chunks<T, W>(s, a, walk, d, head, a.segment / kChunk, rate_of(a, head), lds_address(lds));
    D::store_state(s, walk.carry + ((long long)d.row * a.heads + head) * a.width * a.width, a.width,
                   32 * wave + (lane & 31), lane >> 5);
}

// The states after a document's segments but the last, over their sums: four elements of
// a state per thread, along the segments. Blocks go by documents or by the rows of carry,
// whichever are fewer (16 frames took 2% more by rows; 3,000 windows of 40, 8 heads of
// 64, 294 us, 387 with a block for every document and each of its segments).
__global__ __launch_bounds__(256) void k_decay_join(DecayArgs a, int slices, bool by_row) {
    unsigned id = a.first_block + blockIdx.x;
    const int slice = id % slices;
    id /= slices;
    const int head = id % a.heads;
    const int which = id / a.heads;
    const Part d = by_row ? row_of(a, doc_of_row(a, which), which) : row_of(a, which, -1);
    if (d.none || d.from > 0) return;  // one for each document
    const int parts = (d.n - 1) / a.segment;
    const int size = a.width * a.width, at = (slice * 256 + (int)threadIdx.x) * 4;
    if (at >= size) return;
    const long long pitch = (long long)a.heads * size;
    const Walk& walk = a.walk[0];
    float* sum = walk.carry + d.row * pitch + (long long)head * size + at;
    const float through = fall(rate_of(a, head), a.segment);
    float4 h = make_float4(0, 0, 0, 0);
    if (walk.state) {
        const float* from = walk.state + (long long)d.doc * pitch + (long long)head * size;
        h = *(const float4*)(from + at);
    }
    constexpr int kAhead = 16;
    for (int p = 0; p < parts; p += kAhead) {
        float4 x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) x[j] = *(const float4*)(sum + min(p + j, parts - 1) * pitch);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            h.x = __builtin_fmaf(through, h.x, x[j].x), h.y = __builtin_fmaf(through, h.y, x[j].y);
            h.z = __builtin_fmaf(through, h.z, x[j].z), h.w = __builtin_fmaf(through, h.w, x[j].w);
            if (p + j < parts) *(float4*)(sum + (p + j) * pitch) = h;
        }
    }
}

// A segment of a token or two, all in 32 bits: the block holds the state, four columns and
// kRows rows of it to a thread, and goes through the tokens. It is read and written once: 64
// sequences of 16 heads of 128, 134 MB, take 27 us (5.0 TB/s), 256 of them 106. A kernel of
// its own for a call of few tokens a document took 24, but 925 us for 255 steps next to one
// document of 257 tokens, token by token, where this takes 130.
constexpr int kFew = 2;

template <typename T, int W>
__device__ __forceinline__ void step_through(const DecayArgs& a, const Walk& walk, const Part& d, int head,
                                             const float* from, float* parts) {
    constexpr int kColumns = W / 4, kGroups = 8, kRows = W / kGroups, kPiece = kRows < 8 ? kRows : 8;
    static_assert(kColumns * kGroups == 2 * W, "a thread for each");
    const int c = (threadIdx.x % kColumns) * 4, group = threadIdx.x / kColumns, row = group * kRows;
    const bool on = c < a.width;
    const long long out_row = (long long)a.heads * a.width;
    const float through = fall(rate_of(a, head), 1);
    float4 s[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        s[j] = from && on && row + j < a.width ? *(const float4*)(from + (row + j) * a.width + c) : make_float4(0, 0, 0, 0);
    for (int at = d.from; at < d.to; ++at) {
        const long long token = walk.back ? d.lo + d.n - 1 - at : d.lo + at;
        const T* q = (const T*)walk.q.p + token * walk.q.st + head * walk.q.sh + row;
        const T* k = (const T*)walk.k.p + token * walk.k.st + (head / walk.k.group) * walk.k.sh + row;
        const T* v = (const T*)walk.v.p + token * walk.v.st + (head / walk.v.group) * walk.v.sh;
        float x[4] = {0, 0, 0, 0};
        if (on) Pack<T, 4>::load(v + c, x);
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int p = 0; p < kRows; p += kPiece) {
            float kr[kPiece], qr[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) kr[j] = qr[j] = 0.0f;
            if (row + p < a.width) Pack<T, kPiece>::load(k + p, kr), Pack<T, kPiece>::load(q + p, qr);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                float4& e = s[p + j];
                e.x = __builtin_fmaf(through, e.x, kr[j] * x[0]), e.y = __builtin_fmaf(through, e.y, kr[j] * x[1]);
                e.z = __builtin_fmaf(through, e.z, kr[j] * x[2]), e.w = __builtin_fmaf(through, e.w, kr[j] * x[3]);
                o.x = __builtin_fmaf(qr[j], e.x, o.x), o.y = __builtin_fmaf(qr[j], e.y, o.y);
                o.z = __builtin_fmaf(qr[j], e.z, o.z), o.w = __builtin_fmaf(qr[j], e.w, o.w);
            }
        }
        if (at > d.from) __syncthreads();
        *(float4*)(parts + group * W + c) = o;
        __syncthreads();
        if ((int)threadIdx.x < a.width) {
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) sum += parts[g * W + threadIdx.x];
            ((T*)walk.out)[token * out_row + head * a.width + threadIdx.x] = (T)(sum * walk.enter_by);
        }
    }
    if (!d.last || !walk.last || !on) return;
    float* to = walk.last + ((long long)d.doc * a.heads + head) * a.width * a.width;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        if (row + j < a.width) *(float4*)(to + (row + j) * a.width + c) = s[j];
}

// A segment from the state that enters it. ALONE: that is not in carry, and a block that does not
// begin with its document takes the state up to there first.
template <typename T, int W, bool ALONE>
__global__ __launch_bounds__(2 * W, W == 32 ? 3 : 2) void k_decay_run(DecayArgs a) {
    typedef Decay<T, W> D;
    __shared__ __align__(1024) char lds[D::kBuffers * 3 * D::kTile];
    int head, role;
    const int slot = block_of(a, &head, &role, ALONE && a.first_block == 0 ? a.more * a.heads * a.walks : 0);
    const Walk& walk = a.walk[role];
    const Part d = ALONE ? alone_part(a, slot) : find_part(a, slot);
    if (d.none) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, i = lane & 31;
    const long long out_row = (long long)a.heads * a.width;
    const bool out_wide = walk.out_wide;
    if (d.doc < 0) {  // tokens of no document
        for (int s = d.from; s < d.to; ++s)
            for (int c = threadIdx.x; c < a.width; c += D::NT) {
                const long long at = (d.lo + s) * out_row + head * a.width + c;
                if (out_wide)
                    ((float*)walk.out)[at] = 0.0f;
                else
                    ((T*)walk.out)[at] = (T)0.0f;
            }
        return;
    }
    const long long size = (long long)a.width * a.width;
    const float* from = d.from > 0 && !ALONE ? walk.carry + ((long long)(d.row - 1) * a.heads + head) * size
                        : walk.state             ? walk.state + ((long long)d.doc * a.heads + head) * size
                                                 : nullptr;
    const bool later = ALONE && d.from > 0;
    if (a.walks == 1 && d.to - d.from <= kFew && !later) {  // forward
        step_through<T, W>(a, walk, d, head, from, (float*)lds);
        return;
    }
    const int column = 32 * wave + i;
    const float rate = rate_of(a, head);
    const unsigned base = lds_address(lds);
    typename D::State s;
    bool some = from != nullptr;  // the state holds something
    if (later) {
        D::load_state(s, from, a.width, walk.turned, column, half);
        Part whole = d;
        whole.from = 0;
        add_chunks<T, W>(s, a, walk, whole, head, d.from / kChunk, rate, base);
        __syncthreads();  // all are done with the last tiles
        some = true;
    }
    const int chunks = (d.to - d.from + kChunk - 1) / kChunk;
    const typename D::Rows q_rows(walk.q, head, walk, d), k_rows(walk.k, head, walk, d), v_rows(walk.v, head, walk, d);
    auto issue = [&](int c, int buf) {
        const unsigned to = base + buf * 3 * D::kTile;
        const int left = d.to - d.from - c * kChunk;
        q_rows.load(to, c, left, a.width);
        k_rows.load(to + D::kTile, c, left, a.width);
        v_rows.load(to + 2 * D::kTile, c, left, a.width);
    };
    if (chunks > 0) issue(0, 0);
    if (D::kBuffers > 2 && chunks > 1) issue(1, 1);
    if (!later) D::load_state(s, from, a.width, walk.turned, column, half);
    // settled here: inside the loop their wait would be for the tiles under way as well
#pragma unroll
    for (int b = 0; b < D::kBlocks; ++b) asm volatile("" : "+v"(s[b]));

    float w[16], near[16];
    if (chunks > 1 || walk.last) D::leaving(w, walk, rate, kChunk, half);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int key = 16 * (r / 8) + 8 * half + r % 8;
        near[r] = fall(rate, max(0, i - key)) * walk.near_by;
    }
    const float entering = fall(rate, i + walk.lag) * walk.enter_by;
    typename D::Fall fallen;
    const unsigned q_in = D::row_place(i, half), k_in = D::row_place(D::traded(i), half);
    const uint2 kc_in = D::template column_place<true>(lane), vc_in = D::template column_place<false>(lane);

    uint4 made[2];  // the chunk before, rounded, not yet stored
    acc16 wide;
    auto store = [&](int c) {
        if (out_wide) {
            const int at = d.from + c * kChunk + i;
            if (at >= d.to) return;
            const long long token = walk.back ? d.lo + d.n - 1 - at : d.lo + at;
            const long long row = token * out_row + head * a.width;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = 32 * wave + 8 * q + 4 * half;
                if (col < a.width)
                    *(float4*)((float*)walk.out + row + col) =
                        make_float4(wide[4 * q], wide[4 * q + 1], wide[4 * q + 2], wide[4 * q + 3]);
            }
            return;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            int l = lane;
            if (ALONE && W == 32) asm volatile("" : "+v"(l));  // else one register is spilled around the loop
            const int at = d.from + c * kChunk + 16 * q + (l & 15), col = 32 * wave + 8 * quarter_piece(l);
            const long long token = walk.back ? d.lo + d.n - 1 - at : d.lo + at;
            if (at < d.to && col < a.width) *(uint4*)((T*)walk.out + token * out_row + head * a.width + col) = made[q];
        }
    };

    int buf = 0;
    for (int c = 0; c < chunks; ++c) {
        if (D::kBuffers > 2 && c + 1 < chunks)
            load_wait<6>();
        else
            load_wait<0>();
        __syncthreads();  // this chunk is there, and all are done with the one before
        if (c > 0) store(c - 1);
        if (c + D::kBuffers - 1 < chunks) issue(c + D::kBuffers - 1, buf == 0 ? D::kBuffers - 1 : buf - 1);
        const int m = min(kChunk, d.to - d.from - c * kChunk);
        const unsigned on = base + buf * 3 * D::kTile;
        const unsigned q_at = q_in + on, k_at = k_in + on + D::kTile;

        acc16 p = zero16(), o = zero16();
        float up_s = 1.0f;
        if (D::kHalf && some) {
            float top = 0.0f;
#pragma unroll
            for (int b = 0; b < D::kBlocks; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(s[b][r]));
            up_s = D::to_one(D::wave_max(top));
        }
#pragma unroll
        for (int k = 0; k < W / 16; ++k) {
            const typename D::vec8 q = D::read_row(q_at, k);
            p = Mma<T>::mul(D::read_row(k_at, k), q, p);
            typename D::vec8 x;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (T)(D::kHalf ? s[k / 2][8 * (k & 1) + j] * up_s : s[k / 2][8 * (k & 1) + j]);
            o = Mma<T>::mul(x, q, o);
        }
        float up_p = 1.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) p[r] = i >= 16 * (r / 8) + 8 * half + r % 8 ? p[r] * near[r] : 0.0f;
        if (D::kHalf) {
            float top = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(p[r]));
            // No further than 2^60: what is less is nothing in 16 bits, and the state's share is taken up as far.
            up_p = fminf(D::to_one(fmaxf(top, __shfl_xor(top, 32))), 0x1p60f);
#pragma unroll
            for (int r = 0; r < 16; ++r) p[r] *= up_p;
        }
        // Finite, so that what is zero stays so.
        float in = entering * fallen.now(rate);
        if (D::kHalf) in = fminf(fminf(in / up_s, kLargest) * up_p, kLargest);
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] *= in;
        typename D::vec8 v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[j] = D::read_column(make_uint2(vc_in.x + on + 2 * D::kTile, vc_in.y + on + 2 * D::kTile), wave, j);
            typename D::vec8 x, rest;
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = (T)p[8 * j + r], rest[r] = (T)(p[8 * j + r] - (float)x[r]);
            o = Mma<T>::mul(v[j], rest, o);
            o = Mma<T>::mul(v[j], x, o);
        }
        const float out_by = D::kHalf ? 1.0f / up_p : 1.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) wide[r] = o[r] * out_by;
        if (!out_wide) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                unsigned x0 = Mma<T>::pair(wide[8 * q], wide[8 * q + 1]), x1 = Mma<T>::pair(wide[8 * q + 2], wide[8 * q + 3]);
                unsigned y0 = Mma<T>::pair(wide[8 * q + 4], wide[8 * q + 5]), y1 = Mma<T>::pair(wide[8 * q + 6], wide[8 * q + 7]);
                trade_halves(x0, y0);
                trade_halves(x1, y1);
                made[q] = make_uint4(x0, x1, y0, y1);
            }
            trade_quarters(made[0], made[1]);
        }
        if (c + 1 < chunks || walk.last) {
            if (m < kChunk) D::leaving(w, walk, rate, m, half);
            some = true;
            const float by = fallen.pass(s, rate, m, c + 1 == chunks);
            D::advance(s, make_uint2(kc_in.x + on + D::kTile, kc_in.y + on + D::kTile), v, w, by);
        }
        buf = buf == D::kBuffers - 1 ? 0 : buf + 1;
    }
    if (chunks > 0) store(chunks - 1);
    if (d.last && walk.last) D::store_state(s, walk.last + ((long long)d.doc * a.heads + head) * size, a.width, column, half);
}

// Gradients of shared heads: the query heads' parts, in order, rounded. Of two tensors,
// the second's parts behind the first's.
template <typename T>
__global__ __launch_bounds__(256) void k_decay_share(const float* part, T* out0, T* out1, long long n, int group,
                                                     int width, unsigned first_block) {
    const long long i = (((long long)first_block + blockIdx.x) * 256 + threadIdx.x) * 8;
    if (i >= 2 * n) return;
    const long long at = i < n ? i : i - n;
    const float* from = part + (i < n ? 0 : n * group) + at / width * group * width + at % width;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int g = 0; g < group; ++g) {
        float x[8];
        Pack<float, 8>::load(from + (long long)g * width, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += x[j];
    }
    Pack<T, 8>::store((i < n ? out0 : out1) + at, s);
}

// ---- host --------------------------------------------------------------------

long long round256(long long n) { return (n + 255) / 256 * 256; }
int padded(int width) { return width <= 32 ? 32 : width <= 64 ? 64 : 128; }

// 16-byte pieces; a chunk's rows lie within 2^32 bytes.
bool stride_ok(const int64_t s[2]) {
    return s[0] % 8 == 0 && s[1] % 8 == 0 && s[0] >= 0 && s[1] >= 0 && s[0] < 1ll << 25;
}

bool check(const tok_decay* t) {
    if (!t || (t->dtype != TOK_BF16 && t->dtype != TOK_F16)) return false;
    if (t->heads < 1 || t->kv_heads < 1 || t->heads % t->kv_heads || t->heads > 65536) return false;
    if (t->width < 8 || t->width > 128 || t->width % 8) return false;
    if (t->t < 0 || t->t > kMaxElems || t->t * t->heads > kMaxElems) return false;
    if (t->docs < 1 || t->docs > kMaxDocs || (t->docs + 2ll) * t->heads > (1ll << 30)) return false;
    if ((t->reverse != 0 && t->reverse != 1) || t->reserved || (!t->offsets && t->docs != 1) || !t->decay) return false;
    if (!(t->scale >= 1e-30f) || !(t->scale <= 1e30f)) return false;
    return stride_ok(t->q_stride) && stride_ok(t->k_stride) && stride_ok(t->v_stride);
}

// Short documents that fill the card with one block each (and head), or steps of decoding: no
// states kept and one launch, not three (546 of 30 tokens, 8 heads of 32: 13 us for 18; 256 steps
// of 16 heads of 128: 25 for 35). The host knows no lengths, and one document may hold nearly all
// tokens. Its segments of kAlone tokens go to blocks of their own there, of which each takes the
// state up to where it begins first, at a third of the walk's time a token. Forward of a prompt next
// to as many steps as it has tokens, 8 heads (in one launch; in three; with a block a document):
// 2,048 of 64 56, 74 and 142 us, 2,048 of 128 120, 163 and 224, 8,192 of 32 176, 108 and 390.
// Among fewer short ones it costs most: 8,000 tokens next to 400 of 20, 8 heads of 32: 175, 40 and 336.
// It ends at 16,384 tokens of width 32 and fewer of wider ones.
bool by_doc(const tok_decay& t) {
    return t.t <= 16384 * 32 / padded(t.width) &&
           (t.t <= 2ll * t.docs || (t.t <= 64ll * t.docs && (long long)t.docs * t.heads >= 512));
}

// Tokens of a segment: as many as leave a block for every place the card has (two blocks of
// four wavefronts a CU, and as many more as they have fewer) and none for a second round,
// counting the segments that documents' ends and the tokens of none may add; every
// segment passes memory with its state four times. 122,880 tokens of 8 heads of 128: 536
// blocks take 320 us, 504 take 240. Many documents end within a segment each and leave blocks
// short, which twice as many segments even out. They are taken where two rounds of them end before
// one of the others by a fiftieth, a block's beginning and state counted as 3/4 of the width in tokens,
// and a segment as no longer than a document. (Forward of 8 heads of 64, once and twice: 136,000 tokens in
// 4 documents 215 us and 220, in 12 227 and 217, in 24 240 and 223, in 64 272 and 219, in 128, no
// longer than one segment each, 164 and 209; 34,000 tokens in 16 documents 59 and 67, in 64 76 and
// 69; 2 heads, 136,000 in 16 58 and 69, in 256 76 and 68.) Few narrow heads would have many segments
// of 128 tokens, which their states are joined along one after the other: at least so many
// tokens that the join and a segment's chunks take about as long (100,000 tokens of 2 heads of
// 32: 59 us, 114 without).
int segment_of(const tok_decay& t) {
    if (by_doc(t)) return (int)((t.t + 127) / 128 * 128) + 128;  // one
    const long long each = 512ll * 128 / padded(t.width) / t.heads;  // blocks of a head
    auto length = [&](long long blocks) {
        long long n = blocks - t.docs - 2;
        if (n < blocks / 2) n = blocks / 2;
        if (n < 1) n = 1;
        n = (t.t + n - 1) / n;
        return (n + kChunk - 1) / kChunk * kChunk;
    };
    const long long doc = (t.t + t.docs - 1) / t.docs, more = 3 * padded(t.width) / 4;
    auto takes = [&](long long n) { return (n < doc ? n : doc) + more; };
    long long n = length(each);
    const long long half = length(2 * each);
    if (2 * 50 * takes(half) < 49 * takes(n)) n = half;
    while (n * n < 2 * (t.t / t.docs)) n += kChunk;
    if (n < 128) n = 128;
    if (n > 65536) n = 65536;
    return (int)n;
}
// No document can have a second segment.
bool whole(const tok_decay& t) { return t.t <= segment_of(t); }

long long slots(const tok_decay& t) { return t.t / segment_of(t) + t.docs + 2; }
long long state_elems(const tok_decay& t) { return (long long)t.heads * t.width * t.width; }

Place place(const void* p, const int64_t s[2], int group) { return {p, s[0], s[1], group}; }

DecayArgs make_args(const tok_decay& t) {
    DecayArgs a = {};
    a.offsets = t.offsets, a.decay = t.decay;
    a.t = (int)t.t, a.docs = t.docs, a.heads = t.heads, a.width = t.width;
    a.segment = segment_of(t);
    a.segments = (int)slots(t);
    a.walks = 1;
    a.walk[0].back = t.reverse, a.walk[0].lag = 1;
    a.walk[0].near_by = a.walk[0].enter_by = t.scale, a.walk[0].leave_by = 1.0f;
    return a;
}

template <typename Launch>
void in_launches(long long blocks, int threads, Launch launch) {
    const long long most = most_blocks(threads) / 8 * 8;
    for (long long b = 0; b < blocks; b += most)
        launch((unsigned)b, dim3((unsigned)(blocks - b < most ? blocks - b : most)));
}

// The states that enter the segments of walk 0.
template <typename T, int W>
void states(DecayArgs a, hipStream_t stream) {
    a.walks = 1;
    const long long rows = a.t / a.segment;
    in_launches(rows * a.heads, 2 * W, [&](unsigned first, dim3 grid) {
        a.first_block = first;
        k_decay_sum<T, W><<<grid, dim3(2 * W), 0, stream>>>(a);
    });
    const int slices = (a.width * a.width + 1023) / 1024;
    const bool by_row = rows < a.docs;
    in_launches((by_row ? rows : a.docs) * a.heads * slices, 256, [&](unsigned first, dim3 grid) {
        a.first_block = first;
        k_decay_join<<<grid, dim3(256), 0, stream>>>(a, slices, by_row);
    });
}

template <typename T, int W>
void run(const tok_decay& t, DecayArgs a, hipStream_t stream) {
    const bool alone = by_doc(t);
    if (alone) a.segment = kAlone, a.more = a.t / kAlone, a.segments = t.docs + 2 + a.more;
    in_launches((long long)a.segments * a.heads * a.walks, 2 * W, [&](unsigned first, dim3 grid) {
        a.first_block = first;
        if (alone)
            k_decay_run<T, W, true><<<grid, dim3(2 * W), 0, stream>>>(a);
        else
            k_decay_run<T, W, false><<<grid, dim3(2 * W), 0, stream>>>(a);
    });
}

template <typename T, int W>
int forward(const tok_decay& t, DecayArgs a, hipStream_t stream) {
    if (!whole(t)) states<T, W>(a, stream);
    run<T, W>(t, a, stream);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

struct Gradients {
    Place q, k, v, g;
    const float *state, *grad_last;
    float *carry, *back_carry, *part;  // part: float32 gradients by query head, or null
    void *gq, *gk, *gv;
    float* grad_state;
    int group;
};

template <typename T, int W>
int backward(const tok_decay& t, DecayArgs a, const Gradients& g, hipStream_t stream) {
    const long long n = (long long)a.t * (a.heads / g.group) * a.width;
    // grad_v and the state's gradient, from the other end
    Walk& v = a.walk[0];
    Walk& q = a.walk[2];
    q = v;
    v.back = !v.back, v.lag = 0, v.leave_by = v.enter_by, v.enter_by = 1.0f;
    v.q = g.k, v.k = g.q, v.v = g.g, v.state = g.grad_last, v.carry = g.back_carry, v.last = g.grad_state;
    v.out = g.part ? (void*)g.part : g.gv, v.out_wide = g.part != nullptr;
    if (!whole(t)) states<T, W>(a, stream);
    // grad_k along the same states
    Walk& k = a.walk[1];
    k = v;
    k.q = g.v, k.k = g.g, k.v = g.q, k.turned = 1, k.last = nullptr;
    k.out = g.part ? (void*)(g.part + n * g.group) : g.gk;
    // grad_q: grad against v and k, along the forward's
    q.q = g.g, q.k = g.v, q.v = g.k, q.out = g.gq, q.state = g.state, q.carry = g.carry, q.turned = 1;
    a.walks = 3;
    run<T, W>(t, a, stream);
    if (g.part)
        in_launches((2 * n + 2047) / 2048, 256, [&](unsigned first, dim3 grid) {
            k_decay_share<T><<<grid, dim3(256), 0, stream>>>(g.part, (T*)g.gv, (T*)g.gk, n, g.group, a.width, first);
        });
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

template <typename T, typename F>
int by_width(int width, F f) {
    if (width <= 32) return f(std::integral_constant<int, 32>());
    if (width <= 64) return f(std::integral_constant<int, 64>());
    return f(std::integral_constant<int, 128>());
}

bool aligned16(const void* p) { return ((size_t)p & 15) == 0; }

long long carry_rows(const tok_decay& t) { return whole(t) ? 0 : t.t / segment_of(t); }
long long carry_elems(const tok_decay& t) { return carry_rows(t) * state_elems(t); }
long long part_elems(const tok_decay& t) { return t.heads == t.kv_heads ? 0 : 2 * t.t * t.heads * t.width; }

}  // namespace

extern "C" {

int64_t tok_decay_carry_rows(const tok_decay* t) {
    if (!check(t)) return VOX_EINVAL;
    return carry_rows(*t);
}

int64_t tok_decay_grad_workspace_bytes(const tok_decay* t) {
    if (!check(t)) return VOX_EINVAL;
    return round256(carry_elems(*t) * 4) + round256(part_elems(*t) * 4);
}

int tok_decay_attend(const tok_decay* t, const void* q, const void* k, const void* v, const float* state, void* out,
                     float* last_state, float* carry, hipStream_t stream) {
    if (!check(t)) return VOX_EINVAL;
    if (t->t && (!q || !k || !v || !out)) return VOX_EINVAL;
    if (!whole(*t) && !carry) return VOX_EINVAL;
    const void* all[] = {q, k, v, out, state, last_state, carry};
    for (const void* p : all)
        if (!aligned16(p)) return VOX_EINVAL;
    DecayArgs a = make_args(*t);
    const int group = t->heads / t->kv_heads;
    Walk& w = a.walk[0];
    w.q = place(q, t->q_stride, 1), w.k = place(k, t->k_stride, group), w.v = place(v, t->v_stride, group);
    w.state = state, w.out = out, w.last = last_state, w.carry = carry;
    return by_width<void>(t->width, [&](auto w) {
        return t->dtype == TOK_BF16 ? forward<bf16_t, decltype(w)::value>(*t, a, stream)
                                    : forward<f16_t, decltype(w)::value>(*t, a, stream);
    });
}

int tok_decay_attend_grad(const tok_decay* t, const void* q, const void* k, const void* v, const void* grad_out,
                          const float* state, const float* carry, const float* grad_last, void* grad_q, void* grad_k,
                          void* grad_v, float* grad_state, void* workspace, int64_t workspace_bytes,
                          hipStream_t stream) {
    if (!check(t) || !stride_ok(t->g_stride)) return VOX_EINVAL;
    if (t->t && (!q || !k || !v || !grad_out || !grad_q || !grad_k || !grad_v)) return VOX_EINVAL;
    if (!whole(*t) && !carry) return VOX_EINVAL;
    const void* all[] = {q, k, v, grad_out, state, carry, grad_last, grad_q, grad_k, grad_v, grad_state};
    for (const void* p : all)
        if (!aligned16(p)) return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, tok_decay_grad_workspace_bytes(t))) return VOX_EWORKSPACE;
    const DecayArgs a = make_args(*t);
    const int group = t->heads / t->kv_heads;
    Gradients g = {};
    g.q = place(q, t->q_stride, 1), g.k = place(k, t->k_stride, group), g.v = place(v, t->v_stride, group);
    g.g = place(grad_out, t->g_stride, 1);
    g.state = state, g.grad_last = grad_last, g.carry = const_cast<float*>(carry);
    g.back_carry = (float*)workspace;
    g.part = group > 1 ? (float*)((char*)workspace + round256(carry_elems(*t) * 4)) : nullptr;
    g.gq = grad_q, g.gk = grad_k, g.gv = grad_v, g.grad_state = grad_state, g.group = group;
    return by_width<void>(t->width, [&](auto w) {
        return t->dtype == TOK_BF16 ? backward<bf16_t, decltype(w)::value>(*t, a, g, stream)
                                    : backward<f16_t, decltype(w)::value>(*t, a, g, stream);
    });
}

}  // extern "C"
