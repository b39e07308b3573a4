// The loss over a table's rows (tokens.h): softmax cross entropy of tokens against
// every row, and its gradients, without the logits in memory.
//
// Products. Logits z = scale X W^T are taken as W X^T, so that a lane holds one
// token's logits of many rows: the running maximum and sum stay in the lane. The
// backward takes the logits again, a piece of the rows at a time, and writes
// dZ = (exp(z - lse) - [row is the token's]) grad, rounded, to the workspace, from
// where two products follow: grad_x += dZ W and grad_table = dZ^T X. A piece is as
// many rows as dZ of 256 MB holds, about what the cache between HBM and the XCDs does
// (a training step of 4,096 tokens of 512 by 214,272 rows: a tenth more with pieces of 128 MB,
// whose partial sums of grad_x pass memory twice as often, 3% less with 2 GB). Where 256 rows of all
// tokens are more than that, tokens go by bands.
//
// Tiles of 32 of the inner index go straight from memory into three buffers of LDS
// in turn. X and dZ are kept in pieces of 8 elements, [element / 8][token]: a tile
// is then a few runs of memory, its rows and its columns are both read without
// conflicts, tokens without a row and tokens past the last are zeros, and no
// product asks for either. Tokens of up to 128 elements stay in registers while the rows go
// by, and forward come from x itself.
//
// Bounds. 4,096 tokens of 512 by 214,272 rows take 3.8 ms, of which the forward's logits
// 0.95 (947 TFLOP/s, matrix units busy 47%), dZ in seven pieces 1.23 (733, 33%), the two
// gradients' products 1.60 (1,124, 57%); a library product of 8192 cubed reaches 1,185 to
// 1,290. Two wavefronts a SIMD wait for LDS and barriers; in the logits' passes the
// exponentials come on top, an exp2 and two more instructions a logit forward, three, the
// rounding and 250 MB of stores a piece backward, between the products of a CU's other blocks.
// A frame of 12,000 tokens of 128 by as many rows, forward: 0.65 ms (1,010 TFLOP/s, 47%). A
// few tokens are bound by memory: 110 MB in 22 us.
//
// Roundings. dZ enters the products in the tensors' type; logits, maxima, sums and
// gradients are summed in 32 bits. A token's gradient is nearly one dZ's multiple of its
// row, and shows its rounding: of many tokens that is one rounding more of random sign
// beside the result's own, of a few it may be twice as much. Up to kTwice tokens
// therefore go through the backward twice, the second time with what the rounding of dZ
// left: next to nothing while both fit the tile of 128 (64 tokens of 512 by 214,272 rows 230
// us), a third at 256 (428 us, 327 for 257 tokens). In fp16 dZ is taken 2^14 times the ratio
// of its token's grad to the largest one's power of two: it keeps all its bits down to
// 2^-28 of that.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "mma_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr long long kMaxTokens = 1ll << 25;  // a wavefront for each, in one launch
constexpr long long kMaxRows = (1ll << 31) - 2048;
constexpr long long kMaxWidth = 65536;
constexpr long long kMaxStride = 1ll << 22;  // 256 rows apart in 32 bits of bytes
constexpr int kTokenPad = 128;               // tokens are laid out in whole tiles
constexpr int kRowTile = 256;                // rows of a tile of logits
constexpr int kStep = 32;                    // inner elements of a stage
constexpr long long kPieceBytes = 256ll << 20;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e+38f;
constexpr int kTwice = 256;
constexpr int kBand = 8;  // tiles of tokens
constexpr int kLift = 14;  // fp16: dZ is 2^kLift too large

struct LossArgs {
    const void* x;
    const void* table;
    const void* ids;
    const float* grad;
    const float* lse;
    float* loss;
    float* lse_out;
    void* gx;
    void* gt;
    // workspace
    uint4* xg;         // [width8, x_pad]: X in pieces
    uint4* dz;         // [piece / 8, t_pad]
    int* came;         // [x_pad]: the token's row, or -1
    float* shift;      // [x_pad]: lse in base 2 (backward)
    float* by;         // [x_pad]: grad times the lift (backward)
    float* hit;        // [x_pad]: the logit of the token's row, base 2 (forward)
    float2* part;      // [splits, x_pad]: maximum and sum (forward)
    float* top;        // [tops]: the largest |grad| of each share of the tokens (fp16)
    float* part_x;     // [x_splits, tokens, width]
    float* part_t;     // [bands, t_splits, piece rows, width], or null: grad_table's blocks round themselves
    long long x_stride, t_stride;
    int t, rows, width, width8, id_bytes;
    int x_pad, t_pad;  // tokens laid out, all of them and those of a band
    int t_all;         // t, or twice as much: tokens of the backward
    int x_tokens;      // t of all bands
    int splits, tiles;        // of the rows' tiles
    int token_tiles;
    int row0, piece;          // rows of a piece: a multiple of kRowTile, its last ones past the table's
    int x_splits, t_splits, first;
    int tokens_in;            // tokens that dZ is written for
    int tops;
    float scale, scale2;
};

// A tile's stage by stage products. Blocks of 32: MA x NB per wavefront, WM x WN
// wavefronts.
template <typename T, int MA_, int NB_, int WM_, int WN_>
struct Shape {
    static constexpr int kWidth = 0;  // the width goes by in stages
    static constexpr bool kOnce = NB_ == 1;  // a block's tokens are read from memory about once
    static constexpr int MA = MA_, NB = NB_, WM = WM_, WN = WN_;
    static constexpr int BM = 32 * MA * WM, BN = 32 * NB * WN, NT = 64 * WM * WN;
    static constexpr int kA = BM * kStep * 2, kB = BN * kStep * 2;  // bytes of a stage
    static constexpr int kStage = kA + kB;
    static constexpr int kALoads = BM * 4 / NT, kBLoads = (BN * 4 + NT - 1) / NT;
    static constexpr int kLoads = kALoads + BN * 4 / NT;  // every wavefront's, at least
};

// Tiles of logits of narrow tokens: a wavefront keeps its 64 tokens' whole width (W at most)
// in registers, and a stage is a tile: BM rows of all their width.
template <typename T, int W>
struct Narrow {
    static constexpr bool kOnce = true;
    static constexpr int kWidth = W, MA = W == 128 ? 1 : 2, NB = 2, WM = 2, WN = 2;
    static constexpr int BM = 32 * MA * WM, BN = 32 * NB * WN, NT = 64 * WM * WN;
    static constexpr int kStage = BM * W * 2, kLoads = BM * (W / 8) / NT;
};

// The stages of a block: loads run two ahead of the products. Memory operations of a
// wavefront end in the order they were issued, so a stage is there when no more are
// under way than were issued after its loads: the next stage's, and the stores of a
// tile that ended with the stage before, or the one before that. compute() says how
// many those are (0, or STORES). begin() is what else there is to load, under way with the
// first stages.
template <int LOADS, int STORES, typename Begin, typename Issue, typename Compute>
__device__ __forceinline__ void stages(int total, Begin begin, Issue issue, Compute compute) {
    if (total > 0) issue(0, 0);
    if (total > 1) issue(1, 1);
    begin();
    int buf = 0, since = 2;
    // The loop's place in 64 bytes of code does not change with what comes before it (4,096 tokens of
    // 512 by 214,272 rows, gradients: 2,832 us, 2,815 to 2,875 without).
    asm volatile(".p2align 6");
    for (int i = 0; i < total; ++i) {
        if (i + 1 == total)
            load_wait<0>();
        else if (STORES && since < 2)
            load_wait<LOADS + STORES>();
        else
            load_wait<LOADS>();
        __syncthreads();  // this stage is there, and all are done with the one before
        ++since;
        // compute() starts the loads when its first reads of LDS are under way
        const bool stored = compute(i, buf, [&] {
            if (i + 2 < total) issue(i + 2, buf == 0 ? 2 : buf - 1);
        });
        if (stored) since = 0;
        buf = buf == 2 ? 0 : buf + 1;
    }
}

// Both steps of a stage: what is read, then multiplied. EAGER: all is read before the first
// product, for which an epilogue that keeps its own numbers leaves no registers at the
// widest shape (reads of spilled ones would wait for the loads under way).
template <typename T, typename S, bool EAGER, typename ReadA, typename ReadB, typename Next>
__device__ __forceinline__ void products(acc16 (&acc)[S::MA][S::NB], ReadA read_a, ReadB read_b, Next next) {
    typename Mma<T>::vec8 x[2][S::MA], y[2][S::NB];
    auto read = [&](int s) {
#pragma unroll
        for (int j = 0; j < S::NB; ++j) y[s][j] = read_b(j, s);
#pragma unroll
        for (int i = 0; i < S::MA; ++i) x[s][i] = read_a(i, s);
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int i = 0; i < S::MA; ++i)
#pragma unroll
            for (int j = 0; j < S::NB; ++j) acc[i][j] = Mma<T>::mul(x[s][i], y[s][j], acc[i][j]);
    };
    read(0);
    next();
    if (EAGER) {
        read(1);
        fence();
    }
    multiply(0);
    if (!EAGER) read(1);
    multiply(1);
}

// ---- operands ----------------------------------------------------------------
//
// load() brings a stage to LDS; what of an address is a lane's own is computed once, in
// 32 bits.

// Rows of a matrix in memory, the inner index along a row. In LDS 64 bytes a row,
// its four pieces permuted by XOR with (row >> 2) & 3: 16 rows' pieces of one place
// touch every bank once.
template <typename T, int ROWS, int NT>
struct RowsOfMatrix {
    const T* base;
    long long stride;
    int rows, width;
    unsigned offset;

    __device__ __forceinline__ RowsOfMatrix(const void* p, long long st, int n, int w)
        : base((const T*)p), stride(st), rows(n), width(w) {
        const int row = threadIdx.x >> 2;
        offset = (unsigned)row * (unsigned)(2 * st) + 16u * ((threadIdx.x & 3) ^ ((row >> 2) & 3));
    }
    __device__ __forceinline__ void load(unsigned to, int row0, int k0) const {
        constexpr int kPer = (ROWS * 4 + NT - 1) / NT;
        static_assert(NT / 4 % 16 == 0, "the permutation is that of the first load's rows");
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (ROWS * 4 < NT && wave * 64 >= ROWS * 4) return;
        const T* from = base + row0 * stride + k0;
        if (row0 + ROWS <= rows && k0 + kStep <= width) {
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                load_to_lds(to + 1024u * wave + 16u * NT * p, from + p * (NT / 4) * stride, offset);
            return;
        }
        const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) ^ ((r >> 2) & 3);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int row = p * (NT / 4) + r;
            const bool there = row0 + row < rows && k0 + 8 * c < width;
            load_to_lds(to + 1024u * wave + 16u * NT * p, there ? (const void*)(from + row * stride + 8 * c) : &kNothing);
        }
    }
    static __device__ __forceinline__ unsigned place(int row, int half) {
        return row * 64 + ((half ^ ((row >> 2) & 3)) << 4);
    }
    // at: tile + place of row lane % 32; 32 rows on per block, step s of the stage
    static __device__ __forceinline__ auto read(unsigned at, int block, int s) {
        return lds_read<typename Mma<T>::vec8>((at ^ (s << 5)) + block * 2048);
    }
};

// Whole rows of a matrix of W columns at most, zeros past its width. In LDS 2 W bytes a row,
// its pieces permuted so that 16 rows' pieces of one place touch every bank once.
template <typename T, int W, int ROWS, int NT>
struct WholeRows {
    static constexpr int kPieces = W / 8;
    const T* base;
    long long stride;
    int rows, width;
    unsigned offset;

    static __device__ __forceinline__ int swz(int row) {
        if (W == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
        if (W == 64) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
        return (row >> 2) & 3;
    }
    __device__ __forceinline__ WholeRows(const void* p, long long st, int n, int w)
        : base((const T*)p), stride(st), rows(n), width(w) {
        const int row = threadIdx.x / kPieces;
        offset = (unsigned)row * (unsigned)(2 * st) + 16u * ((threadIdx.x % kPieces) ^ swz(row));
    }
    __device__ __forceinline__ void load(unsigned to, int row0) const {
        constexpr int kPer = ROWS * kPieces / NT;
        static_assert(NT / kPieces % 16 == 0, "the permutation is that of the first load's rows");
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const T* from = base + row0 * stride;
        if (row0 + ROWS <= rows && width == W) {
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                load_to_lds(to + 1024u * wave + 16u * NT * p, from + p * (NT / kPieces) * stride, offset);
            return;
        }
        const int r = threadIdx.x / kPieces, c = (threadIdx.x % kPieces) ^ swz(r);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int row = p * (NT / kPieces) + r;
            const bool there = row0 + row < rows && 8 * c < width;
            load_to_lds(to + 1024u * wave + 16u * NT * p, there ? (const void*)(from + row * stride + 8 * c) : &kNothing);
        }
    }
    static __device__ __forceinline__ unsigned place(int row, int half) {
        return row * 2 * W + ((half ^ swz(row)) << 4);
    }
    static __device__ __forceinline__ auto read(unsigned at, int block, int s) {
        return lds_read<typename Mma<T>::vec8>((at ^ (s << 5)) + block * 64 * W);
    }
};

// Rows of a matrix kept in pieces, [inner / 8][row]. In LDS [4][ROWS] pieces.
template <typename T, int ROWS, int NT>
struct RowsOfPieces {
    const uint4* base;
    long long pitch;
    unsigned offset;

    __device__ __forceinline__ RowsOfPieces(const uint4* p, long long step) : base(p), pitch(step) {
        offset = ((threadIdx.x / ROWS) * (unsigned)step + threadIdx.x % ROWS) * 16u;
    }
    __device__ __forceinline__ void load(unsigned to, int row0, int k0) const {
        constexpr int kPer = (ROWS * 4 + NT - 1) / NT;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint4* from = base + (k0 >> 3) * pitch + row0;
#pragma unroll
        for (int p = 0; p < kPer; ++p)
            if (p * NT + wave * 64 < ROWS * 4)
                load_to_lds(to + 1024u * wave + 16u * NT * p, from + p * (NT / ROWS) * pitch, offset);
    }
    static __device__ __forceinline__ unsigned place(int row, int half) { return (half * ROWS + row) * 16; }
    static __device__ __forceinline__ auto read(unsigned at, int block, int s) {
        return lds_read<typename Mma<T>::vec8>(at + s * (ROWS * 32) + block * 512);
    }
};

// Columns of a matrix in memory whose rows are the inner index. In LDS COLS / 128
// tiles of 32 rows of 256 bytes, the 16 pieces of a row permuted by XOR with a
// number of the row that puts four rows of 64 bytes on all banks.
template <typename T, int COLS, int NT>
struct ColumnsOfMatrix {
    const T* base;
    long long stride;
    int rows, left;   // columns from the first on
    unsigned offset;

    static __device__ __forceinline__ int swz(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }
    __device__ __forceinline__ ColumnsOfMatrix(const void* p, long long st, int n, int col0, int width)
        : base((const T*)p + col0), stride(st), rows(n), left(width - col0) {
        const int row = threadIdx.x >> 4;
        offset = (unsigned)row * (unsigned)(2 * st) + 16u * ((threadIdx.x & 15) ^ swz(row));
    }
    __device__ __forceinline__ void load(unsigned to, int row0) const {
        constexpr int kPer = COLS * 4 / NT;
        static_assert(NT == 256, "16 rows of 128 columns a load");
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const T* from = base + row0 * stride;
        if (row0 + kStep <= rows && left >= COLS) {
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                load_to_lds(to + 1024u * wave + 16u * NT * p, from + (p & 1) * 16 * stride + (p >> 1) * 128, offset);
            return;
        }
        const int r = threadIdx.x >> 4, c = (threadIdx.x & 15) ^ swz(r);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int row = (p & 1) * 16 + r, col = 8 * c + (p >> 1) * 128;
            const bool there = row0 + row < rows && col < left;
            load_to_lds(to + 1024u * wave + 16u * NT * p, there ? (const void*)(from + row * stride + col) : &kNothing);
        }
    }
    // Where the first four of a lane's eight inner rows are (first step, block 0 of a
    // tile of 128), and the others.
    static __device__ __forceinline__ uint2 place(int lane) {
        const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
        const int c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), in = (lane & 1) << 3;
        return make_uint2(row * 256 + ((c ^ swz(row)) << 4) + in, (row + 4) * 256 + ((c ^ swz(row + 4)) << 4) + in);
    }
    static __device__ __forceinline__ auto read(uint2 at, int block, int s) {
        const unsigned on = s * 4096 + (block >> 2) * 8192, flip = (block & 3) << 6;
        return lds_read_columns<typename Mma<T>::vec8>((at.x ^ flip) + on, (at.y ^ flip) + on);
    }
};

// The same of a matrix kept in pieces, [column / 8][inner]. In LDS [COLS / 8][32]
// pieces, the 32 of a column group permuted by XOR with 4 (group % 4). Of a last group before COLS / 8
// the last one is read in place of those past it.
template <typename T, int COLS, int NT, bool LAST = false>
struct ColumnsOfPieces {
    static constexpr int kPer = COLS * 4 / NT, kGroups = NT / 32;
    const uint4* base;
    long long pitch;
    int last;
    unsigned offset[LAST ? kPer : 1];

    __device__ __forceinline__ ColumnsOfPieces(const uint4* p, long long step, int col0, int groups = 0)
        : base(p + (long long)(col0 >> 3) * step), pitch(step), last(groups - 1 - (col0 >> 3)) {
        static_assert(kGroups % 4 == 0, "the permutation is that of the first load's groups");
        const int group = threadIdx.x >> 5, row = (threadIdx.x & 31) ^ ((group & 3) << 2);
#pragma unroll
        for (int l = 0; l < (LAST ? kPer : 1); ++l)
            offset[l] = ((LAST ? min(group, last - first(l)) : group) * (unsigned)step + row) * 16u;
    }
    // The first group of load l.
    __device__ __forceinline__ int first(int l) const { return LAST && last < l * kGroups ? 0 : l * kGroups; }
    __device__ __forceinline__ void load(unsigned to, int row0) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int l = 0; l < kPer; ++l)
            load_to_lds(to + 1024u * wave + 16u * NT * l, base + row0 + first(l) * pitch, offset[LAST ? l : 0]);
    }
    static __device__ __forceinline__ uint2 place(int lane) {
        const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
        const int c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), in = (lane & 1) << 3;
        return make_uint2(c * 512 + ((row ^ (c << 2)) << 4) + in, c * 512 + (((row + 4) ^ (c << 2)) << 4) + in);
    }
    static __device__ __forceinline__ auto read(uint2 at, int block, int s) {
        return lds_read_columns<typename Mma<T>::vec8>((at.x ^ (s << 8)) + block * 2048,
                                                       (at.y ^ (s << 8)) + block * 2048);
    }
};

// ---- tokens in pieces --------------------------------------------------------

__device__ __forceinline__ int id_of(const LossArgs& a, int t) {
    const long long id = a.id_bytes == 4 ? ((const int*)a.ids)[t] : ((const long long*)a.ids)[t];
    return id >= 0 && id < a.rows ? (int)id : -1;
}

// The largest |grad| of tokens that have a row, for fp16, over each block's share; what is
// not finite is left out.
constexpr int kTops = 64;
__global__ __launch_bounds__(1024) void k_loss_top(LossArgs a) {
    __shared__ float tops[16];
    float top = 0.0f;
    for (int t = blockIdx.x * 1024 + threadIdx.x; t < a.t; t += 1024 * gridDim.x) {
        const float g = id_of(a, t) >= 0 ? fabsf(a.grad[t]) : 0.0f;
        top = g <= 3.402823466e+38f ? fmaxf(top, g) : top;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) top = fmaxf(top, tops[w]);
        a.top[blockIdx.x] = top;
    }
}

// The exponent dZ is taken up by.
template <typename T>
__device__ __forceinline__ int lift_of(const LossArgs& a) {
    if (sizeof(T) == 2 && __is_same(T, bf16_t)) return 0;
    float top = 0.0f;
    for (int b = 0; b < a.tops; ++b) top = fmaxf(top, a.top[b]);
    return top > 0.0f ? kLift - __builtin_amdgcn_frexp_expf(top) : 0;
}
// What sums of lifted weights are multiplied with: finite, so that zeros stay so (where it would not
// be, the smallest such sum passes fp16's largest number).
template <typename T>
__device__ __forceinline__ float down_of(const LossArgs& a) {
    return fminf(ldexpf(a.scale, -lift_of<T>(a)), -kLowest);
}

// X as pieces, zeros where a token has no row, is past the last, or past the width.
template <typename T, bool GRAD>
__global__ __launch_bounds__(256) void k_loss_pack(LossArgs a) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(i & 7) + 8 * blockIdx.y, t = (int)(i >> 3);
    if (t >= a.x_pad) return;
    const int from = t < a.t ? t : t - a.t;  // of the second time
    const int id = t < (GRAD ? a.t_all : a.t) ? id_of(a, from) : -1;
    if (c < a.width8) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (id >= 0 && 8 * c < a.width) v = *(const uint4*)((const T*)a.x + from * a.x_stride + 8 * c);
        a.xg[(long long)c * a.x_pad + t] = v;
    }
    if (GRAD && c == 0) {
        a.came[t] = id;
        a.shift[t] = id >= 0 ? a.lse[from] * kLog2e : 0.0f;
        a.by[t] = id >= 0 ? ldexpf(a.grad[from], lift_of<T>(a)) : 0.0f;
    }
}

// ---- logits ------------------------------------------------------------------

// The share of the rows and the tile of tokens of a block. Blocks that run together on an XCD
// are of a few tiles of tokens and a few shares: both stay in its L2 (20,000 tokens of 512 by
// 214,272 rows forward: 4,660 us, 6,140 with all tiles of tokens before the next share). Where tokens
// stay in registers all read one share's rows.
template <typename S>
__device__ __forceinline__ void place_of(const LossArgs& a, int* split, int* token0) {
    const int id = xcd_block(blockIdx.x, gridDim.x);
    const int most = S::kWidth ? a.token_tiles : kBand;
    const int first = id / (most * a.splits) * most, in = id % (most * a.splits);
    const int here = min(most, a.token_tiles - first);
    *split = in / here;
    *token0 = (first + in % here) * S::BN;
}

// Tiles [t0, t1) of the rows against a tile of tokens, from `first_row` on;
// done(tile, acc) gets each tile's products and stores STORES times, or not at all.
// PACKED: the tokens are read as pieces, else from x. (4,096 of 512, which every tile of rows
// reads again: 972 us from pieces, 1,106 from x.)
template <typename T, typename S, int STORES, bool PACKED, typename Done>
__device__ __forceinline__ void logits(const LossArgs& a, char* lds, int first_row, int end_row, int t0, int t1,
                                       int token0, Done done) {
    if constexpr (S::kWidth) {
        typedef WholeRows<T, S::kWidth, S::BM, S::NT> A;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
        const unsigned base = lds_address(lds);
        const unsigned a_at = base + A::place((wave / S::WN) * 32 * S::MA + (lane & 31), half);
        const A table(a.table, a.t_stride, end_row, a.width);
        constexpr int kSteps = S::kWidth / 16;
        typename Mma<T>::vec8 y[kSteps][S::NB];
        auto begin = [&] {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int j = 0; j < S::NB; ++j) {
                    const int t = token0 + (wave % S::WN) * 32 * S::NB + 32 * j + (lane & 31), c = 2 * s + half;
                    uint4 piece = make_uint4(0, 0, 0, 0);
                    if (PACKED) {
                        if (c < a.width8) piece = a.xg[(long long)c * a.x_pad + t];
                    } else if (t < a.t && 8 * c < a.width) {
                        piece = *(const uint4*)((const T*)a.x + t * a.x_stride + 8 * c);
                    }
                    y[s][j] = __builtin_bit_cast(typename Mma<T>::vec8, piece);
                }
            // settled here: inside the loop their wait would be for the tiles under way as well
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int j = 0; j < S::NB; ++j) asm volatile("" : "+v"(y[s][j]));
        };
        stages<S::kLoads, STORES>(
            t1 - t0, begin, [&](int i, int buf) { table.load(base + buf * S::kStage, first_row + (t0 + i) * S::BM); },
            [&](int i, int buf, auto next) {
                next();
                acc16 acc[S::MA][S::NB];
#pragma unroll
                for (int m = 0; m < S::MA; ++m) {
#pragma unroll
                    for (int j = 0; j < S::NB; ++j) acc[m][j] = zero16();
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const typename Mma<T>::vec8 x = A::read(a_at + buf * S::kStage, m, s);
#pragma unroll
                        for (int j = 0; j < S::NB; ++j) acc[m][j] = Mma<T>::mul(x, y[s][j], acc[m][j]);
                    }
                }
                done(t0 + i, acc);
                return true;
            });
    } else {
        typedef RowsOfMatrix<T, S::BM, S::NT> A;
        typedef std::conditional_t<PACKED, RowsOfPieces<T, S::BN, S::NT>, RowsOfMatrix<T, S::BN, S::NT>> B;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
        const int steps = (a.width + kStep - 1) / kStep;
        const unsigned base = lds_address(lds);
        const unsigned a_at = base + A::place((wave / S::WN) * 32 * S::MA + (lane & 31), half);
        const unsigned b_at = base + S::kA + B::place((wave % S::WN) * 32 * S::NB + (lane & 31), half);
        const A table(a.table, a.t_stride, end_row, a.width);
        const B tokens = [&] {
            if constexpr (PACKED)
                return B(a.xg, a.x_pad);
            else
                return B(a.x, a.x_stride, a.t, a.width);
        }();
        int tile_in = t0, k_in = 0, tile = t0, k = 0;
        acc16 acc[S::MA][S::NB];
        stages<S::kLoads, STORES>(
            (t1 - t0) * steps, [] {},
            [&](int, int buf) {
                const unsigned to = base + buf * S::kStage;
                table.load(to, first_row + tile_in * S::BM, k_in * kStep);
                tokens.load(to + S::kA, token0, k_in * kStep);
                if (++k_in == steps) k_in = 0, ++tile_in;
            },
            [&](int, int buf, auto next) {
                if (k == 0)
#pragma unroll
                    for (int i = 0; i < S::MA; ++i)
#pragma unroll
                        for (int j = 0; j < S::NB; ++j) acc[i][j] = zero16();
                products<T, S, S::MA * S::NB < 8>(
                    acc, [&](int m, int s) { return A::read(a_at + buf * S::kStage, m, s); },
                    [&](int j, int s) { return B::read(b_at + buf * S::kStage, j, s); }, next);
                if (++k < steps) return false;
                done(tile, acc);
                k = 0, ++tile;
                return true;
            });
    }
}

// Maxima and sums over a share of the rows, and the logit of each token's own row.
template <typename T, typename S>
__global__ __launch_bounds__(S::NT, 2) void k_loss_sum(LossArgs a) {
    __shared__ __align__(1024) char lds[3 * S::kStage];
    int split, token0;
    place_of<S>(a, &split, &token0);
    const int t0 = (int)((long long)a.tiles * split / a.splits), t1 = (int)((long long)a.tiles * (split + 1) / a.splits);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int row_in = (wave / S::WN) * 32 * S::MA, token_in = (wave % S::WN) * 32 * S::NB + (lane & 31);

    float m[S::NB], l[S::NB];
    int came[S::NB];
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
        const int t = token0 + token_in + 32 * j;
        m[j] = kLowest, l[j] = 0.0f, came[j] = t < a.t ? id_of(a, t) : -1;
    }

    logits<T, S, 0, !S::kOnce>(a, lds, 0, a.rows, t0, t1, token0, [&](int tile, acc16(&acc)[S::MA][S::NB]) {
        const int row0 = tile * S::BM + row_in;
        if (row0 + 32 * S::MA > a.rows) {
#pragma unroll
            for (int i = 0; i < S::MA; ++i)
#pragma unroll
                for (int j = 0; j < S::NB; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (row0 + 32 * i + acc_row(r, half) >= a.rows) acc[i][j][r] = -__builtin_inff();
        }
#pragma unroll
        for (int j = 0; j < S::NB; ++j) {
            const int mine = came[j] - row0;
            if (__any(mine >= 0 && mine < 32 * S::MA)) {
#pragma unroll
                for (int i = 0; i < S::MA; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (mine == 32 * i + acc_row(r, half)) a.hit[token0 + token_in + 32 * j] = acc[i][j][r] * a.scale2;
            }
            // Less the maximum so far. When their sum says that it lags by far (or is the
            // first tile's), it is brought up to date, and they are taken again.
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < S::MA; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], a.scale2, -m[j]));
            const bool lags = !(sum <= 0x1p40f);
            if (__any(lags)) {
                float top = acc[0][j][0];
#pragma unroll
                for (int i = 0; i < S::MA; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
                const float now = lags ? fmaxf(m[j], top * a.scale2) : m[j];
                l[j] *= __builtin_amdgcn_exp2f(m[j] - now);
                m[j] = now;
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < S::MA; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], a.scale2, -m[j]));
            }
            l[j] += sum;
        }
    });

    // the halves of a wavefront, then the wavefronts that share tokens
    __syncthreads();
    float2* all = (float2*)lds;  // [2 WM][BN]
#pragma unroll
    for (int j = 0; j < S::NB; ++j)
        all[(2 * (wave / S::WN) + half) * S::BN + token_in + 32 * j] = make_float2(m[j], l[j]);
    __syncthreads();
    for (int n = threadIdx.x; n < S::BN; n += S::NT) {
        float top = kLowest, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 2 * S::WM; ++w) top = fmaxf(top, all[w * S::BN + n].x);
#pragma unroll
        for (int w = 0; w < 2 * S::WM; ++w)
            sum += all[w * S::BN + n].y * __builtin_amdgcn_exp2f(all[w * S::BN + n].x - top);
        a.part[(long long)split * a.x_pad + token0 + n] = make_float2(top, sum);
    }
}

// A wavefront per token joins the shares, in order of their lanes.
__global__ __launch_bounds__(256) void k_loss_join(LossArgs a) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (t >= a.t) return;
    float m = kLowest, l = 0.0f;
    constexpr int kAhead = 8;
    for (int s = lane; s < a.splits; s += 64 * kAhead) {
        float2 p[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            p[j] = s + 64 * j < a.splits ? a.part[(long long)(s + 64 * j) * a.x_pad + t] : make_float2(kLowest, 0.0f);
        float now = m;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) now = fmaxf(now, p[j].x);
        l *= __builtin_amdgcn_exp2f(m - now);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) l += p[j].y * __builtin_amdgcn_exp2f(p[j].x - now);
        m = now;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const float m1 = __shfl_xor(m, off), l1 = __shfl_xor(l, off), now = fmaxf(m, m1);
        l = l * __builtin_amdgcn_exp2f(m - now) + l1 * __builtin_amdgcn_exp2f(m1 - now);
        m = now;
    }
    if (lane) return;
    const bool has = id_of(a, t) >= 0;
    const float lse2 = m + __builtin_amdgcn_logf(l);
    a.loss[t] = has ? (lse2 - a.hit[t]) * kLn2 : 0.0f;
    if (a.lse_out) a.lse_out[t] = has ? lse2 * kLn2 : 0.0f;
}

// dZ of a piece of the rows.
template <typename T, typename S>
__global__ __launch_bounds__(S::NT, 2) void k_loss_dz(LossArgs a) {
    __shared__ __align__(1024) char lds[3 * S::kStage];
    int split, token0;
    place_of<S>(a, &split, &token0);
    const int t0 = (int)((long long)a.tiles * split / a.splits), t1 = (int)((long long)a.tiles * (split + 1) / a.splits);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int row_in = __builtin_amdgcn_readfirstlane((wave / S::WN) * 32 * S::MA);
    const int token_in = (wave % S::WN) * 32 * S::NB + (lane & 31);

    float shift[S::NB], by[S::NB];
    int came[S::NB];
    const bool twice = a.t_all > a.t;
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
        const int t = token0 + token_in + 32 * j;
        shift[j] = a.shift[t], by[j] = a.by[t], came[j] = a.came[t] - a.row0;
    }
    const int token_at = __builtin_amdgcn_readfirstlane((wave % S::WN) * 32 * S::NB);
    const unsigned lane_at = half * a.t_pad + (lane & 31);
    logits<T, S, S::MA * S::NB * 2, true>(a, lds, a.row0, a.rows, t0, t1, token0, [&](int tile, acc16(&acc)[S::MA][S::NB]) {
        const int row0 = tile * S::BM + row_in;  // in the piece
        const int left = a.rows - a.row0 - row0;
        uint4* to = a.dz + (long long)(row0 >> 3) * a.t_pad + token0 + token_at;
#pragma unroll
        for (int j = 0; j < S::NB; ++j) {
            const int mine = came[j] - row0;
            const bool any = __any(mine >= 0 && mine < 32 * S::MA);
            // without a row: 0 also by a row that is not finite
            const bool none = came[j] < -a.row0, some_none = __any(none);
#pragma unroll
            for (int i = 0; i < S::MA; ++i) {
                acc16& p = acc[i][j];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[r], a.scale2, -shift[j]));
                if (any)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (mine == 32 * i + acc_row(r, half)) p[r] -= 1.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) p[r] *= by[j];
                if (some_none)
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[r] = none ? 0.0f : p[r];
                if (twice && token0 + token_in + 32 * j >= a.t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[r] -= (float)(T)p[r];
                if (left < 32 * S::MA)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (32 * i + acc_row(r, half) >= left) p[r] = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    unsigned x0 = Mma<T>::pair(p[4 * q], p[4 * q + 1]), x1 = Mma<T>::pair(p[4 * q + 2], p[4 * q + 3]);
                    unsigned y0 = Mma<T>::pair(p[4 * q + 4], p[4 * q + 5]), y1 = Mma<T>::pair(p[4 * q + 6], p[4 * q + 7]);
                    trade_halves(x0, y0);
                    trade_halves(x1, y1);
                    uint4* row = to + (long long)(4 * i + q) * a.t_pad + 32 * j;
                    row[lane_at] = make_uint4(x0, x1, y0, y1);
                }
            }
        }
    });
}

// ---- the gradients' products ---------------------------------------------------

// grad_x of a piece: [width x tokens] = W^T dZ over a share of the piece's rows,
// added to what the pieces before left in its part.
template <typename T, typename S>
__device__ __forceinline__ void grad_x(const LossArgs& a, unsigned id, char* lds) {
    typedef ColumnsOfMatrix<T, S::BM, S::NT> A;
    typedef RowsOfPieces<T, S::BN, S::NT> B;
    const int col_tiles = (a.width + S::BM - 1) / S::BM;
    const int col0 = (id % col_tiles) * S::BM;
    id /= col_tiles;
    const int token0 = (id % a.token_tiles) * S::BN, split = id / a.token_tiles;
    const int steps = a.piece / kStep;
    const int k0 = (int)((long long)steps * split / a.x_splits), k1 = (int)((long long)steps * (split + 1) / a.x_splits);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const unsigned base = lds_address(lds);
    const A table(a.table, a.t_stride, a.rows, col0, a.width);
    const B dz(a.dz, a.t_pad);
    const int a_block = (wave / S::WN) * S::MA;
    const uint2 a_at = A::place(lane);
    const unsigned b_at = base + S::kA + B::place((wave % S::WN) * 32 * S::NB + (lane & 31), half);
    acc16 acc[S::MA][S::NB];
#pragma unroll
    for (int i = 0; i < S::MA; ++i)
#pragma unroll
        for (int j = 0; j < S::NB; ++j) acc[i][j] = zero16();
    stages<S::kLoads, 0>(
        k1 - k0, [] {},
        [&](int i, int buf) {
            const unsigned to = base + buf * S::kStage;
            table.load(to, a.row0 + (k0 + i) * kStep);
            dz.load(to + S::kA, token0, (k0 + i) * kStep);
        },
        [&](int, int buf, auto next) {
            const unsigned on = base + buf * S::kStage;
            products<T, S, true>(
                acc, [&](int m, int s) { return A::read(make_uint2(a_at.x + on, a_at.y + on), a_block + m, s); },
                [&](int j, int s) { return B::read(b_at + buf * S::kStage, j, s); }, next);
            return false;
        });
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
        const int t = token0 + (wave % S::WN) * 32 * S::NB + 32 * j + (lane & 31);
        if (t >= a.t_all) continue;
        const bool none = a.came[t] < 0;
        // the second time's are further parts
        const long long part = t < a.t ? 2 * split : 2 * split + 1;
        float* to = a.part_x + ((a.t_all > a.t ? part : split) * a.x_tokens + (t < a.t ? t : t - a.t)) * a.width;
#pragma unroll
        for (int i = 0; i < S::MA; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = col0 + 32 * (a_block + i) + 8 * q + 4 * half;
                if (c >= a.width) continue;
                float4 v = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
                if (none) v = make_float4(0, 0, 0, 0);
                if (!a.first) {
                    const float4 w = *(const float4*)(to + c);
                    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                }
                *(float4*)(to + c) = v;
            }
    }
}

// grad_table of a piece: [width x rows] = X^T dZ over a share of the tokens.
template <typename T, typename S>
__device__ __forceinline__ void grad_table(const LossArgs& a, unsigned id, char* lds) {
    typedef ColumnsOfPieces<T, S::BM, S::NT, S::BM == 128> A;  // the widest's columns are all there
    typedef ColumnsOfPieces<T, S::BN, S::NT> B;
    const int col_tiles = (a.width + S::BM - 1) / S::BM, row_tiles = a.piece / S::BN;
    const int col0 = (id % col_tiles) * S::BM;
    id /= col_tiles;
    const int row0 = (id % row_tiles) * S::BN, split = id / row_tiles;
    const int steps = a.tokens_in / kStep;
    const int k0 = (int)((long long)steps * split / a.t_splits), k1 = (int)((long long)steps * (split + 1) / a.t_splits);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const unsigned base = lds_address(lds);
    const A tokens(a.xg, a.x_pad, col0, a.width8);
    const B dz(a.dz, a.t_pad, row0);
    const int a_block = (wave / S::WN) * S::MA, b_block = (wave % S::WN) * S::NB;
    const uint2 at = A::place(lane);
    acc16 acc[S::MA][S::NB];
#pragma unroll
    for (int i = 0; i < S::MA; ++i)
#pragma unroll
        for (int j = 0; j < S::NB; ++j) acc[i][j] = zero16();
    stages<S::kLoads, 0>(
        k1 - k0, [] {},
        [&](int i, int buf) {
            const unsigned to = base + buf * S::kStage;
            tokens.load(to, (k0 + i) * kStep);
            dz.load(to + S::kA, (k0 + i) * kStep);
        },
        [&](int, int buf, auto next) {
            const unsigned x_on = base + buf * S::kStage, y_on = x_on + S::kA;
            products<T, S, true>(
                acc, [&](int m, int s) { return A::read(make_uint2(at.x + x_on, at.y + x_on), a_block + m, s); },
                [&](int j, int s) { return B::read(make_uint2(at.x + y_on, at.y + y_on), b_block + j, s); }, next);
            return false;
        });
    const float down = down_of<T>(a);
#pragma unroll
    for (int j = 0; j < S::NB; ++j) {
        const int row = row0 + 32 * (b_block + j) + (lane & 31);  // of the piece
#pragma unroll
        for (int i = 0; i < S::MA; ++i) {
            const int c0 = col0 + 32 * (a_block + i);
            if (a.part_t) {
                float* to = a.part_t + ((long long)split * a.piece + row) * a.width;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = c0 + 8 * q + 4 * half;
                    if (c < a.width)
                        *(float4*)(to + c) = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                                         acc[i][j][4 * q + 3]);
                }
                continue;
            }
            uint4 made[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float p[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) p[r] = acc[i][j][8 * q + r] * down;
                unsigned x0 = Mma<T>::pair(p[0], p[1]), x1 = Mma<T>::pair(p[2], p[3]);
                unsigned y0 = Mma<T>::pair(p[4], p[5]), y1 = Mma<T>::pair(p[6], p[7]);
                trade_halves(x0, y0);
                trade_halves(x1, y1);
                made[q] = make_uint4(x0, x1, y0, y1);
            }
            trade_quarters(made[0], made[1]);
            const int c = c0 + 8 * quarter_piece(lane);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const long long at = a.row0 + row0 + 32 * (b_block + j) + 16 * q + (lane & 15);
                if (at < a.rows && c < a.width) *(uint4*)((T*)a.gt + at * a.width + c) = made[q];
            }
        }
    }
}

// Both in one launch, the first x_blocks blocks grad_x's.
template <typename T, typename S>
__global__ __launch_bounds__(S::NT, 2) void k_loss_grads(LossArgs a, unsigned x_blocks) {
    __shared__ __align__(1024) char lds[3 * S::kStage];
    if (blockIdx.x < x_blocks)
        grad_x<T, S>(a, xcd_block(blockIdx.x, x_blocks), lds);
    else
        grad_table<T, S>(a, xcd_block(blockIdx.x - x_blocks, gridDim.x - x_blocks), lds);
}

// Parts joined in order, rounded: n elements of out from `count` parts. A thread has four
// elements and loads eight parts at once.
struct Joined {
    const float* part;
    int count;
    long long n, pitch;
    void* out;
};
template <typename T>
__global__ __launch_bounds__(256) void k_loss_round(LossArgs a, Joined first, Joined second) {
    const float down = down_of<T>(a);
    const Joined& b = blockIdx.y ? second : first;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4; i < b.n; i += 1024ll * gridDim.x) {
        float4 s = make_float4(0, 0, 0, 0);
        constexpr int kAhead = 8;
        for (int p = 0; p < b.count; p += kAhead) {
            float4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) v[j] = *(const float4*)(b.part + min(p + j, b.count - 1) * b.pitch + i);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (p + j < b.count) s.x += v[j].x, s.y += v[j].y, s.z += v[j].z, s.w += v[j].w;
        }
        const float r[4] = {s.x * down, s.y * down, s.z * down, s.w * down};
        Pack<T, 4>::store((T*)b.out + i, r);
    }
}

// Without a token: every row's gradient is zero.
__global__ __launch_bounds__(256) void k_loss_clear(uint4* to, long long n) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x)
        to[i] = make_uint4(0, 0, 0, 0);
}

// ---- host --------------------------------------------------------------------

template <typename T>
using Wide = Shape<T, 4, 2, 2, 2>;   // 256 x 128
template <typename T>
using Even = Shape<T, 2, 2, 2, 2>;   // 128 x 128
template <typename T>
using Slim = Shape<T, 2, 1, 4, 1>;   // 256 x 32: few tokens

long long round256(long long n) { return (n + 255) / 256 * 256; }
long long ceil_div(long long n, long long d) { return (n + d - 1) / d; }
int clamp(long long n, long long lo, long long hi) { return (int)(n < lo ? lo : n > hi ? hi : n); }

// Shares that the tiles of rows are cut into: of eight tiles or more while those fill the
// card's places (and up to 4,096 blocks), else as many as fill them. Fewer tiles than
// that to a block and its beginning counts: 997 tokens by 13,391 rows take 63 us with 768
// blocks and 75 with one for each of 1,680 tiles.
int splits_of(long long tiles, long long token_tiles, int places) {
    const long long of_eight = tiles / 8, most = 4096 / token_tiles;
    const long long n = of_eight * token_tiles < places ? places / token_tiles : of_eight < most ? of_eight : most;
    return clamp(n, 1, tiles);
}

// When the last of a launch's blocks is done, `first` of them of a steps, then `second` of b, on
// `places` at once.
long long finish(long long places, long long first, long long a, long long second, long long b) {
    struct { long long at, n; } free[64] = {{0, places}};
    int count = 1;
    long long end = 0;
    for (int kind = 0; kind < 2; ++kind) {
        long long left = kind ? second : first;
        const long long steps = kind ? b : a;
        // whole rounds at once: what is left over is at most two more
        if (left > 4 * places) {
            const long long rounds = left / places - 2;
            for (int i = 0; i < count; ++i) free[i].at += rounds * steps;
            left -= rounds * places;
        }
        while (left > 0) {
            int next = 0;
            for (int i = 1; i < count; ++i)
                if (free[i].at < free[next].at) next = i;
            const long long n = left < free[next].n ? left : free[next].n, at = free[next].at + steps;
            left -= n;
            if (n == free[next].n || count == 64)
                free[next].at = at;
            else
                free[next].n -= n, free[count++] = {at, n};
            end = at > end ? at : end;
        }
        for (int i = 0; i < count; ++i)
            if (free[i].at > end) end = free[i].at;
    }
    return end;
}

// How a call is cut.
struct Cut {
    long long t_pad, width8, t_all;
    long long band;    // tokens that dZ is written for at once, whole tiles
    int bands;
    int splits, slim;  // splits: at most
    int piece, pieces, x_splits, t_splits;
};

Cut cut(long long t, long long rows, long long width, bool grad) {
    Cut c;
    c.t_all = grad && t <= kTwice ? 2 * t : t;
    c.t_pad = ceil_div(c.t_all, kTokenPad) * kTokenPad;
    c.slim = c.t_all <= 32;
    // whole tiles of columns of the widest shape, and stages where they are read: zeros past the width
    c.width8 = width > 128 ? ceil_div(width, 256) * 32 : c.slim ? ceil_div(width, kStep) * (kStep / 8) : width / 8;
    // so many tokens that 256 rows' dZ is a piece of its own
    c.bands = (int)ceil_div(c.t_pad * 2 * kRowTile, kPieceBytes);
    c.band = ceil_div(ceil_div(c.t_pad, c.bands), kTokenPad) * kTokenPad;
    c.bands = (int)ceil_div(c.t_pad, c.band);
    const long long tiles = ceil_div(rows, kRowTile), token_tiles = c.slim ? 1 : c.t_pad / kTokenPad;
    c.splits = clamp(4096 / token_tiles, 1, 4 * tiles);
    const long long piece = kPieceBytes / (2 * c.band) / kRowTile * kRowTile;
    c.pieces = (int)ceil_div(tiles * kRowTile, piece);
    c.piece = (int)(ceil_div(tiles, c.pieces) * kRowTile);
    c.pieces = (int)ceil_div(tiles * kRowTile, c.piece);
    const long long cols = ceil_div(width, width > 128 ? 256 : 128);
    // Both gradients' products into blocks enough for one on each of 256 CUs, since they run
    // together (a training step of 4,096 tokens of 512 by 214,272 rows: 5% more with twice as many,
    // whose partial sums pass memory twice as often, 15% more with half).
    const long long x_tiles = cols * (c.band / 128), t_tiles = cols * (c.piece / 128);
    c.x_splits = clamp(256 / x_tiles, 1, c.piece / 512 > 1 ? c.piece / 512 : 1);
    c.t_splits = clamp(256 / t_tiles, 1, c.band / 512 > 1 ? c.band / 512 : 1);
    if (!grad) return c;
    // A few blocks more than the card holds begin when the others are done. Where another pair of
    // powers of two ends a quarter sooner it is taken: a step takes about a microsecond with every
    // place taken, and so do 5 MB of partial sums. (Backward of 20,000 tokens of 512 by 214,272
    // rows: 15.6 ms, 18.5 else; of 1,024 by 13,391 rows 1.93 and 2.28. Gains that are smaller by
    // this count were none: 20,000 of 256 by 214,272 rows 10.2 ms, 9.3 without.)
    const long long places = width > 128 ? 512 : 768;
    auto parts = [&](long long x, long long t1) { return 8 * width * (x * c.t_all + (t1 > 1 ? t1 * c.piece : 0)) / 5000000; };
    auto steps = [&](long long x, long long t1) {
        return finish(places, x_tiles * x, ceil_div(c.piece / kStep, x), t_tiles * t1, ceil_div(c.band / kStep, t1));
    };
    long long best = (parts(c.x_splits, c.t_splits) + steps(c.x_splits, c.t_splits)) * 3 / 4;
    for (long long x = 1; x == 1 || (x <= 512 && x * 256 <= c.piece); x *= 2)
        for (long long t1 = 1; t1 == 1 || (t1 <= 256 && t1 * 512 <= c.band); t1 *= 2) {
            if (parts(x, t1) >= best) break;
            const long long time = parts(x, t1) + steps(x, t1);
            if (time < best) best = time, c.x_splits = (int)x, c.t_splits = (int)t1;
        }
    return c;
}

bool sizes_ok(int64_t t, int64_t rows, int64_t width) {
    return t >= 0 && t <= kMaxTokens && rows >= 1 && rows <= kMaxRows && width >= 8 && width <= kMaxWidth &&
           width % 8 == 0;
}

struct Layout {
    long long xg, came, shift, by, hit, part, top, part_x, part_t, dz, total;
};

// grad_table goes through sums in memory: of shares of the tokens, or of their bands.
bool parts_of_table(const Cut& c) { return c.t_splits > 1 || c.bands > 1; }

Layout layout(const Cut& c, long long t, long long width, bool grad) {
    Layout l = {};
    long long at = 0;
    auto take = [&](long long bytes) {
        const long long was = at;
        at += round256(bytes);
        return was;
    };
    if (grad || (!c.slim && width > 128)) l.xg = take(c.width8 * c.t_pad * 16);
    if (!grad) {
        l.hit = take(c.t_pad * 4);
        l.part = take(c.splits * c.t_pad * 8);
    } else {
        l.came = take(c.t_pad * 4);
        l.shift = take(c.t_pad * 4);
        l.by = take(c.t_pad * 4);
        l.top = take(kTops * 4);
        l.part_x = take((long long)c.x_splits * c.t_all * width * 4);
        l.part_t = take(parts_of_table(c) ? (long long)c.bands * c.t_splits * c.piece * width * 4 : 0);
        l.dz = take((long long)c.piece / 8 * c.band * 16);
    }
    l.total = at;
    return l;
}

bool check(const void* x, int64_t x_stride, const void* table, int64_t table_stride, int32_t dtype, int64_t t,
           int64_t rows, int64_t width, const void* ids, int32_t id_bytes, float scale) {
    if (dtype != TOK_BF16 && dtype != TOK_F16) return false;
    if (!sizes_ok(t, rows, width) || (id_bytes != 4 && id_bytes != 8)) return false;
    if (x_stride < 0 || x_stride % 8 || x_stride >= kMaxStride || table_stride < 0 || table_stride % 8 ||
        table_stride >= kMaxStride)
        return false;
    if (!(scale >= 1e-30f) || !(scale <= 1e30f)) return false;
    if (!table || ((size_t)table & 15) || ((size_t)x & 15)) return false;
    return t == 0 || (x && ids && (size_t)ids % id_bytes == 0);
}

LossArgs make_args(const void* x, int64_t x_stride, const void* table, int64_t table_stride, int64_t t, int64_t rows,
                   int64_t width, const void* ids, int32_t id_bytes, float scale, const Cut& c, const Layout& l,
                   char* ws) {
    LossArgs a = {};
    a.x = x, a.x_stride = x_stride, a.table = table, a.t_stride = table_stride;
    a.t = (int)t, a.rows = (int)rows, a.width = (int)width, a.ids = ids, a.id_bytes = id_bytes;
    a.scale = scale, a.scale2 = (float)(scale * 1.4426950408889634);
    a.x_pad = (int)c.t_pad, a.t_pad = (int)c.band, a.x_tokens = a.t;
    a.width8 = (int)c.width8, a.t_all = (int)c.t_all;
    a.xg = (uint4*)(ws + l.xg), a.came = (int*)(ws + l.came);
    a.shift = (float*)(ws + l.shift), a.by = (float*)(ws + l.by), a.hit = (float*)(ws + l.hit);
    a.part = (float2*)(ws + l.part), a.top = (float*)(ws + l.top);
    a.part_x = (float*)(ws + l.part_x), a.part_t = parts_of_table(c) ? (float*)(ws + l.part_t) : nullptr, a.dz = (uint4*)(ws + l.dz);
    a.piece = c.piece, a.x_splits = c.x_splits, a.t_splits = c.t_splits;
    a.tokens_in = c.slim ? 32 : (int)c.band;
    return a;
}

dim3 pack_grid(const LossArgs& a) {
    return dim3((unsigned)(a.x_pad / 32), (unsigned)ceil_div(a.width8, 8));
}

// Blocks that the card holds at once.
template <typename S>
constexpr int places() { return 256 * (160 * 1024 / (3 * S::kStage) < 3 ? 160 * 1024 / (3 * S::kStage) : 3); }

// A launch over tiles of the rows by tiles of the tokens.
template <typename S, typename F>
void over_tiles(LossArgs a, long long rows, long long tokens, F f) {
    a.tiles = (int)ceil_div(rows, S::BM);
    a.token_tiles = (int)ceil_div(tokens, S::BN);
    a.splits = splits_of(a.tiles, a.token_tiles, places<S>());
    f(a, dim3((unsigned)(a.token_tiles * a.splits)), dim3(S::NT));
}

template <typename T>
int forward(const LossArgs& a, const Cut& c, hipStream_t stream) {
    const bool packed = !c.slim && a.width > 128;
    if (packed) k_loss_pack<T, false><<<pack_grid(a), dim3(256), 0, stream>>>(a);
    int splits = 0;
    auto sum = [&](auto shape) {
        typedef decltype(shape) S;
        over_tiles<S>(a, a.rows, a.t, [&](const LossArgs& z, dim3 grid, dim3 block) {
            splits = z.splits;
            k_loss_sum<T, S><<<grid, block, 0, stream>>>(z);
        });
    };
    if (c.slim)
        sum(Slim<T>());
    else if (a.width <= 32)
        sum(Narrow<T, 32>());
    else if (a.width <= 64)
        sum(Narrow<T, 64>());
    else if (a.width <= 128)
        sum(Narrow<T, 128>());
    else
        sum(Even<T>());
    LossArgs z = a;
    z.splits = splits;
    k_loss_join<<<dim3((unsigned)ceil_div(a.t, 4)), dim3(256), 0, stream>>>(z);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

template <typename T, typename S>
void gradients(LossArgs a, hipStream_t stream) {
    a.token_tiles = (int)ceil_div(a.tokens_in, S::BN);
    const long long cols = ceil_div(a.width, S::BM);
    const long long x_blocks = a.gx ? cols * a.token_tiles * a.x_splits : 0;
    const long long blocks = x_blocks + (a.gt ? cols * (a.piece / S::BN) * a.t_splits : 0);
    k_loss_grads<T, S><<<dim3((unsigned)blocks), dim3(S::NT), 0, stream>>>(a, (unsigned)x_blocks);
}

template <typename T>
int backward(LossArgs a, const Cut& c, hipStream_t stream) {
    a.tops = clamp(ceil_div(a.t, 8192), 1, kTops);
    if (__is_same(T, f16_t)) k_loss_top<<<dim3(a.tops), dim3(1024), 0, stream>>>(a);
    k_loss_pack<T, true><<<pack_grid(a), dim3(256), 0, stream>>>(a);
    const long long all = ceil_div(a.rows, kRowTile) * kRowTile;
    for (int p = 0; p < c.pieces; ++p) {
        a.row0 = p * c.piece;
        a.piece = (int)(all - a.row0 < c.piece ? all - a.row0 : c.piece);
        a.first = p == 0;
        for (int band = 0; band < c.bands; ++band) {
            const long long from = band * c.band, left = c.t_pad - from;
            LossArgs b = a;
            if (c.bands > 1) {  // no token goes through twice
                b.tokens_in = (int)(left < c.band ? left : c.band);
                b.t = b.t_all = (int)(a.t - from < c.band ? a.t - from : c.band);
                b.xg += from, b.came += from, b.shift += from, b.by += from, b.part_x += from * a.width;
                b.part_t += (long long)band * a.t_splits * a.piece * a.width;
            }
            auto dz = [&](auto shape) {
                typedef decltype(shape) S;
                over_tiles<S>(b, b.piece, b.tokens_in, [&](const LossArgs& z, dim3 grid, dim3 block) {
                    k_loss_dz<T, S><<<grid, block, 0, stream>>>(z);
                });
            };
            if (c.slim)
                dz(Slim<T>());
            else if (a.width <= 32)
                dz(Narrow<T, 32>());
            else if (a.width <= 64)
                dz(Narrow<T, 64>());
            else if (a.width <= 128)
                dz(Narrow<T, 128>());
            else
                dz(Wide<T>());
            if (a.width > 128)
                gradients<T, Wide<T>>(b, stream);
            else
                gradients<T, Even<T>>(b, stream);
        }
        const bool last = p + 1 == c.pieces;
        const long long there = a.rows - a.row0 < a.piece ? a.rows - a.row0 : a.piece, n = (long long)a.t * a.width;
        Joined joined[2] = {};
        int jobs = 0;
        if (a.gt && a.part_t)
            joined[jobs++] = {a.part_t, c.bands * c.t_splits, there * a.width, (long long)a.piece * a.width,
                              (T*)a.gt + (long long)a.row0 * a.width};
        if (a.gx && last) joined[jobs++] = {a.part_x, c.x_splits * (a.t_all > a.t ? 2 : 1), n, n, a.gx};
        const long long most = joined[0].n > joined[1].n ? joined[0].n : joined[1].n;
        if (jobs)
            k_loss_round<T><<<dim3(clamp(ceil_div(most, 1024), 1, 1 << 20), jobs), dim3(256), 0, stream>>>(
                a, joined[0], joined[1]);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

}  // namespace

extern "C" {

int64_t tok_row_loss_workspace_bytes(int64_t t, int64_t rows, int64_t width) {
    if (!sizes_ok(t, rows, width)) return VOX_EINVAL;
    return t == 0 ? 0 : layout(cut(t, rows, width, false), t, width, false).total;
}

int64_t tok_row_loss_grad_workspace_bytes(int64_t t, int64_t rows, int64_t width) {
    if (!sizes_ok(t, rows, width)) return VOX_EINVAL;
    return t == 0 ? 0 : layout(cut(t, rows, width, true), t, width, true).total;
}

int tok_row_loss(const void* x, int64_t x_stride, const void* table, int64_t table_stride, int32_t dtype,
                 int64_t t, int64_t rows, int64_t width, const void* ids, int32_t id_bytes, float scale, float* loss,
                 float* lse, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!check(x, x_stride, table, table_stride, dtype, t, rows, width, ids, id_bytes, scale)) return VOX_EINVAL;
    if (t == 0) return VOX_OK;
    if (!loss || ((size_t)loss | (size_t)lse) % 4) return VOX_EINVAL;
    const Cut c = cut(t, rows, width, false);
    const Layout l = layout(c, t, width, false);
    if (!workspace_ok(workspace, workspace_bytes, l.total)) return VOX_EWORKSPACE;
    LossArgs a = make_args(x, x_stride, table, table_stride, t, rows, width, ids, id_bytes, scale, c, l, (char*)workspace);
    a.loss = loss, a.lse_out = lse;
    return dtype == TOK_BF16 ? forward<bf16_t>(a, c, stream) : forward<f16_t>(a, c, stream);
}

int tok_row_loss_grad(const float* grad, const void* x, int64_t x_stride, const void* table, int64_t table_stride,
                      int32_t dtype, int64_t t, int64_t rows, int64_t width, const void* ids, int32_t id_bytes,
                      const float* lse, float scale, void* grad_x, void* grad_table, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream) {
    if (!check(x, x_stride, table, table_stride, dtype, t, rows, width, ids, id_bytes, scale)) return VOX_EINVAL;
    if ((t && !grad_x && !grad_table) || (((size_t)grad_x | (size_t)grad_table) & 15)) return VOX_EINVAL;
    if (t && (!grad || !lse || ((size_t)grad | (size_t)lse) % 4)) return VOX_EINVAL;
    if (t == 0) {
        if (!grad_table) return VOX_OK;
        k_loss_clear<<<dim3(2048), dim3(256), 0, stream>>>((uint4*)grad_table, rows * width / 8);
        const hipError_t e = hipGetLastError();
        return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
    }
    const Cut c = cut(t, rows, width, true);
    const Layout l = layout(c, t, width, true);
    if (!workspace_ok(workspace, workspace_bytes, l.total)) return VOX_EWORKSPACE;
    LossArgs a = make_args(x, x_stride, table, table_stride, t, rows, width, ids, id_bytes, scale, c, l, (char*)workspace);
    a.grad = grad, a.lse = lse, a.gx = grad_x, a.gt = grad_table;
    return dtype == TOK_BF16 ? backward<bf16_t>(a, c, stream) : backward<f16_t>(a, c, stream);
}

}  // extern "C"
