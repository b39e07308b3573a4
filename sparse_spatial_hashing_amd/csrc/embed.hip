// Embedding lookup and the gradient of its table (tokens.h).
//
// The lookup moves rows in pieces of up to 16 bytes, one lane per piece.
//
// The gradient sorts (row, token) pairs by row with stable passes from the
// lowest digit up, so the tokens of a row come out in token order, and sums
// equal rows over runs of sorted pairs, a group of lanes per run:
//   k_eg_tiny     up to kTiny tokens: no sort, all in one launch; or
//   k_eg_small    up to kSmall tokens: some blocks sort in LDS while the others
//                 clear the gradient; or
//   per digit
//   k_eg_count    digits of each tile of pairs, counted (the first time other
//                 blocks clear the gradient)
//   k_eg_prefix   one block per digit: where each tile's entries of it start
//   k_eg_scatter  pairs to their places (ranks by ballots, in input order)
//   then
//   k_eg_reduce   sums of rows that start and end in a run go out; a row cut
//                 by a run's border leaves partial sums
//   k_eg_join     partial sums of a cut row added in order
// No floating-point atomics: the order of every sum is that of the tokens.

#include <hip/hip_runtime.h>

#include "token_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kPer = 8;                    // pairs per thread of a sort tile
constexpr int kTile = kBlock * kPer;
constexpr int kMaxBits = 9;                // bits of a digit, at most
constexpr int kMaxDigits = 1 << kMaxBits;
constexpr int kSmall = 16384;              // tokens that are sorted in LDS
constexpr int kSmallBlock = 1024;
constexpr int kSmallSorts = 16;            // blocks that share the sort
constexpr int kBatch = 8;                  // rows in flight per group of lanes
constexpr long long kMaxN = 1ll << 27;
constexpr long long kMaxRows = 1ll << 24;
constexpr long long kMaxWidth = 65536;

// ------------------------------------------------------------------ lookup --

// Bound by memory: 2,097,152 of 60,000 rows of 64 bf16 in 64 us, 5.4 TB/s with
// the table's copies in the eight L2 caches (one row per thread: 71).
// 2^lpr_log lanes share a row of `pieces` pieces of N elements, and R rows,
// one block's rows apart, so that R loads are under way in a thread.
template <typename T, int N, typename Id, int R>
__global__ __launch_bounds__(kBlock) void k_embed(const T* __restrict__ table, long long rows,
                                                  int width, long long stride,
                                                  const Id* __restrict__ ids, long long n,
                                                  float scale, T* __restrict__ out, int lpr_log) {
    const int lpr = 1 << lpr_log;
    const int pieces = width / N;
    const int per = kBlock >> lpr_log;  // rows of the block at a time
    const long long first = (long long)blockIdx.x * per * R + (threadIdx.x >> lpr_log);
    long long id[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long i = first + r * per;
        id[r] = (long long)ids[i < n ? i : n - 1];
    }
    for (int p = threadIdx.x & (lpr - 1); p < pieces; p += lpr) {
        typename Pack<T, N>::vec raw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = id[r] >= 0 && id[r] < rows;
            raw[r] = Pack<T, N>::raw(table + (in ? id[r] : 0) * stride + p * N);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long i = first + r * per;
            if (i >= n) continue;
            const bool in = id[r] >= 0 && id[r] < rows;
            float x[N];
            Pack<T, N>::wide(raw[r], x);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = in ? x[j] * scale : 0.0f;
            Pack<T, N>::store(out + i * width + p * N, x);
        }
    }
}

// -------------------------------------------------------------------- sort --

template <typename Id>
__device__ __forceinline__ unsigned key_of(const Id* ids, long long i, long long rows) {
    const long long id = (long long)ids[i];
    return id >= 0 && id < rows ? (unsigned)id : (unsigned)rows;  // rows: no row, sorted last
}

template <typename Id, bool FIRST>
__device__ __forceinline__ uint2 pair_of(const Id* ids, const uint2* pairs, long long i,
                                         long long rows) {
    if (FIRST) return make_uint2(key_of(ids, i, rows), (unsigned)i);
    return pairs[i];
}

__device__ __forceinline__ void clear(uint4* out, long long pieces, unsigned char* tail, int bytes,
                                      long long block, long long blocks, int threads) {
    const long long step = blocks * threads;
    for (long long p = block * threads + threadIdx.x; p < pieces; p += step)
        out[p] = make_uint4(0, 0, 0, 0);
    if (block == 0 && (int)threadIdx.x < bytes) tail[threadIdx.x] = 0;
}

// Of the first pass, the blocks past the tiles' own clear the gradient.
template <typename Id, bool FIRST>
__global__ __launch_bounds__(kBlock) void k_eg_count(const Id* __restrict__ ids,
                                                     const uint2* __restrict__ pairs, long long n,
                                                     long long rows, int shift, int bits, int tiles,
                                                     unsigned* __restrict__ counts,
                                                     uint4* __restrict__ out, long long pieces,
                                                     unsigned char* __restrict__ tail, int bytes) {
    __shared__ unsigned hist[kMaxDigits];
    if (FIRST && (int)blockIdx.x >= tiles) {
        clear(out, pieces, tail, bytes, (int)blockIdx.x - tiles, (int)gridDim.x - tiles, kBlock);
        return;
    }
    const int digits = 1 << bits;
    for (int d = threadIdx.x; d < digits; d += kBlock) hist[d] = 0;
    __syncthreads();
    const long long base = (long long)blockIdx.x * kTile;
    unsigned key[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long i = base + k * kBlock + threadIdx.x;
        key[k] = pair_of<Id, FIRST>(ids, pairs, i < n ? i : n - 1, rows).x;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (base + k * kBlock + threadIdx.x < n)
            atomicAdd(&hist[(key[k] >> shift) & (digits - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kBlock)
        counts[(long long)d * tiles + blockIdx.x] = hist[d];
}

// Exclusive prefix over the tiles of one digit, in place; totals[d].
__global__ __launch_bounds__(kBlock) void k_eg_prefix(unsigned* __restrict__ counts, int tiles,
                                                      unsigned* __restrict__ totals) {
    __shared__ unsigned wsum[kWsumWords];
    unsigned* c = counts + (long long)blockIdx.x * tiles;
    unsigned run = 0;
    for (int t0 = 0; t0 < tiles; t0 += kBlock) {
        const int t = t0 + threadIdx.x;
        const unsigned v = t < tiles ? c[t] : 0u;
        unsigned total;
        const unsigned ex = block_excl_scan<kWaves>(v, wsum, &total);
        if (t < tiles) c[t] = run + ex;
        run += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// The tile is put in order in LDS first, so that the entries of a digit go out
// together: 14 us a pass over 2,097,152 pairs (straight from the registers 37).
template <typename Id, bool FIRST>
__global__ __launch_bounds__(kBlock) void k_eg_scatter(
    const Id* __restrict__ ids, const uint2* __restrict__ pairs, long long n, long long rows,
    int shift, int bits, int tiles, const unsigned* __restrict__ counts,
    const unsigned* __restrict__ totals, uint2* __restrict__ out) {
    __shared__ unsigned wsum[kWsumWords];
    __shared__ unsigned base[kMaxDigits];       // place of a digit's entries less their place here
    __shared__ unsigned seen[kWaves][kMaxDigits];
    __shared__ uint2 local[kTile];
    const int digits = 1 << bits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // wavefront w ranks its kPer * 64 consecutive pairs in order
    const long long first = (long long)blockIdx.x * kTile + wave * (kPer * kWave);
    uint2 pair[kPer];
    unsigned rank[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long i = first + k * kWave + lane;
        pair[k] = pair_of<Id, FIRST>(ids, pairs, i < n ? i : n - 1, rows);
    }
    for (int d = threadIdx.x; d < kWaves * kMaxDigits; d += kBlock) (&seen[0][0])[d] = 0;
    static_assert(kMaxDigits <= 2 * kBlock, "two digits per thread");
    const int d0 = 2 * threadIdx.x;
    {
        // where this tile's entries of each digit go
        const unsigned u = d0 < digits ? totals[d0] : 0u, v = d0 + 1 < digits ? totals[d0 + 1] : 0u;
        unsigned total;
        const unsigned ex = block_excl_scan<kWaves>(u + v, wsum, &total);
        if (d0 < digits) base[d0] = ex + counts[(long long)d0 * tiles + blockIdx.x];
        if (d0 + 1 < digits)
            base[d0 + 1] = ex + u + counts[(long long)(d0 + 1) * tiles + blockIdx.x];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool valid = first + k * kWave + lane < n;
        const unsigned d = (pair[k].x >> shift) & (digits - 1);
        const unsigned long long m = match_mask(d, valid, bits);
        const unsigned before = valid ? seen[wave][d] : 0u;
        rank[k] = before + (unsigned)__popcll(m & lanes_below(lane));
        if (valid && (m & lanes_above(lane)) == 0)
            seen[wave][d] = before + (unsigned)__popcll(m);
        // the next pair of any lane reads what the last lane of a digit wrote
        asm volatile("" ::: "memory");
    }
    __syncthreads();
    {
        // where each wavefront's entries of a digit go in the tile
        unsigned c[2][kWaves], sum[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                c[j][w] = d0 + j < digits ? seen[w][d0 + j] : 0u;
                sum[j] += c[j][w];
            }
        unsigned total;
        unsigned at = block_excl_scan<kWaves>(sum[0] + sum[1], wsum, &total);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (d0 + j < digits) base[d0 + j] -= at;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (d0 + j < digits) seen[w][d0 + j] = at;
                at += c[j][w];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (first + k * kWave + lane < n)
            local[seen[wave][(pair[k].x >> shift) & (digits - 1)] + rank[k]] = pair[k];
    __syncthreads();
    const int count = (int)(n - (long long)blockIdx.x * kTile < kTile
                                ? n - (long long)blockIdx.x * kTile : (long long)kTile);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int at = k * kBlock + threadIdx.x;
        if (at < count) {
            const uint2 p = local[at];
            out[base[(p.x >> shift) & (digits - 1)] + at] = p;
        }
    }
}

// ------------------------------------------------------------------ reduce --

// kSmallSorts blocks sort n <= kSmall pairs, each those of its share of the
// rows: it reads all ids, keeps its own in token order and counts those of
// lower rows, which is where its own go. Pairs stay in registers and are put in
// order through LDS. The other blocks clear the gradient meanwhile. 12,000
// tokens and 110 MB of gradient: 20 us, which is what clearing alone takes; one
// block sorting all took 28. Through the passes below the same sort takes seven
// launches, 30 us after the clearing.
template <typename Id>
__global__ __launch_bounds__(kSmallBlock) void k_eg_small(const Id* __restrict__ ids, int n,
                                                          long long rows, int share, int passes,
                                                          int bits_all, uint2* __restrict__ out_pairs,
                                                          uint4* __restrict__ out, long long pieces,
                                                          unsigned char* __restrict__ tail,
                                                          int bytes) {
    constexpr int W = kSmallBlock / kWave, E = kSmall / kSmallBlock;
    __shared__ uint2 local[kSmall];
    __shared__ unsigned short seen[W][kMaxDigits];
    __shared__ unsigned wsum[kWsumWords];
    if (blockIdx.x >= kSmallSorts) {
        clear(out, pieces, tail, bytes, blockIdx.x - kSmallSorts, gridDim.x - kSmallSorts, kSmallBlock);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned lo = blockIdx.x * (unsigned)share;  // rows [lo, lo + share), `rows` the last of all
    uint2 pair[E];
    unsigned rank[E];
    unsigned lower = 0, mine = 0;  // of this wavefront's tokens
    {
        const int per = (n + kSmallBlock - 1) / kSmallBlock;  // <= E per thread
        const int first = wave * (per * kWave) + lane;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            pair[k] = make_uint2(0, 0);
            if (k < per) {
                const int i = first + k * kWave;
                pair[k] = make_uint2(key_of(ids, i < n ? i : n - 1, rows), (unsigned)i);
            }
        }
        unsigned long long keep[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const bool valid = k < per && first + k * kWave < n;
            keep[k] = __ballot(valid && pair[k].x >= lo && pair[k].x - lo < (unsigned)share);
            lower += (unsigned)__popcll(__ballot(valid && pair[k].x < lo));
            rank[k] = mine + (unsigned)__popcll(keep[k] & lanes_below(lane));
            mine += (unsigned)__popcll(keep[k]);
        }
        const unsigned sums[2] = {lane == 0 ? mine : 0u, lane == 0 ? lower : 0u};
        unsigned before[2], total[2];
        block_excl_scan_n<W, 2>(sums, wsum, before, total);
        // the wavefront's first lane holds what the wavefronts before it keep
        const unsigned base = (unsigned)__builtin_amdgcn_readfirstlane((int)before[0]);
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (keep[k] >> lane & 1) local[base + rank[k]] = make_uint2(pair[k].x - lo, pair[k].y);
        n = (int)total[0];
        lower = total[1];
    }
    __syncthreads();
    const int per = (n + kSmallBlock - 1) / kSmallBlock;
    const int first = wave * (per * kWave) + lane;
    int shift = 0;
    for (int q = 0; q < passes; ++q) {
        const int bits = (bits_all - shift + passes - q - 1) / (passes - q);
        const int digits = 1 << bits;
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (k < per && first + k * kWave < n) pair[k] = local[first + k * kWave];
        for (int d = threadIdx.x; d < W * kMaxDigits / 2; d += kSmallBlock)
            ((unsigned*)&seen[0][0])[d] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < E; ++k) {
            if (k < per) {
                const bool valid = first + k * kWave < n;
                const unsigned d = (pair[k].x >> shift) & (digits - 1);
                const unsigned long long m = match_mask(d, valid, bits);
                const unsigned before = valid ? seen[wave][d] : 0u;
                rank[k] = before + (unsigned)__popcll(m & lanes_below(lane));
                if (valid && (m & lanes_above(lane)) == 0)
                    seen[wave][d] = (unsigned short)(before + (unsigned)__popcll(m));
                asm volatile("" ::: "memory");
            }
        }
        __syncthreads();
        {
            static_assert(kMaxDigits <= kSmallBlock, "a digit per thread");
            const int d = threadIdx.x;
            unsigned c[W], sum = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                c[w] = d < digits ? seen[w][d] : 0u;
                sum += c[w];
            }
            unsigned total;
            unsigned at = block_excl_scan<W>(sum, wsum, &total);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (d < digits) seen[w][d] = (unsigned short)at;  // < kSmall
                at += c[w];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < E; ++k) {
            if (k < per && first + k * kWave < n)
                local[seen[wave][(pair[k].x >> shift) & (digits - 1)] + rank[k]] = pair[k];
        }
        __syncthreads();
        shift += bits;
    }
    for (int i = threadIdx.x; i < n; i += kSmallBlock)
        out_pairs[lower + i] = make_uint2(local[i].x + lo, local[i].y);
}

// n <= kTiny tokens in one launch: the first `sums` blocks have a wavefront per
// token, which adds the rows of its id if it is the id's first token; the
// others clear the rows that no token has, kTinyRows each.
constexpr int kTiny = 256, kTinyRows = 64;

template <typename T, int N, typename Id>
__global__ __launch_bounds__(kBlock) void k_eg_tiny(const T* __restrict__ grad, long long stride,
                                                    const Id* __restrict__ ids, int n, long long rows,
                                                    int width, float scale, T* __restrict__ out,
                                                    int sums, int lanes_log) {
    static_assert(kTiny <= kBlock && kTiny % kWave == 0, "an id per thread");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int)blockIdx.x < sums) {
        const int token = blockIdx.x * kWaves + wave;
        if (token >= n) return;
        const unsigned key = key_of(ids, token, rows);
        if (key >= rows) return;
        unsigned long long same[kTiny / kWave];
#pragma unroll
        for (int j = 0; j < kTiny / kWave; ++j) {
            const int i = j * kWave + lane;
            same[j] = __ballot(i < n && key_of(ids, i < n ? i : 0, rows) == key);
        }
        for (int col = lane * N; col < width; col += kWave * N) {
            float acc[N];
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.0f;
            bool first = true;
#pragma unroll
            for (int j = 0; j < kTiny / kWave; ++j) {
                unsigned long long m = same[j];
                while (m) {
                    int at[kBatch];
                    int count = 0;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        at[k] = m ? j * kWave + __ffsll((long long)m) - 1 : at[k > 0 ? k - 1 : 0];
                        count += m != 0;
                        m &= m - 1;
                    }
                    if (first && at[0] != token) return;  // not the id's first token
                    first = false;
                    typename Pack<T, N>::vec x[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        x[k] = Pack<T, N>::raw(grad + (long long)at[k] * stride + col);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        float y[N];
                        Pack<T, N>::wide(x[k], y);
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[i] += k < count ? y[i] : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= scale;
            Pack<T, N>::store(out + (long long)key * width + col, acc);
        }
        return;
    }
    __shared__ int taken[kTinyRows];
    if (threadIdx.x < kTinyRows) taken[threadIdx.x] = 0;
    __syncthreads();
    const long long row0 = (long long)((int)blockIdx.x - sums) * kTinyRows;
    if ((int)threadIdx.x < n) {
        const long long at = (long long)key_of(ids, threadIdx.x, rows) - row0;
        if (at >= 0 && at < kTinyRows) taken[at] = 1;
    }
    __syncthreads();
    float zero[N];
#pragma unroll
    for (int j = 0; j < N; ++j) zero[j] = 0.0f;
    for (int r = threadIdx.x >> lanes_log; r < kTinyRows && row0 + r < rows; r += kBlock >> lanes_log) {
        if (taken[r]) continue;
        for (int col = (threadIdx.x & ((1 << lanes_log) - 1)) * N; col < width; col += N << lanes_log)
            Pack<T, N>::store(out + (row0 + r) * width + col, zero);
    }
}

struct Sums {
    const uint2* pairs;   // sorted
    long long n;
    unsigned rows;
    int width, run;       // run: pairs per run, a multiple of kBatch
    int lanes_log;        // lanes of a group
    float scale;
    float* head;          // [runs, width]: of a row that began in an earlier run
    float* tail;          // [runs, width]: of a row that goes on in the next one
};

constexpr unsigned kNone = 0xffffffffu;

// A group of lanes per run and slab of columns: lane l of the group holds
// columns N l .. N l + N - 1. Bound by memory: 2,097,152 rows of 64 bf16, each
// 128 bytes from anywhere, in 56 us, 4.9 TB/s; eight rows under way in a group.
template <typename T, int N>
__global__ __launch_bounds__(kBlock) void k_eg_reduce(const T* __restrict__ grad, long long stride,
                                                      Sums a, T* __restrict__ out) {
    const int tid = blockIdx.x * kBlock + threadIdx.x;
    const long long run = tid >> a.lanes_log;
    const long long p0 = run * a.run;
    if (p0 >= a.n) return;
    const int count = (int)(a.n - p0 < a.run ? a.n - p0 : (long long)a.run);
    const int col = ((blockIdx.y << a.lanes_log) + (tid & ((1 << a.lanes_log) - 1))) * N;
    if (col >= a.width) return;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    bool cut = p0 > 0 && a.pairs[p0 - 1].x == a.pairs[p0].x;  // began in an earlier run
    for (int b = 0; b < count; b += kBatch) {
        uint2 pr[kBatch + 1];
#pragma unroll
        for (int k = 0; k <= kBatch; ++k) {
            const long long p = p0 + b + k;
            pr[k] = p < a.n ? a.pairs[p] : make_uint2(kNone, 0);
        }
        if (pr[0].x >= a.rows) break;  // no row, and so is what follows
        typename Pack<T, N>::vec x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            x[k] = Pack<T, N>::raw(grad + (long long)(pr[k].x < a.rows ? pr[k].y : pr[0].y) * stride + col);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const unsigned key = pr[k].x;
            if (key < a.rows && b + k < count) {
                float y[N];
                Pack<T, N>::wide(x[k], y);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += y[j];
                const bool open = b + k + 1 == a.run && pr[k + 1].x == key;
                if (pr[k + 1].x != key || open) {
                    if (!cut && !open) {
#pragma unroll
                        for (int j = 0; j < N; ++j) y[j] = acc[j] * a.scale;
                        Pack<T, N>::store(out + (long long)key * a.width + col, y);
                    } else {
                        Pack<float, N>::store((cut ? a.head : a.tail) + run * a.width + col, acc);
                    }
                    cut = false;
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
                }
            }
        }
    }
}

// Sum of heads [r0, r1) in order.
template <int N>
__device__ __forceinline__ void add_heads(const Sums& a, long long r0, long long r1, int col,
                                          float (&acc)[N]) {
    for (long long r = r0; r < r1; r += kBatch) {
        float x[kBatch][N];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long q = r + k < r1 ? r + k : r1 - 1;
            Pack<float, N>::load(a.head + q * a.width + col, x[k]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += r + k < r1 ? x[k][j] : 0.0f;
    }
}

// A group of lanes per run whose last row began in it and goes on in the next.
// Rows of more than kLong runs are summed by all groups of the block, each a
// share of the runs, and the shares in order.
template <typename T, int N>
__global__ __launch_bounds__(kBlock) void k_eg_join(Sums a, T* __restrict__ out) {
    constexpr int kLong = 32;
    __shared__ long long list[kBlock][2];
    __shared__ int listed;
    __shared__ float part[kBlock][N];
    if (threadIdx.x == 0) listed = 0;
    __syncthreads();
    const int lanes = 1 << a.lanes_log, groups = kBlock >> a.lanes_log;
    const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> a.lanes_log;
    const long long run = (long long)blockIdx.x * groups + group;
    const long long runs = (a.n + a.run - 1) / a.run;
    const long long p1 = (run + 1) * a.run;  // the next run's first pair
    const int col = ((blockIdx.y << a.lanes_log) + lane) * N;
    const bool on = col < a.width;
    auto first_key = [&](long long r) { return r < runs ? a.pairs[r * a.run].x : kNone; };
    if (p1 < a.n) {
        const unsigned key = a.pairs[p1].x;
        const long long p0 = run * a.run;
        const bool began = !(a.pairs[p0].x == key && p0 > 0 && a.pairs[p0 - 1].x == key);
        if (key < a.rows && a.pairs[p1 - 1].x == key && began) {
            // heads [run + 1, end): runs that start with the row
            long long end = run + 2, step = 1;
            while (first_key(end + step - 1) == key) end += step, step *= 2;
            while (step > 1) {
                step /= 2;
                if (first_key(end + step - 1) == key) end += step;
            }
            if (end - run > kLong) {
                if (lane == 0) {
                    const int at = atomicAdd(&listed, 1);
                    list[at][0] = run;
                    list[at][1] = end;
                }
            } else if (on) {
                float acc[N];
                Pack<float, N>::load(a.tail + run * a.width + col, acc);
                add_heads<N>(a, run + 1, end, col, acc);
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] *= a.scale;
                Pack<T, N>::store(out + (long long)key * a.width + col, acc);
            }
        }
    }
    __syncthreads();
    for (int k = 0; k < listed; ++k) {
        const long long from = list[k][0], end = list[k][1], heads = end - from - 1;
        const long long share = (heads + groups - 1) / groups;
        const long long r0 = from + 1 + group * share < end ? from + 1 + group * share : end;
        const long long r1 = r0 + share < end ? r0 + share : end;
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        if (on) {
            if (group == 0) Pack<float, N>::load(a.tail + from * a.width + col, acc);
            add_heads<N>(a, r0, r1, col, acc);
#pragma unroll
            for (int j = 0; j < N; ++j) part[threadIdx.x][j] = acc[j];
        }
        __syncthreads();
        if (on && group == 0) {
            for (int g = 1; g < groups; ++g)
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += part[(g << a.lanes_log) + lane][j];
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= a.scale;
            Pack<T, N>::store(out + (long long)a.pairs[(from + 1) * a.run].x * a.width + col, acc);
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- host --

int fail(hipError_t e) { return e == hipSuccess ? VOX_OK : ssh_hip_fail(e); }

// Elements per piece: the most (16 bytes, at most `most`) that divide the rows
// and that the addresses are aligned for.
int piece(const void* a, const void* b, long long width, long long stride, int bytes, int most) {
    int n = 16 / bytes < most ? 16 / bytes : most;
    while (n > 1 && (width % n || stride % n || (size_t)a % (n * bytes) || (size_t)b % (n * bytes)))
        n /= 2;
    return n;
}

template <typename T, int N, typename Id>
int embed_run(const void* table, long long rows, long long width, long long stride, const void* ids,
              long long n, float scale, void* out, hipStream_t stream) {
    const long long pieces = width / N;
    int lpr_log = 0;
    while ((1 << lpr_log) < pieces && lpr_log < 8) ++lpr_log;
    // Four rows per thread once that leaves eight wavefronts for every SIMD
    // (2,097,152 rows: 77 us a call, with one 91; 97 rows: the same).
    const long long threads = n << lpr_log;
    const int r = threads >= 4ll * 8 * 64 * 1024 ? 4 : 1;
    const long long per = (long long)(kBlock >> lpr_log) * r, slice = most_blocks(kBlock) * per;
    for (long long first = 0; first < n; first += slice) {
        const long long rest = n - first < slice ? n - first : slice;
        const dim3 grid((unsigned)((rest + per - 1) / per)), block(kBlock);
        const Id* from = (const Id*)ids + first;
        T* to = (T*)out + first * width;
        if (r == 4)
            k_embed<T, N, Id, 4><<<grid, block, 0, stream>>>((const T*)table, rows, (int)width, stride, from,
                                                             rest, scale, to, lpr_log);
        else
            k_embed<T, N, Id, 1><<<grid, block, 0, stream>>>((const T*)table, rows, (int)width, stride, from,
                                                             rest, scale, to, lpr_log);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return fail(e);
    }
    return VOX_OK;
}

template <typename T, int N>
int embed_ids(const void* table, long long rows, long long width, long long stride, const void* ids,
              int id_bytes, long long n, float scale, void* out, hipStream_t stream) {
    if (id_bytes == 4)
        return embed_run<T, N, int32_t>(table, rows, width, stride, ids, n, scale, out, stream);
    return embed_run<T, N, int64_t>(table, rows, width, stride, ids, n, scale, out, stream);
}

template <typename T>
int embed_type(const void* table, long long rows, long long width, long long stride,
               const void* ids, int id_bytes, long long n, float scale, void* out,
               hipStream_t stream) {
    switch (piece(table, out, width, stride, sizeof(T), 8)) {
        case 8:
            if constexpr (sizeof(T) == 2)
                return embed_ids<T, 8>(table, rows, width, stride, ids, id_bytes, n, scale, out, stream);
        case 4: return embed_ids<T, 4>(table, rows, width, stride, ids, id_bytes, n, scale, out, stream);
        case 2: return embed_ids<T, 2>(table, rows, width, stride, ids, id_bytes, n, scale, out, stream);
        default: return embed_ids<T, 1>(table, rows, width, stride, ids, id_bytes, n, scale, out, stream);
    }
}

struct GradPlan {
    int passes, bits[4], shift[4];
    int tiles, run;
    long long runs;
    long long pairs[2], counts, totals, head, tail, bytes;  // workspace offsets
};

bool grad_plan(long long n, long long rows, long long width, GradPlan* p) {
    if (n < 0 || n > kMaxN || rows < 1 || rows > kMaxRows || width < 1 || width > kMaxWidth)
        return false;
    int bits = 1;
    while ((rows >> bits) != 0) ++bits;  // keys 0 .. rows
    p->passes = (bits + kMaxBits - 1) / kMaxBits;
    int at = 0;
    for (int q = 0; q < p->passes; ++q) {
        p->bits[q] = (bits - at + p->passes - q - 1) / (p->passes - q);
        p->shift[q] = at;
        at += p->bits[q];
    }
    p->tiles = (int)((n + kTile - 1) / kTile);
    // few tokens: short runs, or too few groups of lanes have work (12,000
    // tokens: 5.4 us with runs of 8, 11.3 with 32; 2 M: 56 with 64, 59 with 128)
    p->run = n <= kSmall ? 8 : n <= 262144 ? 32 : 64;
    p->runs = (n + p->run - 1) / p->run;
    long long o = 0;
    auto take = [&](long long bytes) {
        const long long here = o;
        o += (bytes + 255) / 256 * 256;
        return here;
    };
    if (n <= kTiny) {
        p->bytes = 0;
        return true;
    }
    for (int k = 0; k < 2; ++k) p->pairs[k] = k == 0 || n > kSmall ? take(8 * n) : 0;
    p->counts = n > kSmall ? take(4ll * kMaxDigits * p->tiles) : 0;
    p->totals = n > kSmall ? take(4ll * kMaxDigits) : 0;
    p->head = take(4 * p->runs * width);
    p->tail = take(4 * p->runs * width);
    p->bytes = o < 256 ? 256 : o;
    return true;
}

template <typename Id, bool FIRST>
int sort_pass(const GradPlan& p, int q, const void* ids, long long n, long long rows, char* ws,
              void* out, long long bytes, hipStream_t stream) {
    const uint2* in = (const uint2*)(ws + p.pairs[(q + 1) & 1]);
    uint2* sorted = (uint2*)(ws + p.pairs[q & 1]);
    unsigned* counts = (unsigned*)(ws + p.counts);
    unsigned* totals = (unsigned*)(ws + p.totals);
    const dim3 tiles((unsigned)p.tiles), block(kBlock);
    const long long pieces = bytes / 16, clears = FIRST ? pieces / kBlock + 1 : 0;
    const dim3 count((unsigned)(p.tiles + (clears < 1024 ? clears : 1024)));
    k_eg_count<Id, FIRST><<<count, block, 0, stream>>>(
        (const Id*)ids, in, n, rows, p.shift[q], p.bits[q], p.tiles, counts, (uint4*)out, pieces,
        (unsigned char*)out + pieces * 16, (int)(bytes % 16));
    k_eg_prefix<<<dim3(1u << p.bits[q]), block, 0, stream>>>(counts, p.tiles, totals);
    k_eg_scatter<Id, FIRST><<<tiles, block, 0, stream>>>((const Id*)ids, in, n, rows, p.shift[q],
                                                         p.bits[q], p.tiles, counts, totals, sorted);
    return fail(hipGetLastError());
}

template <typename T, int N>
int reduce_run(const GradPlan& p, const void* grad, long long stride, long long n, long long rows,
               long long width, float scale, void* out, char* ws, hipStream_t stream) {
    Sums a;
    a.pairs = (const uint2*)(ws + p.pairs[n <= kSmall ? 0 : (p.passes - 1) & 1]);
    a.n = n, a.rows = (unsigned)rows, a.width = (int)width, a.run = p.run, a.scale = scale;
    a.head = (float*)(ws + p.head), a.tail = (float*)(ws + p.tail);
    const long long pieces = width / N;
    a.lanes_log = 0;
    while ((1 << a.lanes_log) < pieces && a.lanes_log < 6) ++a.lanes_log;
    const int groups = kBlock >> a.lanes_log;
    const dim3 grid((unsigned)((p.runs + groups - 1) / groups),
                    (unsigned)((pieces + (1 << a.lanes_log) - 1) >> a.lanes_log));
    k_eg_reduce<T, N><<<grid, dim3(kBlock), 0, stream>>>((const T*)grad, stride, a, (T*)out);
    k_eg_join<T, N><<<grid, dim3(kBlock), 0, stream>>>(a, (T*)out);
    return fail(hipGetLastError());
}

template <typename T, int N>
int tiny_run(const void* grad, long long stride, const void* ids, int id_bytes, long long n,
             long long rows, long long width, float scale, void* out, hipStream_t stream) {
    int lanes_log = 0;
    while ((1 << lanes_log) < width / N && lanes_log < 6) ++lanes_log;
    const int sums = (int)((n + kWaves - 1) / kWaves);
    const dim3 grid((unsigned)(sums + (rows + kTinyRows - 1) / kTinyRows)), block(kBlock);
    if (id_bytes == 4)
        k_eg_tiny<T, N, int32_t><<<grid, block, 0, stream>>>((const T*)grad, stride, (const int32_t*)ids,
                                                             (int)n, rows, (int)width, scale, (T*)out,
                                                             sums, lanes_log);
    else
        k_eg_tiny<T, N, int64_t><<<grid, block, 0, stream>>>((const T*)grad, stride, (const int64_t*)ids,
                                                             (int)n, rows, (int)width, scale, (T*)out,
                                                             sums, lanes_log);
    return fail(hipGetLastError());
}

template <typename T>
int grad_type(const GradPlan& p, const void* grad, long long stride, const void* ids, int id_bytes,
              long long n, long long rows, long long width, float scale, void* out, char* ws,
              hipStream_t stream) {
    if (n <= kTiny) {
        switch (piece(grad, out, width, stride, sizeof(T), 8)) {
            case 8:
                if constexpr (sizeof(T) == 2)
                    return tiny_run<T, 8>(grad, stride, ids, id_bytes, n, rows, width, scale, out, stream);
            case 4: return tiny_run<T, 4>(grad, stride, ids, id_bytes, n, rows, width, scale, out, stream);
            case 2: return tiny_run<T, 2>(grad, stride, ids, id_bytes, n, rows, width, scale, out, stream);
            default: return tiny_run<T, 1>(grad, stride, ids, id_bytes, n, rows, width, scale, out, stream);
        }
    }
    const long long bytes = rows * width * (long long)sizeof(T), pieces = bytes / 16;
    unsigned char* tail = (unsigned char*)out + pieces * 16;
    int rc;
    if (n <= kSmall) {
        const long long blocks = pieces / (4 * kSmallBlock) + 1;
        const dim3 grid((unsigned)(kSmallSorts + (blocks < 240 ? blocks : 240)));
        const int share = (int)((rows + kSmallSorts) / kSmallSorts);  // of keys 0 .. rows
        int bits = 0;
        while (((share - 1) >> bits) != 0) ++bits;
        const int passes = (bits + kMaxBits - 1) / kMaxBits;
        if (id_bytes == 4)
            k_eg_small<int32_t><<<grid, dim3(kSmallBlock), 0, stream>>>(
                (const int32_t*)ids, (int)n, rows, share, passes, bits, (uint2*)(ws + p.pairs[0]),
                (uint4*)out, pieces, tail, (int)(bytes % 16));
        else
            k_eg_small<int64_t><<<grid, dim3(kSmallBlock), 0, stream>>>(
                (const int64_t*)ids, (int)n, rows, share, passes, bits, (uint2*)(ws + p.pairs[0]),
                (uint4*)out, pieces, tail, (int)(bytes % 16));
        rc = fail(hipGetLastError());
    } else {
        rc = VOX_OK;
        for (int q = 0; rc == VOX_OK && q < p.passes; ++q) {
            if (q > 0)
                rc = sort_pass<int32_t, false>(p, q, nullptr, n, rows, ws, out, bytes, stream);
            else if (id_bytes == 4)
                rc = sort_pass<int32_t, true>(p, q, ids, n, rows, ws, out, bytes, stream);
            else
                rc = sort_pass<int64_t, true>(p, q, ids, n, rows, ws, out, bytes, stream);
        }
    }
    if (rc != VOX_OK) return rc;
    switch (piece(grad, out, width, stride, sizeof(T), 8)) {
        case 8:
            if constexpr (sizeof(T) == 2)
                return reduce_run<T, 8>(p, grad, stride, n, rows, width, scale, out, ws, stream);
        case 4: return reduce_run<T, 4>(p, grad, stride, n, rows, width, scale, out, ws, stream);
        case 2: return reduce_run<T, 2>(p, grad, stride, n, rows, width, scale, out, ws, stream);
        default: return reduce_run<T, 1>(p, grad, stride, n, rows, width, scale, out, ws, stream);
    }
}

}  // namespace

extern "C" {

int tok_embed(const void* table, int64_t rows, int64_t width, int64_t row_stride, int32_t dtype,
              const void* ids, int32_t id_bytes, int64_t n, float scale, void* out,
              hipStream_t stream) {
    if (!tok_dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8) || n < 0 || n > 0x7fffffffll ||
        rows < 1 || rows > 0x7fffffffll || width < 1 || width > kMaxWidth || row_stride < 0)
        return VOX_EINVAL;
    if (n == 0) return VOX_OK;
    if (!table || !ids || !out) return VOX_EINVAL;
    const int bytes = tok_elem_bytes(dtype);
    if ((size_t)table % bytes || (size_t)out % bytes || (size_t)ids % id_bytes) return VOX_EINVAL;
    if (dtype == TOK_F32)
        return embed_type<float>(table, rows, width, row_stride, ids, id_bytes, n, scale, out, stream);
    if (dtype == TOK_BF16)
        return embed_type<bf16_t>(table, rows, width, row_stride, ids, id_bytes, n, scale, out, stream);
    return embed_type<f16_t>(table, rows, width, row_stride, ids, id_bytes, n, scale, out, stream);
}

int64_t tok_embed_grad_workspace_bytes(int64_t n, int64_t rows, int64_t width) {
    GradPlan p;
    return grad_plan(n, rows, width, &p) ? p.bytes : VOX_EINVAL;
}

int tok_embed_grad(const void* grad, int64_t grad_stride, int32_t dtype, const void* ids,
                   int32_t id_bytes, int64_t n, int64_t rows, int64_t width, float scale,
                   void* out, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    GradPlan p;
    if (!tok_dtype_ok(dtype) || (id_bytes != 4 && id_bytes != 8) || grad_stride < 0 ||
        !grad_plan(n, rows, width, &p))
        return VOX_EINVAL;
    if (!out || (n && (!grad || !ids))) return VOX_EINVAL;
    const int bytes = tok_elem_bytes(dtype);
    if ((size_t)grad % bytes || (size_t)out % 16 || (size_t)ids % id_bytes) return VOX_EINVAL;
    if (!workspace_ok(workspace, workspace_bytes, p.bytes)) return VOX_EWORKSPACE;
    char* ws = (char*)workspace;
    if (dtype == TOK_F32)
        return grad_type<float>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
    if (dtype == TOK_BF16)
        return grad_type<bf16_t>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
    return grad_type<f16_t>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
}

}  // extern "C"
