// Embedding lookup and the gradient of its table (tokens.h).
//
// The lookup moves rows in pieces of up to 16 bytes, one lane per piece.
//
// The gradient sorts (row, token) pairs by row with stable passes from the
// lowest digit up, so the tokens of a row come out in token order, and sums
// equal rows over runs of kRun sorted pairs, one wavefront per run:
//   k_eg_count    digits of each tile of pairs, counted
//   k_eg_prefix   one block per digit: where each tile's entries of it start
//   k_eg_scatter  pairs to their places (ranks by ballots, in input order)
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
constexpr int kPer = 16;                   // pairs per thread of a sort tile
constexpr int kTile = kBlock * kPer;
constexpr int kMaxBits = 9;                // bits of a digit, at most
constexpr int kMaxDigits = 1 << kMaxBits;
constexpr int kRun = 64;                   // sorted pairs per wavefront of the reduction
constexpr long long kMaxN = 1ll << 27;
constexpr long long kMaxRows = 1ll << 24;
constexpr long long kMaxWidth = 65536;

// ------------------------------------------------------------------ lookup --

// LPR lanes (a power of two) share a row of `pieces` pieces of N elements.
template <typename T, int N, typename Id>
__global__ __launch_bounds__(kBlock) void k_embed(const T* __restrict__ table, long long rows,
                                                  int width, long long stride,
                                                  const Id* __restrict__ ids, long long n,
                                                  float scale, T* __restrict__ out, int lpr_log) {
    const int lpr = 1 << lpr_log;
    const int pieces = width / N;
    const long long tid = (long long)blockIdx.x * kBlock + threadIdx.x;
    const long long i = tid >> lpr_log;
    if (i >= n) return;
    const long long id = (long long)ids[i];
    const bool in = id >= 0 && id < rows;
    const T* src = table + (in ? id : 0) * stride;
    T* dst = out + i * width;
    for (int p = (int)(tid & (lpr - 1)); p < pieces; p += lpr) {
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = 0.0f;
        if (in) Pack<T, N>::load(src + p * N, x);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = in ? x[j] * scale : 0.0f;
        Pack<T, N>::store(dst + p * N, x);
    }
}

// -------------------------------------------------------------------- sort --

template <typename Id>
__device__ __forceinline__ unsigned key_of(const Id* ids, long long i, long long rows) {
    const long long id = (long long)ids[i];
    return id >= 0 && id < rows ? (unsigned)id : (unsigned)rows;  // rows: no row, sorted last
}

template <typename Id, bool FIRST>
__global__ __launch_bounds__(kBlock) void k_eg_count(const Id* __restrict__ ids,
                                                     const unsigned* __restrict__ keys,
                                                     long long n, long long rows, int shift,
                                                     int bits, int tiles,
                                                     unsigned* __restrict__ counts) {
    __shared__ unsigned hist[kMaxDigits];
    const int digits = 1 << bits;
    for (int d = threadIdx.x; d < digits; d += kBlock) hist[d] = 0;
    __syncthreads();
    const long long base = (long long)blockIdx.x * kTile;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long i = base + k * kBlock + threadIdx.x;
        if (i < n) {
            const unsigned key = FIRST ? key_of(ids, i, rows) : keys[i];
            atomicAdd(&hist[(key >> shift) & (digits - 1)], 1u);
        }
    }
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

template <typename Id, bool FIRST>
__global__ __launch_bounds__(kBlock) void k_eg_scatter(
    const Id* __restrict__ ids, const unsigned* __restrict__ keys,
    const unsigned* __restrict__ tokens, long long n, long long rows, int shift, int bits,
    int tiles, const unsigned* __restrict__ counts, const unsigned* __restrict__ totals,
    unsigned* __restrict__ out_keys, unsigned* __restrict__ out_tokens) {
    __shared__ unsigned wsum[kWsumWords];
    __shared__ unsigned base[kMaxDigits];
    __shared__ unsigned seen[kWaves][kMaxDigits];
    const int digits = 1 << bits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = threadIdx.x; d < kWaves * kMaxDigits; d += kBlock) (&seen[0][0])[d] = 0;
    // where this tile's entries of each digit start
    static_assert(kMaxDigits <= 2 * kBlock, "two digits per thread");
    {
        const int d = 2 * threadIdx.x;
        const unsigned u = d < digits ? totals[d] : 0u, v = d + 1 < digits ? totals[d + 1] : 0u;
        unsigned total;
        const unsigned ex = block_excl_scan<kWaves>(u + v, wsum, &total);
        if (d < digits) base[d] = ex + counts[(long long)d * tiles + blockIdx.x];
        if (d + 1 < digits) base[d + 1] = ex + u + counts[(long long)(d + 1) * tiles + blockIdx.x];
    }
    __syncthreads();
    // wavefront w ranks its kPer * 64 consecutive pairs in order
    const long long first = (long long)blockIdx.x * kTile + wave * (kPer * kWave);
    unsigned key[kPer], rank[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long i = first + k * kWave + lane;
        key[k] = i < n ? (FIRST ? key_of(ids, i, rows) : keys[i]) : 0u;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool valid = first + k * kWave + lane < n;
        const unsigned d = (key[k] >> shift) & (digits - 1);
        const unsigned long long m = match_mask(d, valid, bits);
        const unsigned before = valid ? seen[wave][d] : 0u;
        rank[k] = before + (unsigned)__popcll(m & lanes_below(lane));
        if (valid && (m & lanes_above(lane)) == 0)
            seen[wave][d] = before + (unsigned)__popcll(m);
        // the next pair of any lane reads what the last lane of a digit wrote
        asm volatile("" ::: "memory");
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kBlock) {
        unsigned s = base[d];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const unsigned c = seen[w][d];
            seen[w][d] = s;
            s += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long i = first + k * kWave + lane;
        if (i < n) {
            const unsigned d = (key[k] >> shift) & (digits - 1);
            const unsigned at = seen[wave][d] + rank[k];
            out_keys[at] = key[k];
            out_tokens[at] = FIRST ? (unsigned)i : tokens[i];
        }
    }
}

// ------------------------------------------------------------------ reduce --

__global__ __launch_bounds__(kBlock) void k_eg_zero(uint4* __restrict__ out, long long pieces,
                                                    unsigned char* __restrict__ tail, int bytes) {
    const long long step = (long long)gridDim.x * kBlock;
    for (long long p = (long long)blockIdx.x * kBlock + threadIdx.x; p < pieces; p += step)
        out[p] = make_uint4(0, 0, 0, 0);
    if (blockIdx.x == 0 && (int)threadIdx.x < bytes) tail[threadIdx.x] = 0;
}

// One wavefront per run and slab of 64 * N columns: lane l holds columns
// N l .. N l + N - 1 of the slab.
template <typename T, int N>
__global__ __launch_bounds__(kBlock) void k_eg_reduce(const T* __restrict__ grad, long long stride,
                                                      const unsigned* __restrict__ keys,
                                                      const unsigned* __restrict__ tokens,
                                                      long long n, unsigned rows, int width,
                                                      float scale, T* __restrict__ out,
                                                      float* __restrict__ head,
                                                      float* __restrict__ tail) {
    constexpr int kBatch = 8;
    const int lane = threadIdx.x & 63;
    const long long run = (long long)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const long long p0 = run * kRun;
    if (p0 >= n) return;
    const int count = (int)(n - p0 < kRun ? n - p0 : (long long)kRun);
    const int col = (blockIdx.y * kWave + lane) * N;
    const bool mine = col < width;
    const unsigned my_key = lane < count ? keys[p0 + lane] : rows;
    const unsigned my_token = lane < count ? tokens[p0 + lane] : 0u;
    const unsigned prev = p0 > 0 ? keys[p0 - 1] : 0xffffffffu;
    const unsigned next = p0 + kRun < n ? keys[p0 + kRun] : 0xffffffffu;

    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    bool cut = __builtin_amdgcn_readlane((int)my_key, 0) == (int)prev;  // began in an earlier run
    for (int b = 0; b < kRun; b += kBatch) {
        if (b >= count || __builtin_amdgcn_readlane((int)my_key, b) == (int)rows) break;
        float x[kBatch][N];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const unsigned token = (unsigned)__builtin_amdgcn_readlane((int)my_token, b + k);
#pragma unroll
            for (int j = 0; j < N; ++j) x[k][j] = 0.0f;
            if (mine) Pack<T, N>::load(grad + (long long)token * stride + col, x[k]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int p = b + k;
            const unsigned key = (unsigned)__builtin_amdgcn_readlane((int)my_key, p);
            if (p >= count || key == rows) break;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += x[k][j];
            const unsigned after =
                p + 1 < kRun ? (unsigned)__builtin_amdgcn_readlane((int)my_key, (p + 1) & 63) : next;
            const bool open = p + 1 == kRun && after == key;
            if (after != key || open) {
                if (mine) {
                    if (!cut && !open) {
                        float y[N];
#pragma unroll
                        for (int j = 0; j < N; ++j) y[j] = acc[j] * scale;
                        Pack<T, N>::store(out + (long long)key * width + col, y);
                    } else {
                        Pack<float, N>::store((cut ? head : tail) + run * width + col, acc);
                    }
                }
                cut = false;
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = 0.0f;
            }
        }
    }
}

// One wavefront per run whose last row goes on in the next one and began in it.
template <typename T, int N>
__global__ __launch_bounds__(kBlock) void k_eg_join(const unsigned* __restrict__ keys, long long n,
                                                    unsigned rows, int width, float scale,
                                                    T* __restrict__ out,
                                                    const float* __restrict__ head,
                                                    const float* __restrict__ tail) {
    const int lane = threadIdx.x & 63;
    const long long run = (long long)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const long long p0 = run * kRun;
    if (p0 + kRun >= n) return;
    const unsigned key = keys[p0 + kRun];
    if (key == rows || keys[p0 + kRun - 1] != key) return;
    if (keys[p0] == key && p0 > 0 && keys[p0 - 1] == key) return;  // began earlier
    const int col = (blockIdx.y * kWave + lane) * N;
    const bool mine = col < width;
    const long long runs = (n + kRun - 1) / kRun;
    // runs [run + 1, end) hold more of the row
    long long end = run + 2;
    for (;;) {
        const long long r = end + lane;
        const unsigned long long same = __ballot(r < runs && keys[r * kRun] == key);
        if (same == ~0ull) {
            end += 64;
            continue;
        }
        end += __ffsll((long long)~same) - 1;
        break;
    }
    if (!mine) return;
    float acc[N];
    Pack<float, N>::load(tail + run * width + col, acc);
    for (long long r = run + 1; r < end; r += 8) {
        float x[8][N];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const long long q = r + k < end ? r + k : end - 1;
            Pack<float, N>::load(head + q * width + col, x[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (r + k < end) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += x[k][j];
            }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] *= scale;
    Pack<T, N>::store(out + (long long)key * width + col, acc);
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
    const long long blocks = ((n << lpr_log) + kBlock - 1) / kBlock;
    if (blocks > 0x7fffffffll) return VOX_EINVAL;
    k_embed<T, N, Id><<<dim3((unsigned)blocks), dim3(kBlock), 0, stream>>>(
        (const T*)table, rows, (int)width, stride, (const Id*)ids, n, scale, (T*)out, lpr_log);
    return fail(hipGetLastError());
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
    int tiles;
    long long runs;
    long long keys[2], tokens[2], counts, totals, head, tail, bytes;  // workspace offsets
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
    p->runs = (n + kRun - 1) / kRun;
    long long o = 0;
    auto take = [&](long long bytes) {
        const long long here = o;
        o += (bytes + 255) / 256 * 256;
        return here;
    };
    for (int k = 0; k < 2; ++k) {
        p->keys[k] = take(4 * n);
        p->tokens[k] = take(4 * n);
    }
    p->counts = take(4ll * kMaxDigits * p->tiles);
    p->totals = take(4ll * kMaxDigits);
    p->head = take(4 * p->runs * width);
    p->tail = take(4 * p->runs * width);
    p->bytes = o < 256 ? 256 : o;
    return true;
}

template <typename Id, bool FIRST>
int sort_pass(const GradPlan& p, int q, const void* ids, long long n, long long rows, char* ws,
              hipStream_t stream) {
    const unsigned* ik = (const unsigned*)(ws + p.keys[(q + 1) & 1]);
    const unsigned* it = (const unsigned*)(ws + p.tokens[(q + 1) & 1]);
    unsigned* ok = (unsigned*)(ws + p.keys[q & 1]);
    unsigned* ot = (unsigned*)(ws + p.tokens[q & 1]);
    unsigned* counts = (unsigned*)(ws + p.counts);
    unsigned* totals = (unsigned*)(ws + p.totals);
    const dim3 tiles((unsigned)p.tiles), block(kBlock);
    k_eg_count<Id, FIRST><<<tiles, block, 0, stream>>>((const Id*)ids, ik, n, rows, p.shift[q],
                                                       p.bits[q], p.tiles, counts);
    k_eg_prefix<<<dim3(1u << p.bits[q]), block, 0, stream>>>(counts, p.tiles, totals);
    k_eg_scatter<Id, FIRST><<<tiles, block, 0, stream>>>((const Id*)ids, ik, it, n, rows,
                                                         p.shift[q], p.bits[q], p.tiles, counts,
                                                         totals, ok, ot);
    return fail(hipGetLastError());
}

template <typename T, int N>
int reduce_run(const GradPlan& p, const void* grad, long long stride, long long n, long long rows,
               long long width, float scale, void* out, char* ws, hipStream_t stream) {
    const int last = (p.passes - 1) & 1;
    const unsigned* keys = (const unsigned*)(ws + p.keys[last]);
    const unsigned* tokens = (const unsigned*)(ws + p.tokens[last]);
    float* head = (float*)(ws + p.head);
    float* tail = (float*)(ws + p.tail);
    const dim3 grid((unsigned)((p.runs + kWaves - 1) / kWaves),
                    (unsigned)((width + kWave * N - 1) / (kWave * N)));
    k_eg_reduce<T, N><<<grid, dim3(kBlock), 0, stream>>>((const T*)grad, stride, keys, tokens, n,
                                                         (unsigned)rows, (int)width, scale,
                                                         (T*)out, head, tail);
    k_eg_join<T, N><<<grid, dim3(kBlock), 0, stream>>>(keys, n, (unsigned)rows, (int)width, scale,
                                                       (T*)out, head, tail);
    return fail(hipGetLastError());
}

template <typename T>
int grad_type(const GradPlan& p, const void* grad, long long stride, const void* ids, int id_bytes,
              long long n, long long rows, long long width, float scale, void* out, char* ws,
              hipStream_t stream) {
    const long long bytes = rows * width * (long long)sizeof(T);
    const long long blocks = bytes / (16 * kBlock) + 1;
    k_eg_zero<<<dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(kBlock), 0, stream>>>(
        (uint4*)out, bytes / 16, (unsigned char*)out + bytes / 16 * 16, (int)(bytes % 16));
    int rc = fail(hipGetLastError());
    if (rc != VOX_OK || n == 0) return rc;
    for (int q = 0; q < p.passes; ++q) {
        if (q > 0)
            rc = sort_pass<int32_t, false>(p, q, nullptr, n, rows, ws, stream);
        else if (id_bytes == 4)
            rc = sort_pass<int32_t, true>(p, q, ids, n, rows, ws, stream);
        else
            rc = sort_pass<int64_t, true>(p, q, ids, n, rows, ws, stream);
        if (rc != VOX_OK) return rc;
    }
    // as few elements per lane as leave one slab of columns
    const int most = width <= 64 ? 1 : width <= 128 ? 2 : 4;
    switch (piece(grad, out, width, stride, sizeof(T), most)) {
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
    if (!workspace || ((size_t)workspace & 255) || workspace_bytes < p.bytes) return VOX_EWORKSPACE;
    char* ws = (char*)workspace;
    if (dtype == TOK_F32)
        return grad_type<float>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
    if (dtype == TOK_BF16)
        return grad_type<bf16_t>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
    return grad_type<f16_t>(p, grad, grad_stride, ids, id_bytes, n, rows, width, scale, out, ws, stream);
}

}  // extern "C"
