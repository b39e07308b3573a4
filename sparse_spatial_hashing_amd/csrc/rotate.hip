// Rotary positions (tokens.h): pairs of a head's elements turned by a position
// times a frequency.
//
// Bound by memory: every element is read and written once. A thread takes one
// piece of a token (16 bytes where the sizes allow it, or two pieces of as much
// that hold the two halves of its pairs), computes the angles' sines and cosines
// and turns a head or two of the token with them (122,880 tokens of 10 heads of 128 in
// bf16: 113 us, 5.6 TB/s, where a large copy reaches 5.2; with 1, 3 or 10 heads 161, 118 and 130).

#include <hip/hip_runtime.h>

#include "token_ops.h"

int ssh_hip_fail(hipError_t e);  // records the error for vox_last_hip_error()

namespace {

constexpr long long kMaxTokens = (1ll << 31) - 1;
constexpr int kThreads = 256;
constexpr int kHeads = 2;  // of a thread, at most

struct RotateArgs {
    const void* x;
    const int* pos;
    const double* freqs;  // [axes, pairs], radians
    void* out;
    long long x_st, x_sh, pos_st, pos_sa;
    long long items;      // threads of work: tokens * head groups * units
    unsigned first_block;
    int heads, width, axes, pairs;
    int units;            // pieces of a token's head
    int turned_units;     // of them, those with pairs
    int per, groups;      // heads of a thread, and how many threads share a piece
    int step, gap;        // elements from a pair to the next, and between its two
    float sign;           // -1: turned back
};

// The sine and cosine of pos * freq. In turns, of which the whole part is taken off exactly: with what
// the two products' roundings to 64 bits leave, the rest is right to 2^-25 of a turn for any position
// and frequency of less than 2^52 turns. (Their roundings alone: 2^-23.6 at 2^31 radians, 2^-20.5 at ten
// times as many.)
__device__ __forceinline__ void angle(const RotateArgs& a, int pos, int axis, int pair, float& sn, float& cs) {
    constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;  // 1 / (2 pi)
    const double freq = a.freqs[(long long)axis * a.pairs + pair], at = pos;
    const double step = freq * kTurn, step_rest = __builtin_fma(freq, kTurn, -step) + freq * kTurnRest;
    const double turns = step * at, turns_rest = __builtin_fma(step, at, -turns) + step_rest * at;
    const float part = (float)(turns - rint(turns) + turns_rest);
    sincospif(2.0f * part, &sn, &cs);
    sn *= a.sign;
}

// V elements at a time. INTER: pairs are neighbours (V / 2 pairs of a piece);
// else the pairs' two elements lie a gap apart (V pairs of two pieces, or one
// pair of either layout).
template <typename T, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void k_rotate(RotateArgs a) {
    constexpr int P = INTER ? V / 2 : V;  // pairs of a unit
    const long long item = ((long long)a.first_block + blockIdx.x) * kThreads + threadIdx.x;
    if (item >= a.items) return;
    const int unit = (int)(item % a.units);
    const long long rest = item / a.units;
    const int group = (int)(rest % a.groups);
    const long long token = rest / a.groups;
    const int h0 = group * a.per, h1 = min(a.heads, h0 + a.per);
    const T* x = (const T*)a.x + token * a.x_st;
    T* out = (T*)a.out + token * a.heads * a.width;
    constexpr int kAhead = kHeads;  // all loads are under way together

    if (unit >= a.turned_units) {  // past the part that is turned
        const int at = 2 * a.axes * a.pairs + (unit - a.turned_units) * V;
        for (int h = h0; h < h1; h += kAhead) {
            typename Pack<T, V>::vec v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) v[j] = Pack<T, V>::raw(x + min(h + j, h1 - 1) * a.x_sh + at);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (h + j < h1) *(typename Pack<T, V>::vec*)(out + (long long)(h + j) * a.width + at) = v[j];
        }
        return;
    }
    const int of_axis = a.pairs / P;
    const int axis = unit / of_axis, pair = (unit - axis * of_axis) * P;
    const int pos = a.pos[token * a.pos_st + axis * a.pos_sa];
    float sn[P], cs[P];
#pragma unroll
    for (int j = 0; j < P; ++j) angle(a, pos, axis, pair + j, sn[j], cs[j]);
    if constexpr (INTER) {
        const int at = 2 * (axis * a.pairs + pair);
        for (int h = h0; h < h1; h += kAhead) {
            typename Pack<T, V>::vec v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) v[j] = Pack<T, V>::raw(x + min(h + j, h1 - 1) * a.x_sh + at);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (h + j >= h1) break;
                float f[V], r[V];
                Pack<T, V>::wide(v[j], f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    r[2 * i] = f[2 * i] * cs[i] - f[2 * i + 1] * sn[i];
                    r[2 * i + 1] = f[2 * i] * sn[i] + f[2 * i + 1] * cs[i];
                }
                Pack<T, V>::store(out + (long long)(h + j) * a.width + at, r);
            }
        }
    } else {
        const int at = 2 * axis * a.pairs + pair * a.step;
        for (int h = h0; h < h1; h += kAhead) {
            typename Pack<T, V>::vec v[kAhead], w[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const T* from = x + min(h + j, h1 - 1) * a.x_sh + at;
                v[j] = Pack<T, V>::raw(from);
                w[j] = Pack<T, V>::raw(from + a.gap);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (h + j >= h1) break;
                float f[V], g[V], r[V], q[V];
                Pack<T, V>::wide(v[j], f);
                Pack<T, V>::wide(w[j], g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    r[i] = f[i] * cs[i] - g[i] * sn[i];
                    q[i] = f[i] * sn[i] + g[i] * cs[i];
                }
                T* to = out + (long long)(h + j) * a.width + at;
                Pack<T, V>::store(to, r);
                Pack<T, V>::store(to + a.gap, q);
            }
        }
    }
}

template <typename T, int V, bool INTER>
int launch(RotateArgs a, long long tokens, hipStream_t stream) {
    a.turned_units = a.axes * a.pairs / (INTER ? V / 2 : V);
    a.units = a.turned_units + (a.width - 2 * a.axes * a.pairs) / V;
    // An angle is computed once for two heads: 122,880 tokens of 10 heads of 128 take 113 us
    // (5.6 TB/s), 161 with a head each (the angles' instructions bound it), 118 with three
    // and 130 with all ten (a wavefront then reads far apart). One head while that fills
    // the card.
    a.per = tokens * a.units * ((a.heads + 1) / 2) < 65536 ? 1 : a.heads < kHeads ? a.heads : kHeads;
    a.groups = (a.heads + a.per - 1) / a.per;
    a.items = tokens * a.groups * a.units;
    const long long blocks = (a.items + kThreads - 1) / kThreads, most = most_blocks(kThreads);
    for (long long b = 0; b < blocks; b += most) {
        a.first_block = (unsigned)b;
        k_rotate<T, V, INTER><<<dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(kThreads), 0,
                                stream>>>(a);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VOX_OK : ssh_hip_fail(e);
}

// The widest piece, up to 16 bytes, that divides what each side holds of a row.
template <typename T>
int dispatch(const RotateArgs& a, long long tokens, bool interleaved, hipStream_t stream) {
    auto fits = [&](int v) {
        const long long bytes = v * (long long)sizeof(T);
        if ((interleaved ? 2 * a.pairs : a.pairs) % v || (a.width - 2 * a.axes * a.pairs) % v || a.width % v)
            return false;
        return a.x_st % v == 0 && a.x_sh % v == 0 && (size_t)a.x % bytes == 0 && (size_t)a.out % bytes == 0;
    };
    if (interleaved) {
        if (16 / sizeof(T) == 8 && fits(8)) return launch<T, 16 / sizeof(T), true>(a, tokens, stream);
        if (fits(4)) return launch<T, 4, true>(a, tokens, stream);
        if (fits(2)) return launch<T, 2, true>(a, tokens, stream);
        return launch<T, 1, false>(a, tokens, stream);
    }
    if (16 / sizeof(T) == 8 && fits(8)) return launch<T, 16 / sizeof(T), false>(a, tokens, stream);
    if (fits(4)) return launch<T, 4, false>(a, tokens, stream);
    if (fits(2)) return launch<T, 2, false>(a, tokens, stream);
    return launch<T, 1, false>(a, tokens, stream);
}

}  // namespace

extern "C" {

int tok_rotate(const void* x, int64_t tokens, int64_t heads, int64_t width, int64_t token_stride,
               int64_t head_stride, int32_t dtype, const int32_t* pos, int64_t pos_stride,
               int64_t axis_stride, int32_t axes, const double* freqs, int64_t pairs,
               int32_t interleaved, int32_t inverse, void* out, hipStream_t stream) {
    if (!tok_dtype_ok(dtype) || tokens < 0 || tokens > kMaxTokens || heads < 1 || heads > 65536 || width < 1 ||
        width > 65536 || axes < 1 || axes > 3 || pairs < 1 || pairs > width / (2 * axes) || token_stride < 0 ||
        head_stride < 0 || pos_stride < 0 || axis_stride < 0)
        return VOX_EINVAL;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return VOX_EINVAL;
    if (tokens == 0) return VOX_OK;
    if (!x || !pos || !freqs || !out) return VOX_EINVAL;
    if (((size_t)x | (size_t)out) % tok_elem_bytes(dtype) || (size_t)pos % 4 || (size_t)freqs % 8)
        return VOX_EINVAL;
    RotateArgs a = {};
    a.x = x, a.pos = pos, a.freqs = freqs, a.out = out;
    a.x_st = token_stride, a.x_sh = head_stride, a.pos_st = pos_stride, a.pos_sa = axis_stride;
    a.heads = (int)heads, a.width = (int)width, a.axes = axes, a.pairs = (int)pairs;
    a.sign = inverse ? -1.0f : 1.0f;
    a.step = interleaved ? 2 : 1, a.gap = interleaved ? 1 : (int)pairs;
    if (dtype == TOK_F32) return dispatch<float>(a, tokens, interleaved, stream);
    if (dtype == TOK_BF16) return dispatch<bf16_t>(a, tokens, interleaved, stream);
    return dispatch<f16_t>(a, tokens, interleaved, stream);
}

}  // extern "C"
