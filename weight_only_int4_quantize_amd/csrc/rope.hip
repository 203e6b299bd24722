// Rotary positions of queries and keys (include/awq.h, awq_rope).
//
// Mathematics. Pair (a, b) number i of a head at position p turns by the angle
// p f_i: a' = m (a cos - b sin), b' = m (b cos + a sin). Angles of far
// positions need more bits than fp32 has (2^17 positions times 1 radian leave
// 2^-7): p f_i / 2 pi is taken in fp64 and its whole turns are dropped there;
// what is left, at most half a turn, goes to fp32 (2^-25 turns) and to the
// compiler's sincospi, within 4 units of the last place. The rotation is fp32,
// rounded once.
//
// Bound by HBM: 2 bytes read and 2 written a number. A thread keeps the eight
// pairs of one place in the head and goes over the token's heads with them, so
// the angles are computed once for several heads.
#include <algorithm>

#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
typedef half_t half16_t __attribute__((ext_vector_type(16)));
typedef half8_t half8_any __attribute__((aligned(2)));
typedef half16_t half16_any __attribute__((aligned(2)));

// n (up to N) halves from p, the rest 0
template <int N, typename V, typename Any>
__device__ inline V load_n(const half_t* p, int n) {
    if (n >= N) return *reinterpret_cast<const Any*>(p);
    V v = {};
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) v[j] = p[j];
    return v;
}
template <int N, typename V, typename Any>
__device__ inline void store_n(half_t* p, int n, V v) {
    if (n >= N) {
        *reinterpret_cast<Any*>(p) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) p[j] = v[j];
}
__device__ inline half8_t load8(const half_t* p, int n) { return load_n<8, half8_t, half8_any>(p, n); }
__device__ inline void store8(half_t* p, int n, half8_t v) { store_n<8, half8_t, half8_any>(p, n, v); }
__device__ inline half16_t load16(const half_t* p, int n) { return load_n<16, half16_t, half16_any>(p, n); }
__device__ inline void store16(half_t* p, int n, half16_t v) { store_n<16, half16_t, half16_any>(p, n, v); }

// One token per blockIdx.x (of sequence blockIdx.z with BATCH), its heads
// shared out over the blocks along y. A head's work is `rotated` units of
// eight pairs and `passed` units of 16 channels behind them (none in place).
template <bool INTERLEAVED, bool BATCH>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
    int64_t row = blockIdx.x;
    int position;
    if constexpr (BATCH) {
        const int b = blockIdx.z;
        const int row0 = min(max(a.cu[b], 0), a.n_tokens);
        const int rows_end = max(a.cu[b + 1], row0);
        row += row0;
        if (row >= min(rows_end, a.n_tokens)) return;
        position = static_cast<int>(min(max(a.len[b], 0), a.max_len) - rows_end + row);
    } else {
        position = a.positions[row];
    }
    const int half_r = a.rotary / 2;
    const int units = a.rotated + a.passed;
    const int heads = a.q.heads + a.k.heads;
    const int step = kThreads * gridDim.y;
    int at = -1;            // the unit whose angles c and s hold
    float c[8], s[8];
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < heads * units; i += step) {
        const int head = i / units, u = i % units;
        const bool query = head < a.q.heads;
        const RopeHeads& t = query ? a.q : a.k;
        const int h = query ? head : head - a.q.heads;
        const half_t* x = t.in + row * t.in_token + h * t.in_head;
        half_t* y = t.out + row * t.out_token + h * t.out_head;
        if (u >= a.rotated) {
            const int d = a.rotary + 16 * (u - a.rotated);
            store16(y + d, a.dim - d, load16(x + d, a.dim - d));
            continue;
        }
        const int first = 8 * u, n = half_r - first;        // pairs of this unit: the first n of 8
        if (at != u) {
            at = u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double turns = position * (a.freqs[first + min(j, n - 1)] * 0.15915494309189535);
                sincospif(2.0f * static_cast<float>(turns - __builtin_rint(turns)), &s[j], &c[j]);
                s[j] *= a.amplitude;
                c[j] *= a.amplitude;
            }
        }
        const auto rotate = [&](half_t x0, half_t x1, int j, half_t& y0, half_t& y1) {
            const float p = static_cast<float>(x0), q = static_cast<float>(x1);
            y0 = static_cast<half_t>(p * c[j] - q * s[j]);
            y1 = static_cast<half_t>(q * c[j] + p * s[j]);
        };
        if constexpr (INTERLEAVED) {
            const half16_t v = load16(x + 2 * first, 2 * n);
            half16_t w;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                half_t y0, y1;
                rotate(v[2 * j], v[2 * j + 1], j, y0, y1);
                w[2 * j] = y0;
                w[2 * j + 1] = y1;
            }
            store16(y + 2 * first, 2 * n, w);
        } else {
            const half8_t v0 = load8(x + first, n), v1 = load8(x + half_r + first, n);
            half8_t w0, w1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                half_t y0, y1;
                rotate(v0[j], v1[j], j, y0, y1);
                w0[j] = y0;
                w1[j] = y1;
            }
            store8(y + first, n, w0);
            store8(y + half_r + first, n, w1);
        }
    }
}

}  // namespace

awq_status launch_rope(const RopeArgs& args, int64_t tokens, int n_seqs, hipStream_t stream) {
    RopeArgs a = args;
    a.rotated = static_cast<int>(ceil_div(a.rotary / 2, 8));
    const bool in_place = (a.q.heads == 0 || a.q.in == a.q.out) && (a.k.heads == 0 || a.k.in == a.k.out);
    a.passed = in_place ? 0 : static_cast<int>(ceil_div(a.dim - a.rotary, 16));
    const int64_t work = static_cast<int64_t>(a.q.heads + a.k.heads) * (a.rotated + a.passed);
    const unsigned split = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(work, kThreads), 1024 / std::max<int64_t>(1, tokens * n_seqs))));
    const dim3 grid(static_cast<unsigned>(tokens), split, static_cast<unsigned>(n_seqs));
    const bool batch = a.positions == nullptr;
    if (a.interleaved) {
        if (batch) hipLaunchKernelGGL((rope_kernel<true, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((rope_kernel<true, false>), grid, dim3(kThreads), 0, stream, a);
    } else {
        if (batch) hipLaunchKernelGGL((rope_kernel<false, true>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((rope_kernel<false, false>), grid, dim3(kThreads), 0, stream, a);
    }
    return last_launch_status();
}

}  // namespace awq
