// Rotary positions of queries and keys (include/awq.h, awq_rope).
//
// Mathematics. Pair (a, b) number i of a head at position p turns by the angle
// p f_i: a' = m (a cos - b sin), b' = m (b cos + a sin). Angles of far
// positions need more bits than fp32 has (2^17 positions times 1 radian leave
// 2^-7): p f_i / 2 pi is taken in fp64 and its whole turns are dropped there;
// what is left, at most half a turn, goes to fp32 (2^-25 turns) and to the
// hardware's sine and cosine, which take turns: within 2^-22.9 of the true
// values over every multiple of 2^-25 turns (measured against fp64). The
// rotation is fp32, rounded once.
//
// Bound by HBM: 2 bytes read and 2 written a number; a call of few tokens by a
// launch's length. A thread keeps one place in the head and goes over the
// token's heads with it, so the angles are computed once for several heads.
// Measured (us): 8192 tokens, 32 + 8 heads of 128, 168 MB, 36, 4.6 TB/s (a
// copy reaches 5.2); one token of 32 + 32 heads 2.8.
#include <algorithm>

#include "awq_internal.h"

namespace awq {
namespace {

// One wave: with 256 threads a token's heads left more of them idle (the 8192
// tokens above 39.1 us against 37, with 5 heads 11.6 against 8.3).
constexpr int kThreads = 64;

// N halves at any address that their type allows
template <int N>
struct Run {
    half_t v[N];
};
template <int N>
__device__ inline Run<N> load_run(const half_t* p) {
    typedef half_t vec_t __attribute__((ext_vector_type(N)));
    typedef vec_t any_t __attribute__((aligned(2)));
    return __builtin_bit_cast(Run<N>, static_cast<vec_t>(*reinterpret_cast<const any_t*>(p)));
}
template <>
__device__ inline Run<1> load_run<1>(const half_t* p) {
    return Run<1>{{*p}};
}
template <int N>
__device__ inline void store_run(half_t* p, const Run<N>& r) {
    typedef half_t vec_t __attribute__((ext_vector_type(N)));
    typedef vec_t any_t __attribute__((aligned(2)));
    *reinterpret_cast<any_t*>(p) = __builtin_bit_cast(vec_t, r);
}
template <>
__device__ inline void store_run<1>(half_t* p, const Run<1>& r) {
    *p = r.v[0];
}

// One token per blockIdx.x (of sequence blockIdx.z with BATCH), its heads
// shared out over the blocks along y. A head is `rotated` units of U pairs and
// `passed` units of 2 U channels behind them (none in place); U divides both.
template <bool INTERLEAVED, bool BATCH, int U>
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
    const int units = a.rotated + a.passed;
    const int heads = a.q.heads + a.k.heads;
    // a thread keeps its unit, or its units one after the other, through the heads
    const int lanes = min(units, kThreads);
    const int at_once = kThreads / lanes;       // heads
    const int tid = threadIdx.x;
    if (tid >= at_once * lanes) return;
    for (int u = tid % lanes; u < units; u += lanes) {
        const bool turned = u < a.rotated;
        const int first = U * u;
        // a unit's two runs of U channels; the next head's are on their way while
        // this one's turn
        const int rest = a.rotary + 2 * U * (u - a.rotated);
        const int at0 = !turned ? rest : INTERLEAVED ? 2 * first : first;
        const int at1 = turned && !INTERLEAVED ? a.rotary / 2 + first : at0 + U;
        const bool both = U > 1 || at1 < a.dim;         // false: an odd channel
        const int step = at_once * gridDim.y;
        int head = tid / lanes + blockIdx.y * at_once;
        Run<U> v[2], next[2];
        const auto fetch = [&](int head, Run<U> (&r)[2]) {
            const bool query = head < a.q.heads;
            const half_t* x = query ? a.q.in + row * a.q.in_token + head * a.q.in_head
                                    : a.k.in + row * a.k.in_token + (head - a.q.heads) * a.k.in_head;
            r[0] = load_run<U>(x + at0);
            if (both) r[1] = load_run<U>(x + at1);
        };
        if (head < heads) fetch(head, v);
        float c[U], s[U];
        if (turned) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const double turns = position * (a.freqs[first + j] * 0.15915494309189535);
                const float part = static_cast<float>(turns - __builtin_rint(turns));
                c[j] = a.amplitude * __builtin_amdgcn_cosf(part);
                s[j] = a.amplitude * __builtin_amdgcn_sinf(part);
            }
        }
        for (; head < heads; head += step) {
            if (head + step < heads) fetch(head + step, next);
            if (turned) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    half_t& x0 = INTERLEAVED ? v[2 * j / U].v[2 * j % U] : v[0].v[j];
                    half_t& x1 = INTERLEAVED ? v[(2 * j + 1) / U].v[(2 * j + 1) % U] : v[1].v[j];
                    const float p = static_cast<float>(x0), q = static_cast<float>(x1);
                    x0 = static_cast<half_t>(p * c[j] - q * s[j]);
                    x1 = static_cast<half_t>(q * c[j] + p * s[j]);
                }
            }
            const bool query = head < a.q.heads;
            half_t* y = query ? a.q.out + row * a.q.out_token + head * a.q.out_head
                              : a.k.out + row * a.k.out_token + (head - a.q.heads) * a.k.out_head;
            store_run<U>(y + at0, v[0]);
            if (both) store_run<U>(y + at1, v[1]);
            v[0] = next[0];
            v[1] = next[1];
        }
    }
}

template <int U>
awq_status launch_units(RopeArgs a, int64_t tokens, int n_seqs, hipStream_t stream) {
    a.rotated = a.rotary / 2 / U;
    const bool in_place = (a.q.heads == 0 || a.q.in == a.q.out) && (a.k.heads == 0 || a.k.in == a.k.out);
    a.passed = in_place ? 0 : static_cast<int>(ceil_div(a.dim - a.rotary, 2 * U));
    // few tokens: their heads over several blocks, up to four a CU in all
    const int at_once = std::max(1, kThreads / (a.rotated + a.passed));
    const int64_t passes = ceil_div(static_cast<int64_t>(a.q.heads) + a.k.heads, at_once);
    const int64_t split = std::max<int64_t>(1, std::min<int64_t>(passes, 4 * cu_count() / (tokens * n_seqs)));
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(split), static_cast<unsigned>(n_seqs));
    const bool batch = a.positions == nullptr;
    if (a.interleaved) {
        if (batch) hipLaunchKernelGGL((rope_kernel<true, true, U>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((rope_kernel<true, false, U>), grid, dim3(kThreads), 0, stream, a);
    } else {
        if (batch) hipLaunchKernelGGL((rope_kernel<false, true, U>), grid, dim3(kThreads), 0, stream, a);
        else hipLaunchKernelGGL((rope_kernel<false, false, U>), grid, dim3(kThreads), 0, stream, a);
    }
    return last_launch_status();
}

}  // namespace

// Units of 8, 4, 2 or 1 pairs, the most that divide a head (40 of 80 channels
// rotated, 8192 tokens of 40 heads: 27 us in units of 4, 88 in units of 8 with a
// rest by the element).
awq_status launch_rope(const RopeArgs& a, int64_t tokens, int n_seqs, hipStream_t stream) {
    const int sizes = a.rotary / 2 | (a.dim - a.rotary) / 2 | ((a.dim - a.rotary) % 2 ? 1 : 0);
    if (sizes % 8 == 0) return launch_units<8>(a, tokens, n_seqs, stream);
    if (sizes % 4 == 0) return launch_units<4>(a, tokens, n_seqs, stream);
    if (sizes % 2 == 0) return launch_units<2>(a, tokens, n_seqs, stream);
    return launch_units<1>(a, tokens, n_seqs, stream);
}

}  // namespace awq
