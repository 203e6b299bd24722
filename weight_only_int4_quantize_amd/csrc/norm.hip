// Root-mean-square norm of a residual stream plus a layer's output, to fp16 or
// to 8 bits with scales (include/awq.h, awq_rmsnorm).
//
// Mathematics. h = x + r, y = h (o + w) / sqrt(mean h^2 + eps). With
// t = h (o + w) the row's one number 1 / sqrt(..) multiplies t, so the largest
// |y| of a row or group is the largest |t| times it, exactly (a rounded product
// keeps the order): the sum of squares and the maxima come from one pass and
// one exchange, and every element is loaded once and stays in registers. All
// of it in fp32; h is rounded to fp16 only for the stored sum, and y is taken
// from h itself.
//
// Bound by HBM: 2 bytes an element of x, r, the sum and y (4096 x 8192, 268 MB:
// 51 us, 5.3 TB/s, a copy's rate; to int8 by rows or to e4m3 by groups of 128, 236 MB,
// 45-47 in a graph), few rows by a launch's length. Rows narrower than 512 leave
// lanes of their wave idle: 327680 x 128 67 us, where a copy takes 32; x 256, half as
// many, 37.
#include "awq_internal.h"

namespace awq {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// eight numbers at any address that their type allows
typedef half8_t half8_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Elements i .. i + 7 of a row of n, those past it 0.
__device__ inline half8_t load8(const half_t* p, int i, int n) {
    if (i + 8 <= n) return *reinterpret_cast<const half8_any*>(p + i);
    half8_t v = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) v[j] = p[i + j];
    return v;
}
__device__ inline void store8(half_t* p, int i, int n, half8_t v) {
    if (i + 8 <= n) {
        *reinterpret_cast<half8_any*>(p + i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) p[i + j] = v[j];
}
__device__ inline void store8(uint8_t* p, int i, int n, u32x2 v) {
    if (i + 8 <= n) {
        *reinterpret_cast<u32x2_any*>(p + i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) p[i + j] = static_cast<uint8_t>(v[j / 4] >> (8 * (j % 4)));
}

// Magnitudes compare as integers, so that a NaN is the largest of them.
__device__ inline uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

template <int FORMAT>
__device__ inline u32x2 pack8(const float (&y)[8], float inv) {
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (FORMAT == AWQ_NORM_INT8) {
            r[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = static_cast<int>(fminf(fmaxf(__builtin_rintf(y[4 * i + j] * inv), -127.f), 127.f));
                r[i] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * j);
            }
        } else {
            const auto q = [&](int j) { return fminf(fmaxf(y[4 * i + j] * inv, -448.f), 448.f); };
            const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q(0), q(1), 0, false);
            r[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q(2), q(3), w, true));
        }
    }
    return r;
}

// A group's scale from the bits of its largest |y|; 1 / scale, or 0 for a group
// with a NaN, whose scale is NaN and whose codes are 0.
template <int FORMAT>
__device__ inline float scale_of(float top, float& inv) {
    const float a = top < kRangeFloor ? kRangeFloor : top;      // a NaN stays
    const float s = a / (FORMAT == AWQ_NORM_INT8 ? 127.0f : 448.0f);
    inv = s == s ? 1.0f / s : 0.f;
    return s;
}

// A value of the lane 1, 2, 4 .. 32 away in some order, by the wave's own moves
// (over LDS the six steps took 0.2 us more of a 2.8 us call).
template <int STEP>
__device__ inline uint32_t moved(uint32_t v) {
    typedef uint32_t swap_t __attribute__((ext_vector_type(2)));
    if constexpr (STEP == 5) {
        const swap_t r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    } else if constexpr (STEP == 4) {
        const swap_t r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return threadIdx.x & 16 ? r[0] : r[1];
    } else {        // neighbours, pairs, halves of eight, halves of sixteen
        constexpr int kControl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
        return static_cast<uint32_t>(
            __builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), kControl, 0xF, 0xF, true));
    }
}

// (sum of squares, largest magnitude) of a row over its TPR threads
struct Stats {
    float sum;
    uint32_t top;
};
template <int STEP = 0>
__device__ inline void across_wave(Stats& v) {
    v.sum += __builtin_bit_cast(float, moved<STEP>(__builtin_bit_cast(uint32_t, v.sum)));
    v.top = max(v.top, moved<STEP>(v.top));
    if constexpr (STEP < 5) across_wave<STEP + 1>(v);
}
template <int TPR>
__device__ inline Stats across(Stats v) {
    across_wave(v);
    if constexpr (TPR > kWave) {
        constexpr int N = TPR / kWave;
        __shared__ float sums[N];
        __shared__ uint32_t tops[N];
        if (threadIdx.x % kWave == 0) {
            sums[threadIdx.x / kWave] = v.sum;
            tops[threadIdx.x / kWave] = v.top;
        }
        __syncthreads();
        v.sum = 0.f;
        v.top = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v.sum += sums[i];
            v.top = max(v.top, tops[i]);
        }
    }
    return v;
}

// rows that need a wave each share a block
constexpr int rows_per_block(int tpr) { return tpr == kWave ? 4 : 1; }

// One row by TPR threads, thread l taking the pieces of eight elements l,
// l + TPR, ..: P of them, in registers; P = 0: any number, and the row is read
// a second time (from the caches, as far as they hold it).
template <int FORMAT, int TPR, int P>
__global__ __launch_bounds__(TPR * rows_per_block(TPR)) void rmsnorm_kernel(NormArgs a) {
    constexpr int PER_BLOCK = rows_per_block(TPR);
    const int l = threadIdx.x % TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * PER_BLOCK + threadIdx.x / TPR;
    if (PER_BLOCK > 1 && row >= a.rows) return;     // whole waves
    const int K = static_cast<int>(a.width);
    const half_t* x = a.x + row * a.x_stride;
    const half_t* r = a.residual ? a.residual + row * a.residual_stride : nullptr;
    half_t* sum = a.sum ? a.sum + row * a.sum_stride : nullptr;
    const int n_pieces = (K + 7) / 8;
    const int group = a.group;                      // channels, 0: the row
    const int group_pieces = group / 8;

    const auto load_h = [&](int i, float (&h)[8]) {
        const half8_t v = load8(x, i, K);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = static_cast<float>(v[j]);
        if (r) {
            const half8_t u = load8(r, i, K);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] += static_cast<float>(u[j]);
        }
    };
    const auto store_sum = [&](int i, const float (&h)[8]) {
        half8_t v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<half_t>(h[j]);
        store8(sum, i, K, v);
    };
    // h becomes h (o + w)
    const auto weigh = [&](int i, float (&h)[8]) {
        if (!a.weight) return;
        const half8_t w = load8(a.weight, i, K);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] *= a.offset + static_cast<float>(w[j]);
    };
    const auto top_of = [](const float (&t)[8], uint32_t top) {
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, magnitude(t[j]));
        return top;
    };
    // t of piece p (this thread's, or past the row: 0) to the output
    const auto finish = [&](int p, float (&t)[8], float inv, float row_inv) {
        if constexpr (FORMAT == AWQ_NORM_F16) {
            if (p >= n_pieces) return;
            half8_t v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = static_cast<half_t>(t[j] * inv);
            store8(static_cast<half_t*>(a.out) + row * a.out_stride, 8 * p, K, v);
        } else {
            if (group) {        // a group's pieces are neighbouring lanes'
                uint32_t top = top_of(t, 0u);
                for (int o = 1; o < group_pieces; o <<= 1)
                    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
                const float s = scale_of<FORMAT>(__builtin_bit_cast(float, top) * inv, row_inv);
                if (p < n_pieces && p % group_pieces == 0) a.scales[row * (K / group) + p / group_pieces] = s;
            }
            if (p >= n_pieces) return;
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] *= inv;
            u32x2 w = pack8<FORMAT>(t, row_inv);
            if (row_inv == 0.f) w = u32x2{0u, 0u};
            store8(static_cast<uint8_t*>(a.out) + row * a.out_stride, 8 * p, K, w);
        }
    };
    const auto inverse = [&](float squares) {
        return __builtin_amdgcn_rsqf(__builtin_fmaf(squares, a.per_width, a.eps));
    };
    const auto row_scale = [&](uint32_t top, float inv) {
        float row_inv = 0.f;
        if constexpr (FORMAT != AWQ_NORM_F16) {
            if (!group) {
                const float s = scale_of<FORMAT>(__builtin_bit_cast(float, top) * inv, row_inv);
                if (l == 0) a.scales[row] = s;
            }
        }
        return row_inv;
    };

    Stats st = {0.f, 0u};
    if constexpr (P > 0) {
        float t[P][8];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int p = l + i * TPR;
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][j] = 0.f;
            if (p < n_pieces) {
                load_h(8 * p, t[i]);
                if (sum) store_sum(8 * p, t[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) st.sum = __builtin_fmaf(t[i][j], t[i][j], st.sum);
                weigh(8 * p, t[i]);
                if (FORMAT != AWQ_NORM_F16) st.top = top_of(t[i], st.top);
            }
        }
        st = across<TPR>(st);
        const float inv = inverse(st.sum);
        const float row_inv = row_scale(st.top, inv);
#pragma unroll
        for (int i = 0; i < P; ++i) finish(l + i * TPR, t[i], inv, row_inv);
    } else {
        float t[8];
        for (int p = l; p < n_pieces; p += TPR) {
            load_h(8 * p, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) st.sum = __builtin_fmaf(t[j], t[j], st.sum);
            if (FORMAT != AWQ_NORM_F16 && !group) {
                weigh(8 * p, t);
                st.top = top_of(t, st.top);
            }
        }
        st = across<TPR>(st);
        const float inv = inverse(st.sum);
        const float row_inv = row_scale(st.top, inv);
        // (every lane takes part in a group's exchange)
        for (int p = l; p - l < n_pieces; p += TPR) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = 0.f;
            if (p < n_pieces) {
                load_h(8 * p, t);
                if (sum) store_sum(8 * p, t);
                weigh(8 * p, t);
            }
            finish(p, t, inv, row_inv);
        }
    }
}

template <int FORMAT, int TPR, int P>
awq_status launch_p(const NormArgs& a, hipStream_t stream) {
    constexpr int NT = TPR * rows_per_block(TPR);
    const int64_t blocks = ceil_div(a.rows, rows_per_block(TPR));
    if (blocks >= (int64_t{1} << 32) / NT) return AWQ_ERR_SHAPE;      // a launch takes 2^32 threads along x
    hipLaunchKernelGGL((rmsnorm_kernel<FORMAT, TPR, P>), dim3(static_cast<unsigned>(blocks)), dim3(NT), 0, stream, a);
    return last_launch_status();
}
// As many threads to a row as it has pieces of eight, up to 1024: measured with a
// residual and its sum, calls back to back as this rule was made (in a graph 1 x 4096
// takes 2.7, 64 x 8192 e4m3 3.9; us, in brackets with a quarter as many threads and
// four pieces each): 1 x 4096 2.8 (4.4), 1 x 8192 3.3 (4.7), 64 x 8192 e4m3 4.4 (6.0),
// 256 x 4096 3.7 (5.4), 4096 x 8192 50.7 (54.2). Between, 256 threads are some 8%
// better (1024 x 4096 7.8 against 8.5): not worth instances of their own.
template <int FORMAT>
awq_status launch_format(const NormArgs& a, hipStream_t stream) {
    const int64_t pieces = ceil_div(a.width, 8);
    if (pieces <= 64) return launch_p<FORMAT, 64, 1>(a, stream);
    if (pieces <= 128) return launch_p<FORMAT, 128, 1>(a, stream);
    if (pieces <= 256) return launch_p<FORMAT, 256, 1>(a, stream);
    if (pieces <= 512) return launch_p<FORMAT, 512, 1>(a, stream);
    if (pieces <= 1024) return launch_p<FORMAT, 1024, 1>(a, stream);
    if (pieces <= 2048) return launch_p<FORMAT, 1024, 2>(a, stream);
    if (pieces <= 4096) return launch_p<FORMAT, 1024, 4>(a, stream);
    return launch_p<FORMAT, 1024, 0>(a, stream);
}

}  // namespace

awq_status launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
    switch (a.format) {
        case AWQ_NORM_F16: return launch_format<AWQ_NORM_F16>(a, stream);
        case AWQ_NORM_INT8: return launch_format<AWQ_NORM_INT8>(a, stream);
        default: return launch_format<AWQ_NORM_E4M3>(a, stream);
    }
}

}  // namespace awq
