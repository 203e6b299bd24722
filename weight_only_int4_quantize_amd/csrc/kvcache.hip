// Writing and reading the paged 8-bit key / value cache (include/awq.h).
//
// Write. One block per (page that new tokens fall into, head, side): it alone
// reads and writes that page's codes and scale, so nothing is atomic and the
// result does not depend on scheduling. It takes the maximum of the page's
// new values (as 15-bit integers, whose order is the magnitudes'), sets the
// scale, and quantizes the values on a second pass that the caches serve.
// Old codes are touched only when the scale grew. The kernel is bound by
// memory: 2 bytes read and 1 written per value. Measured: 11776 tokens of 32
// heads of 128, keys and values, 86 us, 289 MB, 3.4 TB/s (a copy reaches
// 4.9); one token of 64 sequences, 8 heads, 4.4 us, a launch's length. Values
// kept in registers between the passes were slower (write and read 167 us
// against 154): the first pass then loads 4 bytes at a time in place of 16.
//
// Keys are stored 16 channels to a piece (a thread's 16-byte store), values
// 16 tokens to a piece: a thread takes two channels of 16 tokens, so its
// loads are one 4-byte pair per token (a wave reads whole rows) and its
// store 32 contiguous bytes. A piece that holds old tokens too is read,
// merged and written whole.
#include <algorithm>

#include "kv_internal.h"

namespace awq {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kWriteThreads = 256;

__device__ inline uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}
// larger magnitude bits of two values; NaN counts as 0, infinity as 65504
__device__ inline uint32_t finite_magnitude(uint32_t h) { return h > 0x7C00u ? 0u : min(h, 0x7BFFu); }
__device__ inline float value_of(half_t h) {
    const float v = static_cast<float>(h);
    return v == v ? v : 0.f;
}

template <int FORMAT>
__global__ __launch_bounds__(kWriteThreads) void kv_write_kernel(KvWriteArgs a) {
    constexpr float kTop = FORMAT == AWQ_KV_INT8 ? kInt8Top : kE4m3Top;
    // a byte of value 0
    constexpr uint32_t kZero = FORMAT == AWQ_KV_INT8 ? 0x80u : 0u;
    __shared__ uint32_t s_max[kWriteThreads / kWave];
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int head = blockIdx.y;
    const bool values = blockIdx.z & 1;
    const int b = blockIdx.z >> 1;
    const KvSeq sq = kv_seq(c, b);
    const int lo = max(sq.start, 0);
    if (lo >= sq.end()) return;
    const int p = (lo >> c.log2_page) + static_cast<int>(blockIdx.x);
    const int page_tokens = 1 << c.log2_page;
    if ((static_cast<int64_t>(p) << c.log2_page) >= sq.end()) return;
    const int first = p << c.log2_page;
    const int id = kv_page(c, b, p);
    if (id < 0) return;
    const int t0 = max(lo - first, 0), t1 = min(sq.end() - first, page_tokens);   // the page's new tokens
    const int D = a.head_dim;
    const int64_t token_stride = values ? a.v_token : a.k_token;
    // row of the page's token 0 (rows before t0 are not read)
    const half_t* x = (values ? a.v + head * a.v_head : a.k + head * a.k_head) +
                      (static_cast<int64_t>(sq.row0) + first - sq.start) * token_stride;
    const int64_t block = static_cast<int64_t>(id) * c.heads + head;
    uint8_t* codes = (values ? c.v_codes : c.k_codes) + block * (static_cast<int64_t>(D) << c.log2_page);
    float* scale = (values ? c.v_scales : c.k_scales) + block;

    // ---- largest magnitude of the new tokens ----
    const int per_row = D / 8;
    const int pieces = (t1 - t0) * per_row;
    uint32_t peak = 0;
    for (int i = tid; i < pieces; i += kWriteThreads) {
        const int t = t0 + i / per_row, d8 = i % per_row;
        const kv_u32x4 v = *reinterpret_cast<const kv_u32x4*>(x + t * token_stride + d8 * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) peak = max_u16x2(peak, v[j] & 0x7FFF7FFFu);
    }
    uint32_t top = max(peak & 0xFFFFu, peak >> 16);
    if (top >= 0x7C00u) {       // an infinity or NaN among this thread's: again, finite values only
        top = 0;
        for (int i = tid; i < pieces; i += kWriteThreads) {
            const int t = t0 + i / per_row, d8 = i % per_row;
            const kv_u32x4 v = *reinterpret_cast<const kv_u32x4*>(x + t * token_stride + d8 * 8);
            for (int j = 0; j < 4; ++j)
                top = max(top, max(finite_magnitude(v[j] & 0x7FFFu), finite_magnitude((v[j] >> 16) & 0x7FFFu)));
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
    if ((tid & 63) == 0) s_max[tid >> 6] = top;
    const float old = t0 > 0 ? *scale : 0.f;
    __syncthreads();            // every thread has read the old scale
    top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
    const float put = fmaxf(static_cast<float>(__builtin_bit_cast(half_t, static_cast<uint16_t>(top))), kRangeFloor) /
                      kTop;
    const float s = t0 > 0 ? fmaxf(old, put) : put;
    const bool grown = t0 > 0 && s > old;
    const float inv = 1.0f / s;
    const float shrink = old * inv;
    if (tid == 0) *scale = s;

    auto again = [&](uint32_t w) {      // four old codes at the new scale
        half2_t h0, h1;
        kv_unpack4<FORMAT>(w, h0, h1);
        return kv_pack4<FORMAT>(static_cast<float>(h0[0]) * shrink, static_cast<float>(h0[1]) * shrink,
                                static_cast<float>(h1[0]) * shrink, static_cast<float>(h1[1]) * shrink);
    };

    if (!values) {
        const int chunks = D / 16;
        kv_u32x4* out = reinterpret_cast<kv_u32x4*>(codes);     // [chunk][token]
        for (int i = tid; i < (t1 - t0) * chunks; i += kWriteThreads) {
            const int t = t0 + i / chunks, ch = i % chunks;
            const half_t* src = x + t * token_stride + ch * 16;
            const half8_t v0 = *reinterpret_cast<const half8_t*>(src);
            const half8_t v1 = *reinterpret_cast<const half8_t*>(src + 8);
            kv_u32x4 w;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w[j] = kv_pack4<FORMAT>(value_of(v0[4 * j]) * inv, value_of(v0[4 * j + 1]) * inv,
                                        value_of(v0[4 * j + 2]) * inv, value_of(v0[4 * j + 3]) * inv);
                w[2 + j] = kv_pack4<FORMAT>(value_of(v1[4 * j]) * inv, value_of(v1[4 * j + 1]) * inv,
                                            value_of(v1[4 * j + 2]) * inv, value_of(v1[4 * j + 3]) * inv);
            }
            out[ch * page_tokens + t] = w;
        }
        if (grown) {
            for (int i = tid; i < t0 * chunks; i += kWriteThreads) {
                const int t = i / chunks, ch = i % chunks;
                kv_u32x4 w = out[ch * page_tokens + t];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = again(w[j]);
                out[ch * page_tokens + t] = w;
            }
        }
        return;
    }
    const int pairs = D / 2;
    kv_u32x4* out = reinterpret_cast<kv_u32x4*>(codes);         // [token chunk][channel]
    const int c0 = grown ? 0 : t0 / 16, c1 = (t1 + 15) / 16;
    for (int i = tid; i < (c1 - c0) * pairs; i += kWriteThreads) {
        const int ch = c0 + i / pairs, d = (i % pairs) * 2;
        kv_u32x4 w[2];
        const bool held = ch * 16 < t0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w[e] = kv_u32x4{kZero * 0x01010101u, kZero * 0x01010101u, kZero * 0x01010101u, kZero * 0x01010101u};
            if (held) {
                w[e] = out[ch * D + d + e];
                if (grown) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[e][j] = again(w[e][j]);
                }
            }
        }
        half2_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int t = ch * 16 + j;
            v[j] = half2_t{static_cast<half_t>(0.f), static_cast<half_t>(0.f)};
            if (t >= t0 && t < t1) v[j] = *reinterpret_cast<const half2_t*>(x + t * token_stride + d);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t n = kv_pack4<FORMAT>(value_of(v[4 * j][e]) * inv, value_of(v[4 * j + 1][e]) * inv,
                                                    value_of(v[4 * j + 2][e]) * inv, value_of(v[4 * j + 3][e]) * inv);
                // the old tokens' bytes of this word stay
                const int keep = min(max(t0 - (ch * 16 + 4 * j), 0), 4);
                const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
                w[e][j] = (w[e][j] & mask) | (n & ~mask);
            }
        }
        out[ch * D + d] = w[0];
        out[ch * D + d + 1] = w[1];
    }
}

// Read: one block per (page, head, side) of the tokens asked for; 1 byte read
// and 2 written per value, by the same pieces as the write. The 11776 tokens
// above in 65 us, 4.5 TB/s.
template <int FORMAT>
__global__ __launch_bounds__(kWriteThreads) void kv_read_kernel(KvReadArgs a) {
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int head = blockIdx.y;
    const bool values = blockIdx.z & 1;
    const int b = blockIdx.z >> 1;
    half_t* y = values ? a.v : a.k;
    if (y == nullptr) return;
    const KvSeq sq = kv_seq(c, b);
    const int D = a.head_dim;
    const int64_t token_stride = static_cast<int64_t>(c.heads) * D;
    // row of position 0
    y += head * static_cast<int64_t>(D) + (static_cast<int64_t>(sq.row0) - sq.start) * token_stride;
    const int lo = max(sq.start, 0);
    const kv_u32x4 zero = {0u, 0u, 0u, 0u};
    if (blockIdx.x == 0 && sq.start < 0) {      // rows at positions below 0
        for (int64_t i = tid; i < static_cast<int64_t>(min(-sq.start, sq.n)) * (D / 8); i += kWriteThreads)
            *reinterpret_cast<kv_u32x4*>(y + (sq.start + i / (D / 8)) * token_stride + i % (D / 8) * 8) = zero;
    }
    if (lo >= sq.end()) return;
    const int p = (lo >> c.log2_page) + static_cast<int>(blockIdx.x);
    if ((static_cast<int64_t>(p) << c.log2_page) >= sq.end()) return;
    const int page_tokens = 1 << c.log2_page;
    const int first = p << c.log2_page;
    const int t0 = max(lo - first, 0), t1 = min(sq.end() - first, page_tokens);
    y += first * token_stride;
    const int id = kv_page(c, b, p);
    if (id < 0) {
        for (int i = tid; i < (t1 - t0) * (D / 8); i += kWriteThreads)
            *reinterpret_cast<kv_u32x4*>(y + (t0 + i / (D / 8)) * token_stride + i % (D / 8) * 8) = zero;
        return;
    }
    const int64_t block = static_cast<int64_t>(id) * c.heads + head;
    const kv_u32x4* codes = reinterpret_cast<const kv_u32x4*>((values ? c.v_codes : c.k_codes) +
                                                              block * (static_cast<int64_t>(D) << c.log2_page));
    const float s = (values ? c.v_scales : c.k_scales)[block];
    if (!values) {
        const int chunks = D / 16;
        for (int i = tid; i < (t1 - t0) * chunks; i += kWriteThreads) {
            const int t = t0 + i / chunks, ch = i % chunks;
            const kv_u32x4 w = codes[ch * page_tokens + t];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const half8_t q = kv_unpack8<FORMAT>(w[2 * h], w[2 * h + 1]);
                half8_t r;
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = static_cast<half_t>(static_cast<float>(q[j]) * s);
                *reinterpret_cast<half8_t*>(y + t * token_stride + ch * 16 + h * 8) = r;
            }
        }
        return;
    }
    const int pairs = D / 2;
    const int c0 = t0 / 16, c1 = (t1 + 15) / 16;
    for (int i = tid; i < (c1 - c0) * pairs; i += kWriteThreads) {
        const int ch = c0 + i / pairs, d = (i % pairs) * 2;
        const kv_u32x4 w0 = codes[ch * D + d], w1 = codes[ch * D + d + 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const half8_t q0 = kv_unpack8<FORMAT>(w0[2 * h], w0[2 * h + 1]);
            const half8_t q1 = kv_unpack8<FORMAT>(w1[2 * h], w1[2 * h + 1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = ch * 16 + h * 8 + j;
                if (t >= t0 && t < t1)
                    *reinterpret_cast<half2_t*>(y + t * token_stride + d) =
                        half2_t{static_cast<half_t>(static_cast<float>(q0[j]) * s),
                                static_cast<half_t>(static_cast<float>(q1[j]) * s)};
            }
        }
    }
}

// Blocks along x: the pages that max_tokens consecutive tokens can touch, at
// most a sequence's. One also where a sequence has none: the read's first
// block zeroes the rows at positions below 0.
int64_t touched_pages(const KvPages& c, int64_t max_tokens) {
    const int64_t page = int64_t{1} << c.log2_page;
    return std::max<int64_t>(1, std::min<int64_t>((max_tokens + page - 2) / page + 1, c.max_pages));
}

// a launch takes 2^32 threads along x
bool launchable(const KvPages& c, int64_t max_tokens) {
    return touched_pages(c, max_tokens) < (int64_t{1} << 32) / kWriteThreads;
}

}  // namespace

awq_status launch_kv_write(const KvWriteArgs& a, hipStream_t stream) {
    if (!launchable(a.c, a.max_tokens)) return AWQ_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(touched_pages(a.c, a.max_tokens)), static_cast<unsigned>(a.c.heads),
                    static_cast<unsigned>(2 * a.n_seqs));
    if (a.format == AWQ_KV_INT8)
        hipLaunchKernelGGL((kv_write_kernel<AWQ_KV_INT8>), grid, dim3(kWriteThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((kv_write_kernel<AWQ_KV_E4M3>), grid, dim3(kWriteThreads), 0, stream, a);
    return last_launch_status();
}

awq_status launch_kv_read(const KvReadArgs& a, hipStream_t stream) {
    if (!launchable(a.c, a.max_tokens)) return AWQ_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(touched_pages(a.c, a.max_tokens)), static_cast<unsigned>(a.c.heads),
                    static_cast<unsigned>(2 * a.n_seqs));
    if (a.format == AWQ_KV_INT8)
        hipLaunchKernelGGL((kv_read_kernel<AWQ_KV_INT8>), grid, dim3(kWriteThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((kv_read_kernel<AWQ_KV_E4M3>), grid, dim3(kWriteThreads), 0, stream, a);
    return last_launch_status();
}

}  // namespace awq
