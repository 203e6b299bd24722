// Writing and reading the paged 4-bit key / value cache (include/awq.h,
// AWQ_KV_INT4).
//
// Mathematics. A group (32 channels of a key, a token's values of a head) is
// stored as its smallest number lo, a step s = the largest fp16 number not
// above (max - lo) / 15, and codes c = clamp(rint((x - lo) / s), 0, 15); the
// cached number is fp16(lo + s c). s is not rounded up so that lo + 15 s never
// passes the largest number of the group, nor fp16. lo is one of the group's
// own fp16 numbers, so a group far from zero loses nothing. A token's groups
// depend on nothing else: appending leaves what is there as it is.
//
// Many quotients lie exactly halfway between two codes (x, lo and s are fp16
// numbers), so the quotient has to be the correctly rounded one: with
// inv = 1 / s and q0 = d inv, q0 + (d - q0 s) inv is (Markstein), two
// instructions past the product.
//
// One block per (32 consecutive token slots of a page, head, side), the piece
// of tokens that a 16-byte run of stored values holds: it alone writes that
// piece, so nothing is atomic.
#include <algorithm>

#include "kv_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32;      // tokens

__device__ inline half2_t min2(half2_t a, half2_t b) { return __builtin_elementwise_min(a, b); }
__device__ inline half2_t max2(half2_t a, half2_t b) { return __builtin_elementwise_max(a, b); }

// NaN counts as 0, an infinity as 65504.
__device__ inline half8_t finite8(half8_t v) {
    const kv_u32x4 w = __builtin_bit_cast(kv_u32x4, v) & 0x7FFF7FFFu;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) odd = odd || (w[j] & 0xFFFFu) >= 0x7C00u || w[j] >= 0x7C000000u;
    if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = static_cast<float>(v[j]);
            v[j] = f == f ? static_cast<half_t>(fminf(fmaxf(f, -kHalfMax), kHalfMax)) : static_cast<half_t>(0.f);
        }
    }
    return v;
}
__device__ inline void range8(half8_t v, half_t& lo, half_t& hi) {
    const half2_t a = {v[0], v[1]}, b = {v[2], v[3]}, c = {v[4], v[5]}, d = {v[6], v[7]};
    const half2_t l = min2(min2(a, b), min2(c, d)), h = max2(max2(a, b), max2(c, d));
    lo = l[0] < l[1] ? l[0] : l[1];
    hi = h[0] > h[1] ? h[0] : h[1];
}
// lo and hi over runs of `lanes` lanes (a power of two)
template <int LANES>
__device__ inline void range_across(half_t& lo, half_t& hi) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const uint32_t mine = __builtin_bit_cast(uint32_t, half2_t{lo, hi});
        const uint32_t got = static_cast<uint32_t>(__shfl_xor(static_cast<int>(mine), o));
        const half2_t other = __builtin_bit_cast(half2_t, got);
        lo = other[0] < lo ? other[0] : lo;
        hi = other[1] > hi ? other[1] : hi;
    }
}
// the largest fp16 number not above (hi - lo) / 15
__device__ inline half_t step_of(half_t lo, half_t hi) {
    const float want = (static_cast<float>(hi) - static_cast<float>(lo)) / 15.0f;
    const half_t s = static_cast<half_t>(want);
    const uint16_t bits = __builtin_bit_cast(uint16_t, s);
    return static_cast<float>(s) > want ? __builtin_bit_cast(half_t, static_cast<uint16_t>(bits - 1)) : s;
}
struct Group {
    float lo, s, inv;
    __device__ Group() = default;
    __device__ Group(half_t l, half_t step)
        : lo(static_cast<float>(l)), s(static_cast<float>(step)), inv(s > 0.f ? 1.0f / s : 0.f) {}
    __device__ uint32_t code(half_t x) const {
        const float d = static_cast<float>(x) - lo;
        const float q0 = d * inv;
        const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, d), inv, q0);
        return static_cast<uint32_t>(fminf(fmaxf(__builtin_rintf(q), 0.f), 15.f));
    }
};
// code j of a word: nibble j / 2 + 4 (j % 2)
__device__ constexpr int nibble(int j) { return 4 * (j / 2 + 4 * (j % 2)); }

// The chunk (32 slots) of a block: its tokens t0 .. t1 - 1 of the batch, the
// page's block number (page, head), the first slot, and the row of slot 0.
struct Chunk {
    int t0, t1, slot;
    int64_t block;
    int64_t row;
    bool held;
};
// chunk number `index` of those that the sequence's newest tokens touch
__device__ inline bool chunk_of(const KvPages& c, const KvSeq& sq, int b, int index, int head, Chunk& k) {
    const int lo = max(sq.start, 0);
    if (lo >= sq.end()) return false;
    const int64_t at = static_cast<int64_t>(lo >> 5) + index;
    if (at * kChunk >= sq.end()) return false;
    const int first = static_cast<int>(at) * kChunk;
    k.t0 = max(lo - first, 0);
    k.t1 = min(sq.end() - first, kChunk);
    k.slot = first & ((1 << c.log2_page) - 1);
    k.row = static_cast<int64_t>(sq.row0) + first - sq.start;
    const int id = kv_page(c, b, first >> c.log2_page);
    k.held = id >= 0;
    k.block = static_cast<int64_t>(max(id, 0)) * c.heads + head;
    return true;
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(KvWriteArgs a) {
    constexpr int PC = D / 32;
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int head = blockIdx.y;
    const bool values = blockIdx.z & 1;
    const int b = blockIdx.z >> 1;
    const KvSeq sq = kv_seq(c, b);
    Chunk ch;
    if (!chunk_of(c, sq, b, static_cast<int>(blockIdx.x), head, ch) || !ch.held) return;
    const int64_t token_stride = values ? a.v_token : a.k_token;
    const half_t* x = (values ? a.v + head * a.v_head : a.k + head * a.k_head) + ch.row * token_stride;

    if (!values) {
        // four lanes to a group of 32 channels, a word of codes each
        half2_t* scales = kv4_k_scales(c);
        for (int i = tid; i < (ch.t1 - ch.t0) * (D / 8); i += kThreads) {
            const int t = ch.t0 + i / (D / 8), w = i % (D / 8);
            const half8_t v = finite8(*reinterpret_cast<const half8_t*>(x + t * token_stride + w * 8));
            half_t lo, hi;
            range8(v, lo, hi);
            range_across<4>(lo, hi);
            const half_t s = step_of(lo, hi);
            const Group g(lo, s);
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) word |= g.code(v[j]) << nibble(j);
            const int64_t at = ((ch.block * PC + w / 4) << c.log2_page) + ch.slot + t;
            *reinterpret_cast<uint32_t*>(c.k_codes + at * 16 + (w % 4) * 4) = word;
            if (w % 4 == 0) scales[at] = half2_t{s, lo};
        }
        return;
    }

    // values: a token's range by LANES lanes, its row kept in LDS; then a thread
    // takes eight tokens of a channel
    constexpr int LANES = D <= 64 ? 8 : D <= 128 ? 16 : 32;     // at least D / 8
    constexpr int SX = D + 2;
    __shared__ __attribute__((aligned(4))) half_t rows[kChunk * SX];
    __shared__ Group groups[kChunk];
    half_t* scales = kv4_v_scales(c) + ((2 * ch.block) << c.log2_page) + ch.slot;
    for (int i = tid; i < (ch.t1 - ch.t0) * LANES; i += kThreads) {
        const int t = ch.t0 + i / LANES, w = min(i % LANES, D / 8 - 1);
        const half8_t v = finite8(*reinterpret_cast<const half8_t*>(x + t * token_stride + w * 8));
        half_t lo, hi;
        range8(v, lo, hi);
        range_across<LANES>(lo, hi);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<half2_t*>(rows + t * SX + w * 8 + 2 * j) = half2_t{v[2 * j], v[2 * j + 1]};
        if (i % LANES == 0) {
            const half_t s = step_of(lo, hi);
            groups[t] = Group(lo, s);
            scales[t] = s;
            scales[(1 << c.log2_page) + t] = lo;
        }
    }
    __syncthreads();
    // [slot / 32][D][16]
    uint32_t* out = reinterpret_cast<uint32_t*>(c.v_codes + ((ch.block * D) << (c.log2_page - 1)) +
                                                static_cast<int64_t>(ch.slot >> 5) * D * 16);
    for (int i = tid; i < 4 * D; i += kThreads) {
        const int w = i % 4, d = i / 4;
        const int first = max(ch.t0 - 8 * w, 0), behind = min(ch.t1 - 8 * w, 8);    // new tokens of this word
        if (first >= behind) continue;
        uint32_t word = 0;
        if (first > 0) {        // the old tokens' codes stay
            const uint32_t old = out[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) word |= j < first ? old & (15u << nibble(j)) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= first && j < behind) word |= groups[8 * w + j].code(rows[(8 * w + j) * SX + d]) << nibble(j);
        out[i] = word;
    }
}

// Read: one block per (32 token slots, head, side) of the tokens asked for.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(KvReadArgs a) {
    constexpr int PC = D / 32;
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int head = blockIdx.y;
    const bool values = blockIdx.z & 1;
    const int b = blockIdx.z >> 1;
    half_t* y = values ? a.v : a.k;
    if (y == nullptr) return;
    const KvSeq sq = kv_seq(c, b);
    const int64_t token_stride = static_cast<int64_t>(c.heads) * D;
    y += head * static_cast<int64_t>(D);
    const kv_u32x4 zero = {0u, 0u, 0u, 0u};
    if (blockIdx.x == 0 && sq.start < 0) {      // rows at positions below 0
        for (int64_t i = tid; i < static_cast<int64_t>(min(-sq.start, sq.n)) * (D / 8); i += kThreads)
            *reinterpret_cast<kv_u32x4*>(y + (sq.row0 + i / (D / 8)) * token_stride + i % (D / 8) * 8) = zero;
    }
    Chunk ch;
    if (!chunk_of(c, sq, b, static_cast<int>(blockIdx.x), head, ch)) return;
    y += ch.row * token_stride;
    if (!ch.held) {
        for (int i = tid; i < (ch.t1 - ch.t0) * (D / 8); i += kThreads)
            *reinterpret_cast<kv_u32x4*>(y + (ch.t0 + i / (D / 8)) * token_stride + i % (D / 8) * 8) = zero;
        return;
    }
    if (!values) {
        const half2_t* scales = kv4_k_scales(c);
        for (int i = tid; i < (ch.t1 - ch.t0) * (D / 8); i += kThreads) {
            const int t = ch.t0 + i / (D / 8), w = i % (D / 8);
            const int64_t at = ((ch.block * PC + w / 4) << c.log2_page) + ch.slot + t;
            const uint32_t word = *reinterpret_cast<const uint32_t*>(c.k_codes + at * 16 + (w % 4) * 4);
            *reinterpret_cast<half8_t*>(y + t * token_stride + w * 8) = kv4_numbers8(word, scales[at]);
        }
        return;
    }
    const half_t* scales = kv4_v_scales(c) + ((2 * ch.block) << c.log2_page) + ch.slot;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(c.v_codes + ((ch.block * D) << (c.log2_page - 1)) +
                                                              static_cast<int64_t>(ch.slot >> 5) * D * 16);
    // a thread takes eight tokens of two channels
    for (int i = tid; i < 4 * (D / 2); i += kThreads) {
        const int w = i / (D / 2), d = i % (D / 2) * 2;
        if (8 * w >= ch.t1 || 8 * w + 8 <= ch.t0) continue;
        const half8_t s = *reinterpret_cast<const half8_t*>(scales + 8 * w);
        const half8_t lo = *reinterpret_cast<const half8_t*>(scales + (1 << c.log2_page) + 8 * w);
        const half8_t v0 = kv4_numbers8(codes[d * 4 + w], s, lo), v1 = kv4_numbers8(codes[d * 4 + 4 + w], s, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = 8 * w + j;
            if (t >= ch.t0 && t < ch.t1) *reinterpret_cast<half2_t*>(y + t * token_stride + d) = half2_t{v0[j], v1[j]};
        }
    }
}

// Blocks along x: the 32-token chunks that max_tokens consecutive tokens can
// touch, at most a sequence's. One also where a sequence has none: the read's
// first block zeroes the rows at positions below 0.
int64_t touched_chunks(const KvPages& c, int64_t max_tokens) {
    return std::max<int64_t>(1, std::min<int64_t>((max_tokens + kChunk - 2) / kChunk + 1,
                                                  static_cast<int64_t>(c.max_pages) << (c.log2_page - 5)));
}
// a launch takes 2^32 threads along x
bool launchable(const KvPages& c, int64_t max_tokens) {
    return touched_chunks(c, max_tokens) < (int64_t{1} << 32) / kThreads;
}

template <class Args, class Launch>
awq_status by_dim(const Args& a, const Launch& launch) {
    if (!launchable(a.c, a.max_tokens)) return AWQ_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(touched_chunks(a.c, a.max_tokens)), static_cast<unsigned>(a.c.heads),
                    static_cast<unsigned>(2 * a.n_seqs));
    switch (a.head_dim) {
        case 64: launch(std::integral_constant<int, 64>{}, grid); break;
        case 96: launch(std::integral_constant<int, 96>{}, grid); break;
        case 128: launch(std::integral_constant<int, 128>{}, grid); break;
        case 192: launch(std::integral_constant<int, 192>{}, grid); break;
        case 256: launch(std::integral_constant<int, 256>{}, grid); break;
        default: return AWQ_ERR_CONFIG;
    }
    return last_launch_status();
}

}  // namespace

awq_status launch_kv4_write(const KvWriteArgs& a, hipStream_t stream) {
    return by_dim(a, [&](auto dim, dim3 grid) {
        hipLaunchKernelGGL((kv4_write_kernel<decltype(dim)::value>), grid, dim3(kThreads), 0, stream, a);
    });
}

awq_status launch_kv4_read(const KvReadArgs& a, hipStream_t stream) {
    return by_dim(a, [&](auto dim, dim3 grid) {
        hipLaunchKernelGGL((kv4_read_kernel<decltype(dim)::value>), grid, dim3(kThreads), 0, stream, a);
    });
}

}  // namespace awq
