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
// instructions past the product. A number takes some 14 vector instructions;
// with divisions, clamps and shifts written out it was 27, and the kernel bound
// by them.
//
// One block per (32 consecutive token slots of a page, head), the piece of
// tokens that a 16-byte run of stored values holds: it alone writes that piece,
// so nothing is atomic.
#include <algorithm>

#include "kv_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32;      // tokens

// (as instructions: from the language's maximum the compiler also makes one that
// quiets signalling NaN, of every operand)
__device__ inline half2_t max2(half2_t a, half2_t b) {
    half2_t r;
    asm("v_pk_max_f16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ inline half2_t max2_negated(half2_t a, half2_t b) {      // max(-a, -b)
    half2_t r;
    asm("v_pk_max_f16 %0, %1, %2 neg_lo:[1,1] neg_hi:[1,1]" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
struct Eight {
    half2_t v[4];
};
__device__ inline Eight load8(const half_t* p) { return __builtin_bit_cast(Eight, *reinterpret_cast<const half8_t*>(p)); }

// NaN counts as 0, an infinity as 65504. (A sum of products with 0 is NaN if
// there is either.)
__device__ inline void make_finite(Eight& x) {
    const half2_t zero = {static_cast<half_t>(0.f), static_cast<half_t>(0.f)};
    half2_t t = x.v[0] * zero;
#pragma unroll
    for (int j = 1; j < 4; ++j) t = __builtin_elementwise_fma(x.v[j], zero, t);
    if (t[0] == t[0] && t[1] == t[1]) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float f = static_cast<float>(x.v[j][k]);
            x.v[j][k] = f == f ? static_cast<half_t>(fminf(fmaxf(f, -kHalfMax), kHalfMax)) : static_cast<half_t>(0.f);
        }
}
// (-smallest, largest) of eight finite numbers: one maximum for both from here on
__device__ inline half2_t range8(const Eight& x) {
    const half2_t l = max2(max2_negated(x.v[0], x.v[1]), max2_negated(x.v[2], x.v[3]));
    const half2_t h = max2(max2(x.v[0], x.v[1]), max2(x.v[2], x.v[3]));
    return max2(half2_t{l[0], h[0]}, half2_t{l[1], h[1]});
}
// the same over runs of LANES lanes (4 .. 32, a power of two)
template <int LANES>
__device__ inline half2_t range_across(half2_t r) {
    const auto dpp = [&](auto control) {
        const int bits = __builtin_bit_cast(int, r);
        const uint32_t got =
            static_cast<uint32_t>(__builtin_amdgcn_update_dpp(bits, bits, decltype(control)::value, 0xF, 0xF, true));
        r = max2(r, __builtin_bit_cast(half2_t, got));
    };
    dpp(std::integral_constant<int, 0xB1>{});       // quad_perm: neighbours
    dpp(std::integral_constant<int, 0x4E>{});       // quad_perm: pairs
    if (LANES >= 8) dpp(std::integral_constant<int, 0x141>{});      // row_half_mirror
    if (LANES >= 16) dpp(std::integral_constant<int, 0x140>{});     // row_mirror
    if (LANES >= 32) {
        const uint32_t got = static_cast<uint32_t>(__shfl_xor(__builtin_bit_cast(int, r), 16));
        r = max2(r, __builtin_bit_cast(half2_t, got));
    }
    return r;
}
// A group: lo, s = the largest fp16 number not above (hi - lo) / 15, and 1 / s
// (0 for s = 0). Quotient and reciprocal as nearest numbers, by Markstein's
// steps and one of Newton's: no difference from the division for any fp16 s, nor
// for 6.7e7 random ranges.
struct Group {
    float lo, s, inv;
    __device__ half2_t stored() const { return half2_t{static_cast<half_t>(s), static_cast<half_t>(lo)}; }
};
__device__ inline Group group_of(half2_t range) {
    Group g;
    g.lo = -static_cast<float>(range[0]);
    const float span = static_cast<float>(range[1]) - g.lo;
    constexpr float kFifteenth = 1.0f / 15.0f;
    const float q0 = span * kFifteenth;
    const float want = __builtin_fmaf(__builtin_fmaf(-q0, 15.0f, span), kFifteenth, q0);
    const half_t s = static_cast<half_t>(want);
    const uint16_t bits = __builtin_bit_cast(uint16_t, s);
    g.s = static_cast<float>(
        __builtin_bit_cast(half_t, static_cast<uint16_t>(bits - (static_cast<float>(s) > want ? 1 : 0))));
    const float r = __builtin_amdgcn_rcpf(g.s);
    g.inv = g.s > 0.f ? __builtin_fmaf(__builtin_fmaf(-g.s, r, 1.0f), r, r) : 0.f;
    return g;
}
// The code of x's lower or upper half, as a whole fp32 number 0 .. 15 whatever x
// and g hold.
template <int HIGH>
__device__ inline float code_of(const Group& g, half2_t x) {
    float d;
    if constexpr (HIGH)
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(d) : "v"(x), "v"(g.lo));
    else
        asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(d) : "v"(x), "v"(g.lo));
    const float q0 = d * g.inv;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, g.s, d), g.inv, q0);
    return __builtin_rintf(__builtin_amdgcn_fmed3f(q, 0.f, 15.f));
}
// Codes c[0 .. 7] to a word, code 2 j in nibble j, code 2 j + 1 in nibble j + 4:
// 16 bits at a time, exact in fp32.
__device__ inline uint32_t word_of(const float (&c)[8]) {
    const auto half = [](float a, float b, float d, float e) {
        return static_cast<uint32_t>(__builtin_fmaf(
            __builtin_fmaf(__builtin_fmaf(e, 16.f, d), 16.f, b), 16.f, a));
    };
    return half(c[0], c[2], c[4], c[6]) | (half(c[1], c[3], c[5], c[7]) << 16);
}
// the bits of codes first .. 7 (first 0 .. 8): nibbles (first + 1) / 2 .. 3 of
// the lower half, first / 2 .. 3 of the upper
__device__ inline uint32_t from_code(int first) {
    const uint32_t low = 0xFFFFu & (0xFFFFu << (4 * ((first + 1) / 2)));
    return low | ((0xFFFFu << (4 * (first / 2))) << 16);
}

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
    const int id = kv_page_shared(c, b, first >> c.log2_page);
    k.held = id >= 0;
    k.block = static_cast<int64_t>(max(id, 0)) * c.heads + head;
    return true;
}

// Both sides by one block, all of a thread's loads on their way at once, before
// the page is known. Keys: four lanes to a group of 32 channels, a word of codes
// each, neighbouring tokens next to each other, as they are stored (neighbouring
// groups instead read whole rows and store runs of 64 bytes: no difference).
// Values: a token's range by LANES lanes, its row kept in LDS; then a
// thread takes eight tokens of pairs of channels. Rows are D + 4 halves apart:
// the four words' rows are then 16 banks apart.
// Bound by HBM: 11776 tokens of 32 heads of 128, 193 MB read and 55 MB written,
// 55 us alone, 4.5 TB/s (a copy reaches 5.2). 64 x 1 token of 8 heads 4.9 us,
// latencies.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(KvWriteArgs a, KvDivisor by_heads) {
    constexpr int PC = D / 32;
    constexpr int KL = D / 8;                                   // lanes to a token's keys
    constexpr int VL = D <= 64 ? 8 : D <= 128 ? 16 : 32;        // to its values, at least D / 8
    constexpr int KN = (kChunk * KL + kThreads - 1) / kThreads;
    constexpr int VN = (kChunk * VL + kThreads - 1) / kThreads;
    constexpr int SX = D + 4;
    __shared__ __attribute__((aligned(16))) half_t rows[kChunk * SX];
    __shared__ __attribute__((aligned(16))) float lo[kChunk], step[kChunk], inv[kChunk];
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int index = by_heads.of(blockIdx.x);
    const int head = blockIdx.x - index * c.heads;
    const int b = blockIdx.y;
    const KvSeq sq = kv_seq_shared(c, b);
    Chunk ch;
    if (!chunk_of(c, sq, b, index, head, ch)) return;
    const half_t* xk = a.k + head * a.k_head + ch.row * a.k_token;
    const half_t* xv = a.v + head * a.v_head + ch.row * a.v_token;
    const int tokens = ch.t1 - ch.t0;
    Eight v[VN], k[KN];     // (outside the new tokens: the next of them, and not used)
#pragma unroll
    for (int n = 0; n < VN; ++n) {
        const int i = min(tid + n * kThreads, tokens * VL - 1);
        v[n] = load8(xv + (ch.t0 + i / VL) * a.v_token + min(i % VL, KL - 1) * 8);
    }
#pragma unroll
    for (int n = 0; n < KN; ++n) {
        const int i = tid + n * kThreads;
        const int t = min(max(i / 4 % kChunk, ch.t0), ch.t1 - 1), g = min(i / (4 * kChunk), PC - 1);
        k[n] = load8(xk + t * a.k_token + g * 32 + i % 4 * 8);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!ch.held) return;

    // ---- values: ranges, rows to LDS ----
#pragma unroll
    for (int n = 0; n < VN; ++n) {
        const int i = tid + n * kThreads;
        if (i >= tokens * VL) break;
        const int t = ch.t0 + i / VL, w = min(i % VL, KL - 1);
        make_finite(v[n]);
        const Group g = group_of(range_across<VL>(range8(v[n])));
        half2_t* row = reinterpret_cast<half2_t*>(rows + t * SX + w * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) row[j] = v[n].v[j];
        if (i % VL == 0) {
            lo[t] = g.lo;
            step[t] = g.s;
            inv[t] = g.inv;
        }
    }
    // ---- keys ----
    half2_t* k_scales = kv4_k_scales(c);
#pragma unroll
    for (int n = 0; n < KN; ++n) {
        const int i = tid + n * kThreads;
        const int t = i / 4 % kChunk, piece = i / (4 * kChunk), w = i % 4;
        if (t < ch.t0 || t >= ch.t1 || piece >= PC) continue;
        make_finite(k[n]);
        const Group g = group_of(range_across<4>(range8(k[n])));
        float code[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            code[2 * j] = code_of<0>(g, k[n].v[j]);
            code[2 * j + 1] = code_of<1>(g, k[n].v[j]);
        }
        const int64_t at = ((ch.block * PC + piece) << c.log2_page) + ch.slot + t;
        *reinterpret_cast<uint32_t*>(c.k_codes + at * 16 + w * 4) = word_of(code);
        if (w == 0) k_scales[at] = g.stored();
    }
    __syncthreads();
    if (const int t = tid % kChunk; tid < 2 * kChunk && t >= ch.t0 && t < ch.t1) {
        half_t* out = kv4_v_scales(c) + ((2 * ch.block) << c.log2_page) + ch.slot + t;
        if (tid < kChunk) *out = static_cast<half_t>(step[t]);
        else out[1 << c.log2_page] = static_cast<half_t>(lo[t]);
    }
    // ---- values: codes ----
    const int w = tid % 4;
    const int first = max(ch.t0 - 8 * w, 0), behind = min(ch.t1 - 8 * w, 8);    // new tokens of this word
    if (first >= behind) return;
    // (whatever LDS holds in the place of the others gives codes, masked out below)
    Group g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = Group{lo[8 * w + j], step[8 * w + j], inv[8 * w + j]};
    const uint32_t mine = from_code(first) & ~from_code(behind);
    // [slot / 32][D][16]
    uint32_t* out = reinterpret_cast<uint32_t*>(c.v_codes + ((ch.block * D) << (c.log2_page - 1)) +
                                                static_cast<int64_t>(ch.slot >> 5) * D * 16);
    for (int d = tid / 4 * 2; d < D; d += kThreads / 4 * 2) {
        float code[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const half2_t x = *reinterpret_cast<const half2_t*>(rows + (8 * w + j) * SX + d);
            code[0][j] = code_of<0>(g[j], x);
            code[1][j] = code_of<1>(g[j], x);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t* word = out + (d + e) * 4 + w;
            uint32_t bits = word_of(code[e]) & mine;
            if (mine != ~0u) bits |= *word & ~mine;     // the other tokens' codes stay
            *word = bits;
        }
    }
}

// Read: one block per (32 token slots, head, side) of the tokens asked for.
// Bound by the stores to HBM: the tokens above 55 us alone, 4.5 TB/s; the pair,
// write and read, 107 us. Stored past the caches the read alone took 39 us, but
// with what reads its result 125 against 108.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(KvReadArgs a, KvDivisor by_heads) {
    constexpr int PC = D / 32;
    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int index = by_heads.of(blockIdx.x);
    const int head = blockIdx.x - index * c.heads;
    const bool values = blockIdx.y & 1;
    const int b = blockIdx.y >> 1;
    half_t* y = values ? a.v : a.k;
    if (y == nullptr) return;
    const KvSeq sq = kv_seq_shared(c, b);
    const int64_t token_stride = static_cast<int64_t>(c.heads) * D;
    y += head * static_cast<int64_t>(D);
    const kv_u32x4 zero = {0u, 0u, 0u, 0u};
    if (index == 0 && sq.start < 0) {      // rows at positions below 0
        for (int64_t i = tid; i < static_cast<int64_t>(min(-sq.start, sq.n)) * (D / 8); i += kThreads)
            *reinterpret_cast<kv_u32x4*>(y + (sq.row0 + i / (D / 8)) * token_stride + i % (D / 8) * 8) = zero;
    }
    Chunk ch;
    if (!chunk_of(c, sq, b, index, head, ch)) return;
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
    // a thread takes eight tokens of two channels to LDS, and whole 16-byte
    // pieces of rows from there (stored from registers, 4 bytes of a row each, the
    // call took 60.6 us, now 55.8)
    constexpr int SX = D + 8;
    __shared__ __attribute__((aligned(16))) half_t rows[kChunk * SX];
    const int w = tid % 4;
    if (8 * w < ch.t1 && 8 * w + 8 > ch.t0) {
        const half8_t s = *reinterpret_cast<const half8_t*>(scales + 8 * w);
        const half8_t lo = *reinterpret_cast<const half8_t*>(scales + (1 << c.log2_page) + 8 * w);
        for (int d = tid / 4 * 2; d < D; d += kThreads / 4 * 2) {
            const half8_t v0 = kv4_numbers8(codes[d * 4 + w], s, lo), v1 = kv4_numbers8(codes[d * 4 + 4 + w], s, lo);
#pragma unroll
            for (int j = 0; j < 8; ++j) *reinterpret_cast<half2_t*>(rows + (8 * w + j) * SX + d) = half2_t{v0[j], v1[j]};
        }
    }
    __syncthreads();
    for (int i = tid; i < (ch.t1 - ch.t0) * (D / 8); i += kThreads) {
        const int t = ch.t0 + i / (D / 8), d = i % (D / 8) * 8;
        *reinterpret_cast<half8_t*>(y + t * token_stride + d) = *reinterpret_cast<const half8_t*>(rows + t * SX + d);
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
    return touched_chunks(c, max_tokens) < (int64_t{1} << 32) / kThreads / c.heads;
}

template <class Args, class Launch>
awq_status by_dim(const Args& a, int sides, const Launch& launch) {
    if (!launchable(a.c, a.max_tokens)) return AWQ_ERR_SHAPE;
    // Heads fastest: the blocks at work together read whole rows of the token
    // tensors (the same head's chunks next to each other: a read of 11776 tokens, 32 heads of
    // 128, 58 us against 45 behind the write).
    const dim3 grid(static_cast<unsigned>(touched_chunks(a.c, a.max_tokens) * a.c.heads),
                    static_cast<unsigned>(sides * a.n_seqs));
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
    return by_dim(a, 1, [&](auto dim, dim3 grid) {
        hipLaunchKernelGGL((kv4_write_kernel<decltype(dim)::value>), grid, dim3(kThreads), 0, stream, a,
                           KvDivisor(static_cast<uint32_t>(a.c.heads)));
    });
}

awq_status launch_kv4_read(const KvReadArgs& a, hipStream_t stream) {
    return by_dim(a, 2, [&](auto dim, dim3 grid) {
        hipLaunchKernelGGL((kv4_read_kernel<decltype(dim)::value>), grid, dim3(kThreads), 0, stream, a,
                           KvDivisor(static_cast<uint32_t>(a.c.heads)));
    });
}

}  // namespace awq
