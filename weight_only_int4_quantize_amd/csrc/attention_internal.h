// What the attention kernels share, over the 8-bit cache (attention.hip) and
// the 4-bit one (attention4.hip): the rows' spans, the join of a row tile's
// parts, and the split of a call over the GPU.
#pragma once

#include <algorithm>

#include "kv_internal.h"

namespace awq {
namespace {

constexpr float kNone = -1.0e38f;       // running maximum before any visible key
constexpr int kSc1 = 16;                // cache-policy bit sc1 (device scope)
constexpr float kLn2 = 0.69314718056f;

// Splits of the keys over blocks: split s takes positions
// [s * tokens, (s + 1) * tokens).
struct Split {
    int tokens;
    KvDivisor by_tokens;
    float* partials;    // per (row tile, split): [rows][D] outputs, [rows] maxima, [rows] sums
    int* counters;      // per row tile, zero between launches
};
// The rows of one kv head that a block has summed up, and where the other
// blocks park their parts of them.
struct Rows {
    int kv_head, row0, rows;
    int parts;              // 1: the block has all of it
    int mine;               // this block's part
    float* base;            // part p's floats at base + offset(p)
    int64_t bytes;          // of the whole region
    int* counter;
};

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                             0x00020000);
}

// The larger of a value and its copies half a wave and a quarter away, by the
// wave's swaps (v_permlane32_swap, v_permlane16_swap). Elements are taken out
// of the result as integers first: a bit cast of a vector element reads
// element 0.
typedef uint32_t swap_t __attribute__((ext_vector_type(2)));
__device__ inline float larger_of(swap_t v) {
    const uint32_t a = v[0], b = v[1];
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ inline float across_halves_max(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    return larger_of(__builtin_amdgcn_permlane32_swap(u, u, false, false));
}
__device__ inline float across_quarters_max(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, across_halves_max(v));
    return larger_of(__builtin_amdgcn_permlane16_swap(u, u, false, false));
}

// Two weights as two fp16 numbers each, both toward zero: hi + lo is within
// 2^-20 of the weight. The rounding is one instruction for the pair (to the
// nearest it takes three), the difference, exact, one each. Written out as
// w - float(half(w)) with w a product, it went wrong: the compiler rounded
// the exact product for the difference and the rounded one for the operand,
// which differ by a step of fp16 at ties, so that one weight in some 2^14
// was off by 2^-11 of itself.
__device__ inline void two_parts(float w0, float w1, half2_t& hi, half2_t& lo) {
    hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_pkrtz(w0, w1));
    float r0, r1;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(r0) : "v"(hi), "v"(w0));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r1) : "v"(hi), "v"(w1));
    lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_pkrtz(r0, r1));
}

// Query rows of a kv head that the call works on. New tokens past max_tokens are
// left out, also where a block has room for them: they would widen what the
// block's rows see to positions that may hold anything.
__device__ inline int rows_of(const KvAttentionArgs& a, const KvSeq& sq) {
    return static_cast<int>(min(static_cast<int64_t>(sq.n), a.max_tokens)) * a.ratio;
}
// The positions rows [row0, row0 + rows) of a kv head see.
struct Span {
    int begin, end;             // any of them
    int all_begin, all_end;     // every one of them
};
__device__ inline void visible(const KvAttentionArgs& a, const KvSeq& sq, int token, int& lo, int& hi) {
    const int p = sq.start + token;
    hi = a.causal ? min(sq.len, p + 1) : sq.len;
    lo = a.window > 0 ? max(0, max(p, -1) - a.window + 1) : 0;
}
__device__ inline Span row_span(const KvAttentionArgs& a, const KvSeq& sq, int row0, int rows) {
    const int first = a.by_ratio.of(row0);
    const int last = min(sq.n - 1, a.by_ratio.of(row0 + rows - 1));
    Span s;
    visible(a, sq, first, s.begin, s.all_end);
    visible(a, sq, last, s.all_begin, s.end);
    return s;
}

// The output of one row: o (in true units) / sum, and its lse.
__device__ inline void store_lse(const KvAttentionArgs& a, const KvSeq& sq, int kv_head, int row, float m, float sum) {
    if (a.lse == nullptr) return;
    const int token = a.by_ratio.of(row), head = (kv_head - token) * a.ratio + row;
    a.lse[(static_cast<int64_t>(sq.row0) + token) * (static_cast<int64_t>(a.c.heads) * a.ratio) + head] =
        sum == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}
__device__ inline half_t* out_row(const KvAttentionArgs& a, const KvSeq& sq, int kv_head, int row) {
    const int token = a.by_ratio.of(row), head = (kv_head - token) * a.ratio + row;
    return a.out + (static_cast<int64_t>(sq.row0) + token) * a.out_token + head * a.out_head;
}

typedef half_t half4_t __attribute__((ext_vector_type(4)));
constexpr int kJoin = 4096;     // floats of the join's weights and sums: 2 splits rows
constexpr int max_splits(int rows) { return kJoin / 2 / rows; }
constexpr int part_floats(int rows, int dim) { return rows * (dim + 2); }
// floats of LDS the join takes (over the outputs, which are parked by then)
constexpr int join_floats(int rows, int threads) { return kJoin + rows + threads * 4; }

// A block's rows are complete: so [ROWS][D] outputs in true units, sm and sl
// their maxima and sums, all in LDS. With one split they are divided and
// stored; otherwise parked, and the last of the tile's blocks to arrive adds
// the splits in order (deterministic; nobody waits on anybody).
// ALONE: each thread joins the parts of its own outputs, eight parts' loads in
// flight, without LDS and barriers, in less code (which a block reaches once, and
// cold: 0.3 us a kilobyte). Over the 4-bit cache, 128 channels, in a graph (us, in
// brackets by the join below): 1 x 512 to 4000 tokens of 32 heads, 2 to 8 parts,
// 7.6 (9.0), 8.2 (9.6), 10.5 (12.0); 1 x 8000 of 8 heads, 32 parts, 1 / 8 query rows
// 11.5 (11.7) / 11.7 (12.9); 128 parts of one head of 32768, 1 / 8 / 16 rows
// 16.7 (13.4) / 16.8 (19.4) / 25.5 (27.1). So one row of 64 parts and more, 32
// threads at work on them one batch after the other, is slower by 1 to 3.5 us: one
// sequence of four kv heads or fewer that share no queries. A second instance for
// that alone was not made. The 8-bit decode kernel still takes the join below; this
// one measured 7.8 (9.1) for 1 x 1000 of 32 heads, 11.2 (12.1) for 1 x 8000 of 8 with
// 4 rows, 34.9 (31.8) for 1 x 131072 of 4 with one.
template <int D, int ROWS, int NT, bool ALONE = false, class Offset>
__device__ inline void finish_rows(const KvAttentionArgs& a, const KvSeq& sq, const Rows& rw, const Offset& offset,
                                   const float* so, int so_stride, const float* sm, const float* sl, float* scratch,
                                   int* s_flag) {
    const int tid = threadIdx.x;
    const int kv_head = rw.kv_head, row0 = rw.row0, rows = rw.rows;
    if (rw.parts <= 1) {
        for (int i = tid; i < rows * (D / 4); i += NT) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float inv = sl[r] > 0.f ? 1.0f / sl[r] : 0.f;
            half4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = static_cast<half_t>(so[r * so_stride + d + j] * inv);
            *reinterpret_cast<half4_t*>(out_row(a, sq, kv_head, row0 + r) + d) = v;
        }
        for (int r = tid; r < rows; r += NT) store_lse(a, sq, kv_head, row0 + r, sm[r], sl[r]);
        return;
    }
    const auto rs = rsrc(rw.base, static_cast<uint32_t>(rw.bytes));
    const int base = offset(rw.mine) * 4;
    for (int i = tid; i < rows * (D / 4); i += NT) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        const float4_t v = *reinterpret_cast<const float4_t*>(so + r * so_stride + d);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(kv_u32x4, v), rs, (r * D + d) * 4, base, kSc1);
    }
    for (int r = tid; r < rows; r += NT) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, sm[r]), rs, (ROWS * D + r) * 4, base, kSc1);
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, sl[r]), rs, (ROWS * D + ROWS + r) * 4, base,
                                              kSc1);
    }
    // sc1 stores and loads go past the per-XCD L2s; every store is complete
    // before the counter moves, and the loads are issued after it is read
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
        *s_flag = __hip_atomic_fetch_add(rw.counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == rw.parts - 1;
    __syncthreads();
    if (!*s_flag) return;
    // ---- the last block: every split's maxima and sums first (all at once),
    // from them the splits' weights, then the outputs, eight splits' loads in
    // flight and the splits shared out over the threads there are beyond one
    // per four outputs. One split after the other, a join of 64 splits took
    // 60 us of a 110 us call (2 x 131072 tokens, 8 heads of 128).
    const int n = rw.parts;
    if constexpr (ALONE) {
        constexpr int BATCH = 8;
        for (int i = tid; i < rows * (D / 4); i += NT) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float jm = kNone, jsum = 0.f;
            float4_t o = {0.f, 0.f, 0.f, 0.f};
            for (int s0 = 0; s0 < n; s0 += BATCH) {
                float mx[BATCH], sum[BATCH];
                float4_t v[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int at = offset(min(s0 + k, n - 1)) * 4;
                    mx[k] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(rs, (ROWS * D + r) * 4, at, kSc1));
                    sum[k] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(rs, (ROWS * D + ROWS + r) * 4, at, kSc1));
                    v[k] = __builtin_bit_cast(
                        float4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (r * D + d) * 4, at, kSc1));
                }
                float top = jm;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) top = fmaxf(top, mx[k]);
                const float carry = __builtin_amdgcn_exp2f(jm - top);
                jsum *= carry;
                o *= carry;
                jm = top;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const float w = s0 + k < n ? __builtin_amdgcn_exp2f(mx[k] - jm) : 0.f;
                    jsum = __builtin_fmaf(w, sum[k], jsum);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(w, v[k][j], o[j]);
                }
            }
            const float inv = jsum > 0.f ? 1.0f / jsum : 0.f;
            half4_t h;
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = static_cast<half_t>(o[j] * inv);
            *reinterpret_cast<half4_t*>(out_row(a, sq, kv_head, row0 + r) + d) = h;
            if (d == 0) store_lse(a, sq, kv_head, row0 + r, jm, jsum);
        }
        if (tid == 0) __hip_atomic_store(rw.counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }
    float* wt = scratch;                    // [n][ROWS] maxima, then weights
    float* ls = scratch + kJoin / 2;        // [n][ROWS] sums
    for (int i = tid; i < n * ROWS; i += NT) {
        const int s = i / ROWS, r = i % ROWS;
        if (r < rows) {
            // (per-lane split: a vector offset)
            const int at = (offset(s) + ROWS * D + r) * 4;
            wt[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, kSc1));
            ls[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, at + ROWS * 4, 0, kSc1));
        }
    }
    __syncthreads();
    constexpr int TPR = NT / ROWS;          // threads per row
    const int jr = tid / TPR, jl = tid % TPR;
    float jm = kNone, jsum = 0.f;
    if (jr < rows)
        for (int s = jl; s < n; s += TPR) jm = fmaxf(jm, wt[s * ROWS + jr]);
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1) jm = fmaxf(jm, __shfl_xor(jm, o));
    if (jr < rows)
        for (int s = jl; s < n; s += TPR) {
            const float w = __builtin_amdgcn_exp2f(wt[s * ROWS + jr] - jm);
            wt[s * ROWS + jr] = w;
            jsum += w * ls[s * ROWS + jr];
        }
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1) jsum += __shfl_xor(jsum, o);
    float* total = scratch + kJoin;         // [ROWS] 1 / sum
    if (jr < rows && jl == 0) {
        total[jr] = jsum > 0.f ? 1.0f / jsum : 0.f;
        store_lse(a, sq, kv_head, row0 + jr, jm, jsum);
    }
    __syncthreads();
    const int items = rows * (D / 4);
    const int groups = items < NT ? NT / items : 1;
    float4_t* red = reinterpret_cast<float4_t*>(total + ROWS);      // [groups][items], groups > 1
    for (int i0 = 0; i0 < items; i0 += NT) {
        const int i = groups > 1 ? tid % items : i0 + tid;
        const int g = groups > 1 ? tid / items : 0;
        const bool mine = i < items && g < groups;
        const int r = mine ? i / (D / 4) : 0, d = mine ? i % (D / 4) * 4 : 0;
        float4_t o = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = mine ? g : n; s0 < n; s0 += 8 * groups) {
            float4_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int s = min(s0 + k * groups, n - 1);
                v[k] = __builtin_bit_cast(
                    float4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (offset(s) + r * D + d) * 4, 0, kSc1));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float w = s0 + k * groups < n ? wt[(s0 + k * groups) * ROWS + r] : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += w * v[k][j];
            }
        }
        if (groups > 1) {
            if (mine) red[tid] = o;
            __syncthreads();
            if (g == 0)
                for (int k = 1; k < groups; ++k) {
                    const float4_t v = red[k * items + i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] += v[j];
                }
        }
        if (mine && g == 0) {
            const float inv = total[r];
            half4_t h;
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = static_cast<half_t>(o[j] * inv);
            *reinterpret_cast<half4_t*>(out_row(a, sq, kv_head, row0 + r) + d) = h;
        }
    }
    if (tid == 0) __hip_atomic_store(rw.counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- the split of a call

constexpr int kDecodeRows = 16;
constexpr int kDecodeWaves = 4;
constexpr int kTile = 64;
constexpr int kPrefillWaves = 4;
constexpr int kPrefillRows = 32 * kPrefillWaves;
constexpr int kWideDim = 128;               // over the 4-bit cache: see plan_for

// Counters at the workspace's start, whatever the call: a split launch has at
// most this many row tiles.
constexpr int kCounters = 4096;
constexpr size_t kCounterBytes = kCounters * sizeof(int);

struct Plan {
    bool decode;
    int rows;               // of a block
    int64_t row_tiles;      // per sequence and kv head
    int splits;
    int tokens;             // positions per split
};

// Up to 32 query rows per kv head go to the decode kernel, longer runs to the
// prefill kernel. The keys are split until the blocks fill the GPU: two
// blocks per CU of at least 1024 positions, which cover what a block costs apart from its
// tiles (some 8 us: its first loads, and the join); short launches of under a
// block per CU split down to 256 positions, a tile per wave. Measured (us):
// 16 x 4096 tokens, 4 heads of 256: 23 at 1024 positions, 33 at 512, 45 at
// 256; 1 x 131072, 8 heads of 128: 54 at 2048, 62 at 1024; 1 x 1000, 32
// heads: 10.1 at 256, 11.0 whole. Dealing the tiles of all sequences out
// evenly to 512 blocks instead, which a ragged batch would ask for, was
// slower on every shape (64 x 8192 to 2048: 145 against 134), as a block then
// pays for two or more pieces.
// Over the 4-bit cache, 17 to 32 rows are one block's, which unpacks the keys and
// values once for both sixteens, where the sequences' kv heads are two to a CU, or
// enough for few parts to join and long. Measured in a graph, 8 query heads a kv
// head, 8 kv heads of 128, 4 tokens (us, as two blocks of 16 rows, as one):
//   taken     64 x 64 11.1, 9.1; 64 x 4096 102, 78; 16 x 4096 30.3, 26.9; 8 x 8192
//             30.5, 27.3; 4 x 16384 30.5, 29.1; 8 x 32768 105, 78; 2 x 65536 55, 50;
//             2 x 131072 104, 84; 16 kv heads 1 x 65536 53, 49; one 16 x 65536 55, 50
//   not       16 x 2000 19.3, 19.7; 2 x 32768 31.8, 34.4; 1 x 65536 35.2, 42.3;
//             1 x 131072 56.2, 58.7; 1 x 1000 8.8, 11.2; one kv head 1 x 262144 40, 59;
//             and, where it would gain, 32 x 1000 17.7, 16.6
// (another card, calls back to back: 64 x 4096 109, 87; 2 x 131072 115, 93). With
// 192 channels and more it leaves one wave per SIMD: 64 x 4096 171, 152, but 16 x
// 4096 48, 54.
inline Plan plan_for(int format, int head_dim, int n_seqs, int kv_heads, int ratio, int64_t max_tokens, int64_t max_len,
                     bool have_workspace) {
    Plan p;
    const int64_t rows = max_tokens * ratio;
    p.decode = rows <= 2 * kDecodeRows;
    const int64_t cu = cu_count();
    const int64_t pairs = static_cast<int64_t>(n_seqs) * kv_heads;
    const bool wide = format == AWQ_KV_INT4 && rows > kDecodeRows && head_dim <= kWideDim &&
                      (pairs >= 2 * cu || (pairs >= 32 && pairs * max_len >= int64_t{1} << 19) ||
                       (pairs >= 16 && pairs * max_len >= int64_t{1} << 20));
    const int per_block = p.rows = !p.decode ? kPrefillRows : wide ? 2 * kDecodeRows : kDecodeRows;
    p.row_tiles = ceil_div(rows, per_block);
    const int64_t tiles = p.row_tiles * n_seqs * kv_heads;
    const int64_t most = max_splits(per_block);
    int64_t splits = 1, unit = p.decode ? 1024 : kTile * 8;
    if (have_workspace && tiles <= kCounters) {
        splits = std::min({ceil_div(max_len, unit), 2 * cu / tiles, most});
        if (p.decode && splits * tiles < cu) {
            unit = kTile * kDecodeWaves;
            splits = std::min({ceil_div(max_len, unit), cu / tiles, most});
        }
        splits = std::max<int64_t>(1, splits);
    }
    const int64_t units = std::max<int64_t>(1, ceil_div(max_len, unit));
    p.tokens = static_cast<int>(ceil_div(units, splits) * unit);      // at most kKvMaxLen
    p.splits = static_cast<int>(std::max<int64_t>(1, ceil_div(max_len, p.tokens)));
    return p;
}

inline size_t plan_bytes(const Plan& p, int n_seqs, int kv_heads, int head_dim) {
    const size_t tiles = static_cast<size_t>(p.row_tiles) * n_seqs * kv_heads;
    const size_t floats = part_floats(p.rows, head_dim);
    return kCounterBytes + (p.splits > 1 ? tiles * p.splits * floats * sizeof(float) : 0);
}

inline Split split_of(const Plan& p, void* workspace) {
    Split sp;
    sp.tokens = p.tokens;
    sp.by_tokens = KvDivisor(static_cast<uint32_t>(p.tokens));
    sp.counters = static_cast<int*>(workspace);
    sp.partials = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes) : nullptr;
    return sp;
}

// a launch takes 65535 blocks along y and 2^32 threads along x
inline bool launchable(const Plan& p, int kv_heads) {
    return p.decode ? p.row_tiles * kv_heads <= 65535
                    : p.row_tiles * p.splits * kv_heads < (int64_t{1} << 32) / (kPrefillWaves * kWave);
}

}  // namespace
}  // namespace awq
