// Softmax attention of a batch's newest tokens over the paged 4-bit cache
// (include/awq.h, awq_kv_attention with AWQ_KV_INT4).
//
// Mathematics. A cached number is fp16(lo + s c), one fused multiply-add of
// the code c, so the products' operands are the cache's own numbers, exactly.
// With logits t = (q . k) scale log2 e and the running maximum m, the weights
// are p = 2^(t - m + 12); the unit 2^12 is in the sum and in the outputs and
// divides out. Maxima move only when one would be passed by 3, so weights stay
// below 2^15 and the outputs are rarely rescaled; each enters the second
// product as two fp16 numbers (attention_internal.h: one rounded alone would
// add as much error as the output's own rounding), within 2^-36 of the row's
// largest. Logits, maxima, sums and outputs are fp32.
//
// Both kernels compute the transposed products S^T = K . Q^T and
// O^T = V^T . P^T: a lane owns one query (a column), and S^T's accumulator is
// P^T's operand once the tile's tokens are dealt to S^T's rows so that a lane's
// registers hold 16 consecutive tokens, half a stored piece of the values.
#include "attention_internal.h"

namespace awq {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kUnit = 12.0f;      // log2 of the weights' unit
constexpr float kSlack = 3.0f;      // what a logit may pass the maximum by
constexpr float kTinyScale = 1.0e-30f;  // |scale log2 e| below it counts as it (a masked logit times 0 would be NaN)

// s and lo of the first n tokens, or of those from n on, as they are, of the
// others 0 (what none of the rows sees may be anything, NaN among it, and 0 times
// that is NaN)
__device__ inline half8_t first_n(half8_t v, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] : static_cast<half_t>(0.f);
    return v;
}
__device__ inline half8_t from_n(half8_t v, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? static_cast<half_t>(0.f) : v[j];
    return v;
}

// ---------------------------------------------------------------- few rows

// Decode: 16 query rows per block, or 32 in two sets whose products share the
// unpacked keys and values, the four waves walking the split's
// 64-token tiles in turn, each on its own, as over the 8-bit cache.
// v_mfma_f32_16x16x32_f16: lane l supplies row / column l % 16 and k-slots
// 8 (l / 16) .. + 7, and holds results 4 (l / 16) + e of column l % 16.
// S^T row r of sub-tile s4 is token 16 (r / 4) + 4 s4 + r % 4 of the tile, so
// quarter q of the wave holds the 16 tokens 16 q .. of its query. A quarter
// takes whole pieces of 32 channels of a key, piece q + 4 i (at 64 channels
// half a piece each), so a lane needs one (s, lo) per piece and token.
// Bound by HBM reads: 64 sequences of 8192 down to 2048 tokens, 8 heads of 128,
// 390 MB, 86-87 us, 4.5 TB/s (the kernel's loads alone 5.5; the VALU busy 66% of
// the time, the matrix cores 20%); 131072 and 131072 tokens 60 us, 5.2 TB/s.
// 1 x 1000 tokens of 32 heads 7.7-8.2 us, a row of latencies. One kv head leaves
// CUs idle: 1 x 262144 29 us (39 MB, 7.5 at a copy's rate), at most 128 blocks.
// Not faster: six, eight or sixteen waves a block, two tiles in flight, splits of
// 512 positions.
template <int D, int NP, int SETS>
__global__ __launch_bounds__(kDecodeWaves* kWave, SETS == 2 ? 2 : D <= 96 ? 4 : D <= 128 ? 3 : 2) void
kv4_decode_kernel(KvAttentionArgs a, Split sp, int n_splits, int row_tiles) {
    constexpr int PC = D / 32;              // pieces of a key
    constexpr bool HALF = D == 64;          // half pieces
    constexpr int KC = HALF ? 1 : (PC + 3) / 4;
    constexpr int KW = HALF ? 2 : 4;        // words of a lane's piece
    constexpr int DT = D / 16;              // 16-channel tiles of the output
    constexpr int NT = kDecodeWaves * kWave;
    constexpr int ROWS = 16 * SETS;
    constexpr int SO = D + 4;
    constexpr int kFloats = part_floats(ROWS, D);
    typedef uint32_t words_t __attribute__((ext_vector_type(KW)));
    __shared__ __attribute__((aligned(16))) float so_all[kDecodeWaves * ROWS * SO];
    float(*so)[ROWS][SO] = reinterpret_cast<float(*)[ROWS][SO]>(so_all);
    __shared__ float sm[kDecodeWaves][ROWS], sl[kDecodeWaves][ROWS];
    __shared__ int s_flag;

    const KvPages& c = a.c;
    const half2_t* k_scales = kv4_k_scales(c);
    const half_t* v_scales = kv4_v_scales(c);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    // Blocks go to the 8 XCDs in turn: heads run fastest, so that each XCD gets
    // splits of every sequence, and splits slowest, the last first, which only
    // long sequences have. (With splits fastest, two of them put every
    // sequence's first on the even XCDs and the seconds, often short or empty,
    // on the odd: 64 sequences of 8192 down to 2048 tokens 100 us, now 87.)
    const int kv_head = blockIdx.x;
    const int row0 = (blockIdx.y & (row_tiles - 1)) * ROWS;     // one row tile or two
    const int b = blockIdx.y >> (row_tiles - 1);
    const int split = n_splits - 1 - blockIdx.z;
    const KvSeq sq = kv_seq_shared(c, b);
    const int all_rows = rows_of(a, sq);
    if (row0 >= all_rows) return;
    const int rows = min(ROWS, all_rows - row0);
    const Span span = row_span(a, sq, row0, rows);
    // the splits that hold a visible position; none at all: split 0 writes zeros
    const int first_split = span.begin < span.end ? sp.by_tokens.of(span.begin) : 0;
    const int last_split = span.begin < span.end ? sp.by_tokens.of(span.end - 1) : 0;
    if (split < first_split || split > last_split) return;
    const int page = 1 << c.log2_page;
    const int from = max(span.begin, split * sp.tokens) / kTile;
    const int to = (min(static_cast<int64_t>(span.end), (static_cast<int64_t>(split) + 1) * sp.tokens) + kTile - 1) / kTile;

    // ---- queries, in LDS in operand order: word w of piece i holds the channels of
    // that word (in registers they are 16 to 32 a lane, and 256 channels leave room
    // for one wave per SIMD in place of two)
    __shared__ half8_t qs[SETS][KC * KW][kWave];
    int lo[SETS], hi[SETS];
#pragma unroll
    for (int r = 0; r < SETS; ++r) {
        const int row = row0 + 16 * r + col;
        lo[r] = hi[r] = 0;
        if (16 * r + col < rows) {
            const int token = a.by_ratio.of(row);
            visible(a, sq, token, lo[r], hi[r]);
            const half_t* q = a.q + (static_cast<int64_t>(sq.row0) + token) * a.q_token +
                              ((kv_head - token) * a.ratio + row) * a.q_head;
            for (int i = wave; i < KC * KW; i += kDecodeWaves) {
                const int first = (HALF ? 16 * quarter : 32 * (quarter + 4 * (i / KW))) + 8 * (i % KW);
                half8_t v = {};
                if (first < D) v = *reinterpret_cast<const half8_t*>(q + first);
                qs[r][i][lane] = a.scale_log2 < 0.f ? -v : v;
            }
        } else {
            for (int i = wave; i < KC * KW; i += kDecodeWaves) qs[r][i][lane] = half8_t{};
        }
    }
    __syncthreads();
    const float qscale = fmaxf(fabsf(a.scale_log2), kTinyScale);

    float m[SETS], sum[SETS];
    float4_t acc[SETS][DT];
#pragma unroll
    for (int r = 0; r < SETS; ++r) {
        m[r] = kNone;
        sum[r] = 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t) acc[r][t] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    // The pages of a tile: one or two, by scalar loads. A page past what the rows
    // see counts as not held, whatever its entry.
    struct Pages {
        int64_t block[NP];
        bool held[NP];
    };
    auto pages_of = [&](int tile) {
        Pages g;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = (tile * kTile >> c.log2_page) + i;
            const int id = (p << c.log2_page) < span.end ? kv_page_shared(c, b, p) : -1;
            g.held[i] = id >= 0;
            g.block[i] = static_cast<int64_t>(max(id, 0)) * c.heads + kv_head;
        }
        return g;
    };
    words_t kr[4][KC];
    half2_t ksc[4][KC];
    u32x2 vr[DT];
    half8_t vs[2], vlo[2];
    auto load_k = [&](int tile, const Pages& g) {
        const int slot = tile * kTile & (page - 1);
        // (block, piece) pieces of `page` tokens, 16 bytes and one (s, lo) each
        const int64_t base = (NP == 2 && (col >> 3) ? g.block[NP - 1] : g.block[0]) * PC;
        const int slot0 = NP == 2 ? 16 * ((col >> 2) & 1) + (col & 3) : slot + 16 * (col >> 2) + (col & 3);
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const int piece = HALF ? quarter >> 1 : min(quarter + 4 * i, PC - 1);   // past D: the queries' slots are 0
            const int64_t at = ((base + piece) << c.log2_page) + slot0;
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
                kr[s4][i] = *reinterpret_cast<const words_t*>(c.k_codes + (at + 4 * s4) * 16 + (HALF ? 8 * (quarter & 1) : 0));
                ksc[s4][i] = k_scales[at + 4 * s4];
            }
        }
    };
    auto load_v = [&](int tile, const Pages& g) {
        const int slot = tile * kTile & (page - 1);
        const int64_t block = NP == 2 && (quarter >> 1) ? g.block[NP - 1] : g.block[0];
        const int slot16 = NP == 2 ? 16 * (quarter & 1) : slot + 16 * quarter;      // the quarter's first token
        const uint8_t* base = c.v_codes + ((block * D) << (c.log2_page - 1)) +
                              ((slot16 >> 5) * D + col) * 16 + 8 * (quarter & 1);
#pragma unroll
        for (int t = 0; t < DT; ++t) vr[t] = *reinterpret_cast<const u32x2*>(base + 16 * 16 * t);
        const half_t* sc = v_scales + ((2 * block) << c.log2_page) + slot16;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            vs[j] = *reinterpret_cast<const half8_t*>(sc + 8 * j);
            vlo[j] = *reinterpret_cast<const half8_t*>(sc + page + 8 * j);
        }
    };

    // A tile's keys are in flight while the one before it is in its softmax
    // and second product, its values from the end of that product on; the
    // registers are those the tile before has just given up. The last tile's
    // wave asks for its own again (from the cache).
    int tile = from + wave;
    if (tile < to) {
        Pages now = pages_of(tile);
        load_k(tile, now);
        load_v(tile, now);
        for (; tile < to; tile += kDecodeWaves) {
            const int tb = tile * kTile;
            const int next = tile + kDecodeWaves < to ? tile + kDecodeWaves : tile;
            const Pages then = pages_of(next);

            // ---- logits (unscaled) ----
            float s[SETS][16];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
                float4_t x[SETS] = {};
#pragma unroll
                for (int i = 0; i < KC; ++i)
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const half8_t k = kv4_numbers8(kr[s4][i][w], ksc[s4][i]);
#pragma unroll
                        for (int r = 0; r < SETS; ++r)
                            x[r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qs[r][i * KW + w][lane], x[r], 0, 0, 0);
                    }
#pragma unroll
                for (int r = 0; r < SETS; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][4 * s4 + e] = x[r][e];
            }
            load_k(next, then);
            __builtin_amdgcn_sched_barrier(0);
            bool whole = tb >= span.all_begin && tb + kTile <= span.all_end;
#pragma unroll
            for (int i = 0; i < NP; ++i) whole = whole && now.held[i];
            if (!whole) {
                const bool ok = NP == 2 && quarter >= 2 ? now.held[NP - 1] : now.held[0];
                const int j0 = tb + 16 * quarter;
#pragma unroll
                for (int r = 0; r < SETS; ++r)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[r][i] = ok && j0 + i >= lo[r] && j0 + i < hi[r] ? s[r][i] : -__builtin_huge_valf();
                const int n = ok ? span.end - j0 : 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    vs[j] = first_n(vs[j], n - 8 * j);
                    vlo[j] = first_n(vlo[j], n - 8 * j);
                }
                if (span.begin > tb) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        vs[j] = from_n(vs[j], span.begin - j0 - 8 * j);
                        vlo[j] = from_n(vlo[j], span.begin - j0 - 8 * j);
                    }
                }
            }

            // ---- softmax ----
            half8_t pf[SETS][2], pl[SETS][2];
#pragma unroll
            for (int r = 0; r < SETS; ++r) {
                float top = s[r][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) top = fmaxf(top, s[r][i]);
                top = across_quarters_max(top) * qscale;
                if (__any(top > m[r] + kSlack)) {
                    const float mn = fmaxf(m[r], top);
                    const float carry = __builtin_amdgcn_exp2f(m[r] - mn);
                    sum[r] *= carry;
#pragma unroll
                    for (int t = 0; t < DT; ++t) acc[r][t] *= carry;
                    m[r] = mn;
                }
                const float shift = kUnit - m[r];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][i], qscale, shift));
                    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][i + 1], qscale, shift));
                    sum[r] += p0;
                    sum[r] += p1;
                    half2_t ph, pr;
                    two_parts(p0, p1, ph, pr);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        pf[r][i >> 3][(i & 7) + j] = ph[j];
                        pl[r][i >> 3][(i & 7) + j] = pr[j];
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                const half8_t v0 = kv4_numbers8(vr[t][0], vs[0], vlo[0]), v1 = kv4_numbers8(vr[t][1], vs[1], vlo[1]);
#pragma unroll
                for (int r = 0; r < SETS; ++r) {
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[r][0], acc[r][t], 0, 0, 0);
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[r][1], acc[r][t], 0, 0, 0);
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[r][0], acc[r][t], 0, 0, 0);
                    acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[r][1], acc[r][t], 0, 0, 0);
                }
            }
            load_v(next, then);
            __builtin_amdgcn_sched_barrier(0);
            now = then;
        }
    }

    // ---- the waves' results; sums and outputs carry 2^kUnit ----
#pragma unroll
    for (int r = 0; r < SETS; ++r) {
        sum[r] += __shfl_xor(sum[r], 16);
        sum[r] += __shfl_xor(sum[r], 32);
#pragma unroll
        for (int t = 0; t < DT; ++t)
            *reinterpret_cast<float4_t*>(&so[wave][16 * r + col][16 * t + 4 * quarter]) = acc[r][t];
        if (quarter == 0) {
            sm[wave][16 * r + col] = m[r] - kUnit;
            sl[wave][16 * r + col] = sum[r];
        }
    }
    __syncthreads();
    float mm = kNone, ll = 0.f;
    const int mine = tid % ROWS;
    float w[kDecodeWaves];
#pragma unroll
    for (int v = 0; v < kDecodeWaves; ++v) mm = fmaxf(mm, sm[v][mine]);
#pragma unroll
    for (int v = 0; v < kDecodeWaves; ++v) {
        w[v] = __builtin_amdgcn_exp2f(sm[v][mine] - mm);
        ll += w[v] * sl[v][mine];
    }
    for (int d = tid / ROWS * 4; d < D; d += NT / ROWS * 4) {
        float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kDecodeWaves; ++v) o += *reinterpret_cast<const float4_t*>(&so[v][mine][d]) * w[v];
        *reinterpret_cast<float4_t*>(&so[0][mine][d]) = o;
    }
    __syncthreads();
    if (tid < ROWS) {
        sm[0][tid] = mm;
        sl[0][tid] = ll;
    }
    __syncthreads();
    const int64_t tile_id = static_cast<int64_t>(blockIdx.y) * c.heads + kv_head;
    const Rows rw{kv_head, row0, rows, last_split - first_split + 1, split - first_split,
                  sp.partials + tile_id * n_splits * kFloats, static_cast<int64_t>(n_splits) * kFloats * 4,
                  sp.counters + tile_id};
    finish_rows<D, ROWS, NT, true>(a, sq, rw, [&](int p) { return (first_split + p) * kFloats; }, so_all, SO, &sm[0][0],
                                   &sl[0][0], so_all, &s_flag);
}

// ---------------------------------------------------------------- many rows

// Prefill: 128 query rows per block, 32 per wave. A 64-token tile of keys and
// values becomes fp16 numbers once per block, in LDS as 16-byte pieces in the
// operands' order, the next tile's bytes in flight meanwhile.
// v_mfma_f32_32x32x16_f16: lane l supplies row / column l % 32 and k-slots
// 8 (l / 32) .. + 7, and holds results 8 (i / 4) + 4 (l / 32) + i % 4 of
// column l % 32. S^T row r is token 16 ((r / 4) % 2) + 4 (r / 8) + r % 4 of a
// 32-token unit, so half h of the wave holds tokens 16 h + i.
// Wave w unpacks the values of tokens 16 w .. + 15, whose s and lo are then the
// wave's own: scalar loads.
// Bound by the matrix cores and the VALU, neither of them full (52% and 58%
// busy): 2 x 2048 tokens of 4096 (the second sequence's 1707 of 2560), 32 heads on 8
// of 128, 242-249 us on different cards, 607-623 TFLOP/s, or 905-930 with the
// weights' second parts, where a large matrix product reaches 1226. With one part,
// rounded, 200 us, and an error of 2.9e-4 in place of 2.1e-4. Not faster: the next
// tile's logits before this one's softmax, the instructions dealt out in a fixed
// order, raised wave priorities, eight waves.
template <int D, int NP>
__global__ __launch_bounds__(kPrefillWaves* kWave, D <= 128 ? 2 : 1) void kv4_prefill_kernel(KvAttentionArgs a, Split sp,
                                                                                           int n_splits) {
    constexpr int PC = D / 32;                      // pieces of a key
    constexpr int DC = D / 16;
    constexpr int DT = D / 32;
    constexpr int NT = kPrefillWaves * kWave;
    constexpr int K_PIECES = kTile * PC;            // 16-byte pieces of a tile's keys
    constexpr int KN = (K_PIECES + NT - 1) / NT;
    constexpr int VN = (D + kWave - 1) / kWave;     // channels of a lane, values
    constexpr int SO = D + 4;
    constexpr int kStage = kTile * D * 2;           // halves of one stage (keys, then values)
    constexpr size_t kBytes = std::max<size_t>(2 * kStage * sizeof(half_t), size_t{kPrefillRows} * SO * 4);
    static_assert(kTile / 16 == kPrefillWaves, "16 tokens of the values per wave");
    __shared__ __attribute__((aligned(16))) unsigned char lds[kBytes];
    __shared__ float sm[kPrefillRows], sl[kPrefillRows];
    __shared__ int s_flag;
    half8_t* kst[2];
    half8_t* vst[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        kst[i] = reinterpret_cast<half8_t*>(reinterpret_cast<half_t*>(lds) + i * kStage);
        vst[i] = kst[i] + kTile * D / 8;
    }

    const KvPages& c = a.c;
    const half2_t* k_scales = kv4_k_scales(c);
    const half_t* v_scales = kv4_v_scales(c);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    // Heads run fastest over the blocks, which go to the 8 XCDs in turn: with a
    // multiple of 8 heads the row tiles of one head share an XCD, and its L2
    // the head's keys and values. The last rows of a causal chunk see the
    // most: first.
    const int b = blockIdx.z;
    const int kv_head = blockIdx.x % c.heads;
    const int rest = blockIdx.x / c.heads;
    const int split = rest % n_splits;
    const int row_tiles = gridDim.x / c.heads / n_splits;
    const int row_tile = row_tiles - 1 - rest / n_splits;
    const int row0 = row_tile * kPrefillRows;
    const KvSeq sq = kv_seq_shared(c, b);
    const int all_rows = rows_of(a, sq);
    if (row0 >= all_rows) return;
    const int rows = min(kPrefillRows, all_rows - row0);
    const Span span = row_span(a, sq, row0, rows);
    const int first_split = span.begin < span.end ? sp.by_tokens.of(span.begin) : 0;
    const int last_split = span.begin < span.end ? sp.by_tokens.of(span.end - 1) : 0;
    if (split < first_split || split > last_split) return;

    const int wrow = wave * 32 + col;
    int lo = 0, hi = 0;
    half8_t qf[DC];
#pragma unroll
    for (int i = 0; i < DC; ++i) qf[i] = half8_t{};
    if (wrow < rows) {
        const int token = a.by_ratio.of(row0 + wrow);
        visible(a, sq, token, lo, hi);
        const half_t* q = a.q + (static_cast<int64_t>(sq.row0) + token) * a.q_token +
                          ((kv_head - token) * a.ratio + row0 + wrow) * a.q_head;
#pragma unroll
        for (int i = 0; i < DC; ++i) {
            qf[i] = *reinterpret_cast<const half8_t*>(q + 16 * i + 8 * half);
            if (a.scale_log2 < 0.f) qf[i] = -qf[i];
        }
    }
    const float qscale = fmaxf(fabsf(a.scale_log2), kTinyScale);
    // what this wave's rows see
    const Span wspan = wave * 32 < rows ? row_span(a, sq, row0 + wave * 32, min(32, rows - wave * 32))
                                        : Span{0, 0, 0, 0};

    const int page = 1 << c.log2_page;
    const int from = max(span.begin, split * sp.tokens) / kTile;
    const int to = (min(static_cast<int64_t>(span.end), (static_cast<int64_t>(split) + 1) * sp.tokens) + kTile - 1) / kTile;

    struct Pages {
        bool held[NP];
    };
    // token of a 32-token unit that S^T row r holds
    auto token_of = [](int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); };
    kv_u32x4 kr[KN];
    half2_t ksc[KN];
    u32x2 vr[VN];
    half8_t vs[2], vlo[2];      // of the wave's 16 tokens
    auto load = [&](int tile, Pages& pg) {
        const int tb = tile * kTile;
        int64_t block[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = (tb >> c.log2_page) + i;
            // a page past what the rows see counts as not held, whatever its entry
            const int id = (p << c.log2_page) < span.end ? kv_page_shared(c, b, p) : -1;
            pg.held[i] = id >= 0;
            block[i] = static_cast<int64_t>(max(id, 0)) * c.heads + kv_head;
        }
        const int slot0 = NP == 2 ? 0 : tb & (page - 1);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int e = tid + i * NT;
            if (K_PIECES % NT != 0 && e >= K_PIECES) break;
            // key piece: the token of S^T row e % 64 (so that both the LDS write
            // and the operand reads are of neighbouring pieces), channels 32 ch ..
            const int t = (e & 32) + token_of(e & 31), ch = e / kTile;
            const int64_t at = (((NP == 2 && t >= 32 ? block[NP - 1] : block[0]) * PC + ch) << c.log2_page) +
                               (NP == 2 ? t & 31 : slot0 + t);
            kr[i] = *reinterpret_cast<const kv_u32x4*>(c.k_codes + at * 16);
            ksc[i] = k_scales[at];
        }
        const int64_t vblock = NP == 2 && wave >= 2 ? block[NP - 1] : block[0];
        const int slot16 = NP == 2 ? 16 * (wave & 1) : slot0 + 16 * wave;
        const uint8_t* base = c.v_codes + ((vblock * D) << (c.log2_page - 1)) + (slot16 >> 5) * D * 16 + 8 * (wave & 1);
#pragma unroll
        for (int i = 0; i < VN; ++i)
            vr[i] = *reinterpret_cast<const u32x2*>(base + min(lane + i * kWave, D - 1) * 16);
        const half_t* sc = v_scales + ((2 * vblock) << c.log2_page) + slot16;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            vs[j] = __builtin_bit_cast(half8_t, kv_shared_load(reinterpret_cast<const kv_u32x4*>(sc + 8 * j)));
            vlo[j] = __builtin_bit_cast(half8_t, kv_shared_load(reinterpret_cast<const kv_u32x4*>(sc + page + 8 * j)));
        }
    };
    auto stage = [&](int tile, const Pages& pg, half8_t* ks, half8_t* vst_) {
        const int tb = tile * kTile;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int e = tid + i * NT;
            if (K_PIECES % NT != 0 && e >= K_PIECES) break;
            const int t = e % kTile, ch = e / kTile;
#pragma unroll
            for (int w = 0; w < 4; ++w) ks[(4 * ch + w) * kTile + t] = kv4_numbers8(kr[i][w], ksc[i]);
        }
        const int n = (pg.held[NP == 2 ? wave >> 1 : 0] ? span.end : 0) - (tb + 16 * wave);
        if (n < 16) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                vs[j] = first_n(vs[j], n - 8 * j);
                vlo[j] = first_n(vlo[j], n - 8 * j);
            }
        }
        if (span.begin > tb) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                vs[j] = from_n(vs[j], span.begin - tb - 16 * wave - 8 * j);
                vlo[j] = from_n(vlo[j], span.begin - tb - 16 * wave - 8 * j);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int d = lane + i * kWave;
            if (D % kWave != 0 && d >= D) break;
#pragma unroll
            for (int j = 0; j < 2; ++j) vst_[(2 * wave + j) * D + d] = kv4_numbers8(vr[i][j], vs[j], vlo[j]);
        }
    };

    float m = kNone, sum = 0.f;
    float16_t acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[t][e] = 0.f;

    auto compute = [&](int tile, const Pages& pg, const half8_t* ks, const half8_t* vst_) {
        const int tb = tile * kTile;
        if (tb >= wspan.end || tb + kTile <= wspan.begin) return;      // none of this wave's rows sees it
        float16_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[u][e] = 0.f;
#pragma unroll
            for (int i = 0; i < DC; ++i)
                s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ks[(2 * i + half) * kTile + 32 * u + col], qf[i], s[u], 0,
                                                              0, 0);
        }
        bool whole = tb >= wspan.all_begin && tb + kTile <= wspan.all_end;
#pragma unroll
        for (int i = 0; i < NP; ++i) whole = whole && pg.held[i];
        if (!whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = tb + 32 * u + 16 * half + e;
                    s[u][e] = pg.held[NP == 2 ? u : 0] && j >= lo && j < hi ? s[u][e] : -__builtin_huge_valf();
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[u][e]);
        top = across_halves_max(top) * qscale;
        if (__any(top > m + kSlack)) {
            const float mn = fmaxf(m, top);
            const float carry = __builtin_amdgcn_exp2f(m - mn);
            sum *= carry;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[t][e] *= carry;
            m = mn;
        }
        // one unit's weights, then its products: the next unit's exponentials
        // run beside them
        const float shift = kUnit - m;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            half8_t pf[2], pl[2];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e + j], qscale, shift));
                    sum += w[j];
                }
                half2_t ph, pr;
                two_parts(w[0], w[1], ph, pr);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pf[e >> 3][(e & 7) + j] = ph[j];
                    pl[e >> 3][(e & 7) + j] = pr[j];
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    const half8_t v = vst_[(4 * u + 2 * half + k) * D + 32 * t + col];
                    acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pf[k], acc[t], 0, 0, 0);
                    acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pl[k], acc[t], 0, 0, 0);
                }
        }
    };

    if (from < to) {
        Pages pg[2];
        load(from, pg[0]);
        stage(from, pg[0], kst[0], vst[0]);
        __syncthreads();
        for (int tile = from; tile < to; tile += 2) {
            if (tile + 1 < to) load(tile + 1, pg[1]);
            compute(tile, pg[0], kst[0], vst[0]);
            if (tile + 1 >= to) break;
            stage(tile + 1, pg[1], kst[1], vst[1]);
            __syncthreads();
            if (tile + 2 < to) load(tile + 2, pg[0]);
            compute(tile + 1, pg[1], kst[1], vst[1]);
            if (tile + 2 < to) stage(tile + 2, pg[0], kst[0], vst[0]);
            __syncthreads();
        }
    }
    __syncthreads();        // the stages are free: the outputs take their place

    sum += __shfl_xor(sum, 32);
    float* so = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4_t*>(so + wrow * SO + 32 * t + 8 * q + 4 * half) =
                float4_t{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
    if (half == 0) {
        sm[wrow] = m - kUnit;       // sums and outputs carry 2^kUnit
        sl[wrow] = sum;
    }
    __syncthreads();
    const int64_t tile_id = (static_cast<int64_t>(b) * c.heads + kv_head) * row_tiles + row_tile;
    constexpr int kFloats = part_floats(kPrefillRows, D);
    const Rows rw{kv_head, row0, rows, last_split - first_split + 1, split - first_split,
                  sp.partials + tile_id * n_splits * kFloats, static_cast<int64_t>(n_splits) * kFloats * 4,
                  sp.counters + tile_id};
    finish_rows<D, kPrefillRows, NT>(a, sq, rw, [&](int p) { return (first_split + p) * kFloats; }, so, SO, sm, sl, so,
                                     &s_flag);
    static_assert(kBytes >= join_floats(kPrefillRows, NT) * 4, "room for the join");
}

// ---------------------------------------------------------------- launch

template <int D, int NP>
awq_status launch_np(const KvAttentionArgs& a, const Plan& p, const Split& sp, hipStream_t stream) {
    const auto decode = [&](auto sets) {
        hipLaunchKernelGGL((kv4_decode_kernel<D, NP, decltype(sets)::value>),
                           dim3(static_cast<unsigned>(a.c.heads), static_cast<unsigned>(p.row_tiles * a.n_seqs),
                                static_cast<unsigned>(p.splits)),
                           dim3(kDecodeWaves * kWave), 0, stream, a, sp, p.splits, static_cast<int>(p.row_tiles));
    };
    if (!p.decode) {
        hipLaunchKernelGGL((kv4_prefill_kernel<D, NP>),
                           dim3(static_cast<unsigned>(p.row_tiles * p.splits * a.c.heads), 1,
                                static_cast<unsigned>(a.n_seqs)),
                           dim3(kPrefillWaves * kWave), 0, stream, a, sp, p.splits);
    } else if (p.rows == kDecodeRows) {
        decode(std::integral_constant<int, 1>{});
    } else if constexpr (D <= kWideDim) {
        decode(std::integral_constant<int, 2>{});
    } else {
        return AWQ_ERR_CONFIG;      // no plan asks for it
    }
    return last_launch_status();
}
template <int D>
awq_status launch_d(const KvAttentionArgs& a, const Plan& p, const Split& sp, hipStream_t stream) {
    return a.c.log2_page == 5 ? launch_np<D, 2>(a, p, sp, stream) : launch_np<D, 1>(a, p, sp, stream);
}

}  // namespace

awq_status launch_kv4_attention(const KvAttentionArgs& a, void* workspace, hipStream_t stream) {
    const Plan p = plan_for(a.format, a.head_dim, a.n_seqs, a.c.heads, a.ratio, a.max_tokens, a.c.max_len, workspace != nullptr);
    if (!launchable(p, a.c.heads)) return AWQ_ERR_SHAPE;
    const Split sp = split_of(p, workspace);
    switch (a.head_dim) {
        case 64: return launch_d<64>(a, p, sp, stream);
        case 96: return launch_d<96>(a, p, sp, stream);
        case 128: return launch_d<128>(a, p, sp, stream);
        case 192: return launch_d<192>(a, p, sp, stream);
        case 256: return launch_d<256>(a, p, sp, stream);
        default: return AWQ_ERR_CONFIG;
    }
}

}  // namespace awq
