// Softmax attention of a batch's newest tokens over the paged 8-bit cache
// (include/awq.h, awq_kv_attention).
//
// Mathematics. A tile of keys gives logits t = ks * (q . kc) * scale * log2 e
// from the exact fp16 numbers kc of the stored bytes; with the running
// maximum m the weights are p = 2^(t - m), and sums and outputs carried from
// earlier tiles are multiplied by 2^(m_old - m). The values' page scale
// vs = f 2^e (1/2 <= f < 1) goes into the weights: the outputs have a maximum
// of their own, M, a whole number that is at least every t + e seen by the
// row, and f 2^(t + e - M) times a power of two (2^15 in decode, 2^12 in
// prefill, where t + e may pass M by 3) is what enters the second product, as
// two fp16 numbers: it cut to fp16, and what that left. (The rounding of one
// alone would add as much error as the output's own: 2.9e-4 of a prefill's
// outputs against 2.07e-4, of which 2.07e-4 is the output's.) A row's largest
// weight times scale is at least 2^13 (2^10) in these units, and what fp16's
// subnormals lose is at most 2^-37 (2^-34) of it for each key, however far
// the pages' scales lie apart and whatever scales the masked pages have.
// (Both exponents stay whole where scales enter, so no bits go with them.)
// Logits, maxima, sums and outputs are fp32.
//
// Both kernels compute the transposed products: S^T = K . Q^T and
// O^T = V^T . P^T. A lane then owns one query (a column), so the softmax's
// statistics are a few registers per lane, and S^T's accumulator layout is
// P^T's operand layout once the tile's tokens are dealt to S^T's rows so
// that a lane's registers hold the 16 consecutive tokens of one piece of the
// stored values. Nothing moves between lanes but the row maxima.
//
// Rows. The query rows of a kv head are its tokens times the r query heads
// that share it (row = token * ratio + head), so grouped heads read each key
// once.
#include "attention_internal.h"

namespace awq {
namespace {

constexpr float kWeightUnit = 15.0f;    // log2 of the unit of the rounded weights
constexpr float kPrefillUnit = 12.0f;   // the same in prefill
constexpr float kSlack = 3.0f;          // what t and t + e may pass their maxima by there
constexpr float kTinyScale = 1.0e-20f;  // scales at or below it count as it

// Ones in the first n bytes of 16.
__device__ inline kv_u32x4 first_bytes(int n) {
    kv_u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = min(max(n - 4 * j, 0), 4);
        r[j] = k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
    }
    return r;
}
// whether any of the rows sees a position of page p
__device__ inline bool seen(const Span& s, int p, int log2_page) {
    return (p << log2_page) < s.end && (p + 1) << log2_page > s.begin;
}

// ---------------------------------------------------------------- few rows

// Decode: up to 16 query rows per block. The four waves walk the split's
// 64-token tiles in turn, each on its own (no LDS in the loop), straight from
// the cache into MFMA operands, and are joined in LDS at the end.
// v_mfma_f32_16x16x32_f16: lane l supplies row / column l % 16 and k-slots
// 8 (l / 16) .. + 7, and holds results 4 (l / 16) + e of column l % 16.
// S^T row r of sub-tile s4 (0 .. 3) is token 16 (r / 4) + 4 s4 + r % 4 of the
// tile: quarter q of the wave then holds the 16 tokens 16 q .. of its query,
// whose values are one 16-byte piece per channel. (A load thus takes 64-byte
// runs of keys; whole kilobytes in a copy of the loop without the arithmetic
// read no faster, 6.0 against 6.1 TB/s.)
// Bound by HBM: 2 D bytes per cached token and kv head. Measured (one MI355X,
// int8, 128 channels): 64 sequences of 8192 down to 2048 tokens, 64 heads on
// 8, 680 MB, 126-134 us, 5.1-5.4 TB/s, the ragged lengths leaving few waves
// at the end; 32 of 2048 down, 32 heads, 63 us, 5.4 TB/s; 2 of 131072 and
// 81920 (e4m3, 8 heads) 84-88 us, 5.0-5.2 TB/s; a plain read reaches 6.1 to
// 6.2. The 163 VGPRs at 128 channels leave room for three blocks per CU, where
// 190 left two: no difference was measured. Non-temporal loads gained 7% on
// the 680 MB case and lost as much on caches that the 256 MB last-level cache
// holds.
// NP: pages a 64-token tile spans (2 for pages of 32, else 1)
template <int D, int FORMAT, int NP>
__global__ __launch_bounds__(kDecodeWaves* kWave, D <= 64 ? 4 : D <= 96 ? 3 : D <= 192 ? 2 : 1) void kv_decode_kernel(
    KvAttentionArgs a, Split sp, int n_splits) {
    constexpr int DC = D / 16;              // channel pieces of a key
    constexpr int KC = (DC + 3) / 4;        // of them per lane
    constexpr int DT = D / 16;              // 16-channel tiles of the output
    constexpr int NT = kDecodeWaves * kWave;
    constexpr int SO = D + 4;
    constexpr int kFloats = part_floats(kDecodeRows, D);
    __shared__ __attribute__((aligned(16))) float so_all[std::max(kDecodeWaves * kDecodeRows * SO,
                                                                 join_floats(kDecodeRows, NT))];
    float(*so)[kDecodeRows][SO] = reinterpret_cast<float(*)[kDecodeRows][SO]>(so_all);
    __shared__ float sm[kDecodeWaves][kDecodeRows], sl[kDecodeWaves][kDecodeRows];
    __shared__ int s_flag;

    const KvPages& c = a.c;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int split = blockIdx.x;
    const int b = blockIdx.z;
    const int kv_head = blockIdx.y % c.heads;
    const int row0 = blockIdx.y / c.heads * kDecodeRows;
    const KvSeq sq = kv_seq_shared(c, b);
    const int all_rows = rows_of(a, sq);
    if (row0 >= all_rows) return;
    const int rows = min(kDecodeRows, all_rows - row0);
    const Span span = row_span(a, sq, row0, rows);
    // the splits that hold a visible position; none at all: split 0 writes zeros
    const int first_split = span.begin < span.end ? sp.by_tokens.of(span.begin) : 0;
    const int last_split = span.begin < span.end ? sp.by_tokens.of(span.end - 1) : 0;
    if (split < first_split || split > last_split) return;
    const int page_mask = (1 << c.log2_page) - 1;
    const int64_t page_bytes = static_cast<int64_t>(D) << c.log2_page;
    const int from = max(span.begin, split * sp.tokens) / kTile;
    const int to = (min(static_cast<int64_t>(span.end), (static_cast<int64_t>(split) + 1) * sp.tokens) + kTile - 1) / kTile;

    // ---- queries: k-slots of step 2 i + h are channels 16 (quarter + 4 i) + 8 h .. + 7 ----
    const int row = row0 + col;
    int lo = 0, hi = 0;
    half8_t qf[2 * KC];
#pragma unroll
    for (int i = 0; i < 2 * KC; ++i) qf[i] = half8_t{};
    if (col < rows) {
        const int token = a.by_ratio.of(row);
        visible(a, sq, token, lo, hi);
        const half_t* q = a.q + (static_cast<int64_t>(sq.row0) + token) * a.q_token +
                          ((kv_head - token) * a.ratio + row) * a.q_head;
#pragma unroll
        for (int i = 0; i < KC; ++i)
            if (quarter + 4 * i < DC) {
                qf[2 * i] = *reinterpret_cast<const half8_t*>(q + 16 * (quarter + 4 * i));
                qf[2 * i + 1] = *reinterpret_cast<const half8_t*>(q + 16 * (quarter + 4 * i) + 8);
            }
    }

    float m = kNone, om = kNone, sum = 0.f;     // om: the outputs' maximum
    float4_t acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};

    // The pages of a tile: one or two, by scalar loads. A page that none of the
    // rows sees counts as not held, whatever its entry: its scales may be anything.
    struct Pages {
        int64_t block[NP];
        bool held[NP];
    };
    auto pages_of = [&](int tile) {
        Pages g;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = (tile * kTile >> c.log2_page) + i;
            const int id = seen(span, p, c.log2_page) ? kv_page_shared(c, b, p) : -1;
            g.held[i] = id >= 0;
            g.block[i] = static_cast<int64_t>(max(id, 0)) * c.heads + kv_head;
        }
        return g;
    };
    kv_u32x4 kr[4][KC], vr[DT];
    auto load_k = [&](int tile, const Pages& g) {
        const int slot = tile * kTile & page_mask;
        const uint8_t* base = c.k_codes + (NP == 2 && (col >> 3) ? g.block[NP - 1] : g.block[0]) * page_bytes;
        const int slot0 = NP == 2 ? 16 * ((col >> 2) & 1) + (col & 3) : slot + 16 * (col >> 2) + (col & 3);
#pragma unroll
        for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const int piece = min(quarter + 4 * i, DC - 1);     // past D: the queries' slots are 0
                kr[s4][i] = *reinterpret_cast<const kv_u32x4*>(base + ((piece << c.log2_page) + slot0 + 4 * s4) * 16);
            }
    };
    auto load_v = [&](int tile, const Pages& g) {
        const int slot = tile * kTile & page_mask;
        const uint8_t* base = c.v_codes + (NP == 2 && (quarter >> 1) ? g.block[NP - 1] : g.block[0]) * page_bytes;
        const int piece0 = NP == 2 ? quarter & 1 : (slot >> 4) + quarter;
#pragma unroll
        for (int t = 0; t < DT; ++t)
            vr[t] = *reinterpret_cast<const kv_u32x4*>(base + (piece0 * D + 16 * t + col) * 16);
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
            float ks[NP], vs[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                ks[i] = now.held[i] ? kv_shared_load(c.k_scales + now.block[i]) : 0.f;
                vs[i] = now.held[i] ? fmaxf(kv_shared_load(c.v_scales + now.block[i]), kTinyScale) : kTinyScale;
            }

            // ---- logits ----
            float s[16];
            const float kscale = (NP == 2 && quarter >= 2 ? ks[NP - 1] : ks[0]) * a.scale_log2;
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
                float4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KC; ++i) {
                    x = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv_unpack8<FORMAT>(kr[s4][i][0], kr[s4][i][1]),
                                                               qf[2 * i], x, 0, 0, 0);
                    x = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv_unpack8<FORMAT>(kr[s4][i][2], kr[s4][i][3]),
                                                               qf[2 * i + 1], x, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[4 * s4 + e] = x[e] * kscale;
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
                for (int i = 0; i < 16; ++i)
                    s[i] = ok && j0 + i >= lo && j0 + i < hi ? s[i] : -__builtin_huge_valf();
                // bytes that none of the rows sees may be anything, fp8 NaN among them
                kv_u32x4 keep = first_bytes(ok ? span.end - j0 : 0);
                if (span.begin > tb) keep &= ~first_bytes(span.begin - j0);
#pragma unroll
                for (int t = 0; t < DT; ++t) vr[t] &= keep;
            }

            // ---- softmax ----
            const float scale = NP == 2 && quarter >= 2 ? vs[NP - 1] : vs[0];
            const float vm = __builtin_amdgcn_frexp_mantf(scale);
            const float ve = static_cast<float>(__builtin_amdgcn_frexp_expf(scale));
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
            const float out_top = NP == 2 ? across_quarters_max(top + ve) : 0.f;
            top = across_quarters_max(top);
            const float mn = fmaxf(m, top);
            const float on = fmaxf(om, __builtin_ceilf(NP == 2 ? out_top : top + ve));
            const float shrink = __builtin_amdgcn_exp2f(m - mn);
            const float carry = __builtin_amdgcn_exp2f(om - on);
            const float shift = ve + kWeightUnit - on;
            // (the second part's matrix time is free here)
            half8_t pf[2], pl[2];
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float p0 = __builtin_amdgcn_exp2f(s[i] + shift), p1 = __builtin_amdgcn_exp2f(s[i + 1] + shift);
                part += p0;
                part += p1;
                half2_t hi, lo;
                two_parts(p0 * vm, p1 * vm, hi, lo);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pf[i >> 3][(i & 7) + j] = hi[j];
                    pl[i >> 3][(i & 7) + j] = lo[j];
                }
            }
            sum = __builtin_fmaf(part, __builtin_amdgcn_exp2f(on - mn - (ve + kWeightUnit)), sum * shrink);
            m = mn;
            om = on;
#pragma unroll
            for (int t = 0; t < DT; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] *= carry;
                const half8_t v0 = kv_unpack8<FORMAT>(vr[t][0], vr[t][1]), v1 = kv_unpack8<FORMAT>(vr[t][2], vr[t][3]);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[0], acc[t], 0, 0, 0);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[1], acc[t], 0, 0, 0);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pl[0], acc[t], 0, 0, 0);
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pl[1], acc[t], 0, 0, 0);
            }
            load_v(next, then);
            __builtin_amdgcn_sched_barrier(0);
            now = then;
        }
    }

    // ---- the waves' results, in true units ----
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    const float true_unit = __builtin_amdgcn_exp2f(om - m - kWeightUnit);
#pragma unroll
    for (int t = 0; t < DT; ++t) *reinterpret_cast<float4_t*>(&so[wave][col][16 * t + 4 * quarter]) = acc[t] * true_unit;
    if (quarter == 0) {
        sm[wave][col] = m;
        sl[wave][col] = sum;
    }
    __syncthreads();
    float mm = kNone, ll = 0.f;
    const int r16 = tid % kDecodeRows;
    float w[kDecodeWaves];
#pragma unroll
    for (int v = 0; v < kDecodeWaves; ++v) mm = fmaxf(mm, sm[v][r16]);
#pragma unroll
    for (int v = 0; v < kDecodeWaves; ++v) {
        w[v] = __builtin_amdgcn_exp2f(sm[v][r16] - mm);
        ll += w[v] * sl[v][r16];
    }
    for (int d = tid / kDecodeRows * 4; d < D; d += NT / kDecodeRows * 4) {
        float4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kDecodeWaves; ++v) o += *reinterpret_cast<const float4_t*>(&so[v][r16][d]) * w[v];
        *reinterpret_cast<float4_t*>(&so[0][r16][d]) = o;
    }
    __syncthreads();
    if (tid < kDecodeRows) {
        sm[0][tid] = mm;
        sl[0][tid] = ll;
    }
    __syncthreads();
    const int64_t tile_id = static_cast<int64_t>(b) * gridDim.y + blockIdx.y;
    const Rows rw{kv_head, row0, rows, last_split - first_split + 1, split - first_split,
                  sp.partials + tile_id * n_splits * kFloats, static_cast<int64_t>(n_splits) * kFloats * 4,
                  sp.counters + tile_id};
    finish_rows<D, kDecodeRows, NT>(a, sq, rw, [&](int p) { return (first_split + p) * kFloats; }, so_all, SO, &sm[0][0],
                                    &sl[0][0], so_all, &s_flag);
}

// ---------------------------------------------------------------- many rows

// Prefill: 128 query rows per block, 32 per wave. A 64-token tile of keys and
// values is unpacked to fp16 once per block, into LDS as 16-byte pieces in
// the operands' order (keys: 8 channels of a token, values: 8 tokens of a
// channel; neighbouring lanes read neighbouring pieces, so without bank
// conflicts), the next tile's bytes in flight meanwhile.
// v_mfma_f32_32x32x16_f16: lane l supplies row / column l % 32 and k-slots
// 8 (l / 32) .. + 7, and holds results 8 (i / 4) + 4 (l / 32) + i % 4 of
// column l % 32. S^T row r is token 16 ((r / 4) % 2) + 4 (r / 8) + r % 4 of a
// 32-token unit, so half h of the wave holds tokens 16 h + i.
// Bound by neither unit alone: per wave and tile some 390 vector instructions
// (32 of them exponentials, 64 to unpack) and 48 MFMAs, the counters reading
// 56% and 51% of the time, which two waves per SIMD (206 VGPRs) overlap in
// part. 16 of the 48 are the weights' second parts. Measured (8 kv heads of
// 128, 32 query heads, causal; us, in brackets with one part): 2 x 2048
// tokens of 4096 247 (197), 609 TFLOP/s, e4m3 241 (184); 8192 of 8192 785
// (607); 64 channels 146 (110); 4 kv heads of 192 213 (186), of 256 277
// (240). A large fp16 matrix product reaches 1158 TFLOP/s.
template <int D, int FORMAT, int NP>
__global__ __launch_bounds__(kPrefillWaves* kWave, D <= 128 ? 2 : 1) void kv_prefill_kernel(KvAttentionArgs a, Split sp,
                                                                                          int n_splits) {
    constexpr int DC = D / 16;
    constexpr int DT = D / 32;
    constexpr int NT = kPrefillWaves * kWave;
    constexpr int TILE_PIECES = kTile * DC;         // stored 16-byte pieces of a tile, keys and values each
    constexpr int PIECES = (TILE_PIECES + NT - 1) / NT;
    constexpr int SO = D + 4;
    constexpr int kStage = kTile * D * 2;           // halves of one stage (keys, then values)
    constexpr size_t kBytes = std::max<size_t>(2 * kStage * sizeof(half_t), size_t{kPrefillRows} * SO * 4);
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
    const float qscale = fabsf(a.scale_log2);
    // what this wave's rows see
    const Span wspan = wave * 32 < rows ? row_span(a, sq, row0 + wave * 32, min(32, rows - wave * 32))
                                        : Span{0, 0, 0, 0};

    const int page_mask = (1 << c.log2_page) - 1;
    const int64_t page_bytes = static_cast<int64_t>(D) << c.log2_page;
    const int from = max(span.begin, split * sp.tokens) / kTile;
    const int to = (min(static_cast<int64_t>(span.end), (static_cast<int64_t>(split) + 1) * sp.tokens) + kTile - 1) / kTile;

    struct Pages {
        bool held[NP];
        float ks[NP], vs[NP];
    };
    // token of a 32-token unit that S^T row r holds
    auto token_of = [](int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); };
    kv_u32x4 kr[PIECES], vr[PIECES];
    auto load = [&](int tile, Pages& pg) {
        const int tb = tile * kTile;
        int64_t block[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = (tb >> c.log2_page) + i;
            // a page that none of the rows sees counts as not held, whatever its entry
            const int id = seen(span, p, c.log2_page) ? kv_page_shared(c, b, p) : -1;
            pg.held[i] = id >= 0;
            block[i] = static_cast<int64_t>(max(id, 0)) * c.heads + kv_head;
            pg.ks[i] = pg.held[i] ? kv_shared_load(c.k_scales + block[i]) : 0.f;
            pg.vs[i] = pg.held[i] ? fmaxf(kv_shared_load(c.v_scales + block[i]), kTinyScale) : kTinyScale;
        }
        const int slot0 = NP == 2 ? 0 : tb & page_mask;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int e = tid + i * NT;
            if (TILE_PIECES % NT != 0 && e >= TILE_PIECES) break;
            // key piece: the token of S^T row e % 64 (so that both the LDS write
            // and the operand reads are of neighbouring pieces), channels 16 ch ..
            const int t = (e & 32) + token_of(e & 31), ch = e / kTile;
            const int kslot = NP == 2 ? t & 31 : slot0 + t;
            kr[i] = *reinterpret_cast<const kv_u32x4*>(c.k_codes + (NP == 2 && t >= 32 ? block[NP - 1] : block[0]) * page_bytes +
                                                       ((ch << c.log2_page) + kslot) * 16);
            const int d = e % D, tc = e / D;                    // value piece: channel d, tokens 16 tc ..
            const int vpiece = NP == 2 ? tc & 1 : (slot0 >> 4) + tc;
            vr[i] = *reinterpret_cast<const kv_u32x4*>(c.v_codes + (NP == 2 && tc >= 2 ? block[NP - 1] : block[0]) * page_bytes +
                                                       (vpiece * D + d) * 16);
        }
    };
    auto stage = [&](int tile, const Pages& pg, half8_t* ks, half8_t* vs) {
        const int tb = tile * kTile;
        bool whole = tb >= span.begin && tb + kTile <= span.end;
#pragma unroll
        for (int i = 0; i < NP; ++i) whole = whole && pg.held[i];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int e = tid + i * NT;
            if (TILE_PIECES % NT != 0 && e >= TILE_PIECES) break;
            const int t = e % kTile, ch = e / kTile;
            ks[(2 * ch) * kTile + t] = kv_unpack8<FORMAT>(kr[i][0], kr[i][1]);
            ks[(2 * ch + 1) * kTile + t] = kv_unpack8<FORMAT>(kr[i][2], kr[i][3]);
            const int d = e % D, tc = e / D;
            if (!whole) {
                // bytes that none of the rows sees may be anything, fp8 NaN among them
                const bool ok = NP == 2 && tc >= 2 ? pg.held[NP - 1] : pg.held[0];
                const int j0 = tb + 16 * tc;
                vr[i] &= first_bytes(ok ? span.end - j0 : 0);
                if (span.begin > tb) vr[i] &= ~first_bytes(span.begin - j0);
            }
            vs[(2 * tc) * D + d] = kv_unpack8<FORMAT>(vr[i][0], vr[i][1]);
            vs[(2 * tc + 1) * D + d] = kv_unpack8<FORMAT>(vr[i][2], vr[i][3]);
        }
    };

    float m = kNone, om = kNone, sum = 0.f;     // om: the outputs' maximum
    float16_t acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[t][e] = 0.f;

    auto compute = [&](int tile, const Pages& pg, const half8_t* ks, const half8_t* vs) {
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
        // ---- softmax: the logits stay unscaled, the page's scale (over 0, the
        // sign of `scale` is in the queries) goes into the exponent's fma, and
        // so do the values' scale and the weights' unit:
        //   2^(x kscale + log2 f + (e + 12 - M)), the bracket exact
        float top[2], ksc[2], vm[2], ve[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ksc[u] = fmaxf(pg.ks[NP == 2 ? u : 0] * qscale, kTinyScale);
            vm[u] = __builtin_amdgcn_frexp_mantf(pg.vs[NP == 2 ? u : 0]);
            ve[u] = static_cast<float>(__builtin_amdgcn_frexp_expf(pg.vs[NP == 2 ? u : 0]));
            top[u] = s[u][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top[u] = fmaxf(top[u], s[u][e]);
            top[u] *= ksc[u];
        }
        const float mt = across_halves_max(fmaxf(top[0], top[1]));
        const float ot = NP == 2 ? across_halves_max(fmaxf(top[0] + ve[0], top[1] + ve[1])) : mt + ve[0];
        // The maxima move only when one would be passed by 3 (weights stay
        // below 2^15): rarely after the first tiles, and the outputs need no
        // rescaling until then.
        if (__any(mt > m + kSlack || ot > om + kSlack)) {
            const float mn = fmaxf(m, mt), on = fmaxf(om, __builtin_ceilf(ot));
            const float carry = __builtin_amdgcn_exp2f(om - on);
            sum *= __builtin_amdgcn_exp2f(m - mn);
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[t][e] *= carry;
            m = mn;
            om = on;
        }
        // one unit's weights, then its products: the next unit's exponentials
        // run beside them
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            half8_t pf[2], pl[2];
            const float shift = __builtin_amdgcn_logf(vm[u]) + (ve[u] + kPrefillUnit - om);
            float part = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e + j], ksc[u], shift));
                    part += w[j];
                }
                half2_t hi, lo;
                two_parts(w[0], w[1], hi, lo);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pf[e >> 3][(e & 7) + j] = hi[j];
                    pl[e >> 3][(e & 7) + j] = lo[j];
                }
            }
            const float back = __builtin_amdgcn_exp2f(om - m - (ve[u] + kPrefillUnit)) * __builtin_amdgcn_rcpf(vm[u]);
            sum = __builtin_fmaf(part, back, sum);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    const half8_t v = vs[(4 * u + 2 * half + k) * D + 32 * t + col];
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
    const float true_unit = __builtin_amdgcn_exp2f(om - m - kPrefillUnit);
    float* so = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4_t v = {acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
            *reinterpret_cast<float4_t*>(so + wrow * SO + 32 * t + 8 * q + 4 * half) = v * true_unit;
        }
    if (half == 0) {
        sm[wrow] = m;
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

template <int D, int FORMAT, int NP>
void launch_np(const KvAttentionArgs& a, const Plan& p, const Split& sp, hipStream_t stream) {
    if (p.decode)
        hipLaunchKernelGGL((kv_decode_kernel<D, FORMAT, NP>),
                           dim3(static_cast<unsigned>(p.splits), static_cast<unsigned>(p.row_tiles * a.c.heads),
                                static_cast<unsigned>(a.n_seqs)),
                           dim3(kDecodeWaves * kWave), 0, stream, a, sp, p.splits);
    else
        hipLaunchKernelGGL((kv_prefill_kernel<D, FORMAT, NP>),
                           dim3(static_cast<unsigned>(p.row_tiles * p.splits * a.c.heads), 1,
                                static_cast<unsigned>(a.n_seqs)),
                           dim3(kPrefillWaves * kWave), 0, stream, a, sp, p.splits);
}
template <int D>
void launch_d(const KvAttentionArgs& a, const Plan& p, const Split& sp, hipStream_t stream) {
    const bool two = a.c.log2_page == 5;
    if (a.format == AWQ_KV_INT8) {
        if (two) launch_np<D, AWQ_KV_INT8, 2>(a, p, sp, stream);
        else launch_np<D, AWQ_KV_INT8, 1>(a, p, sp, stream);
    } else {
        if (two) launch_np<D, AWQ_KV_E4M3, 2>(a, p, sp, stream);
        else launch_np<D, AWQ_KV_E4M3, 1>(a, p, sp, stream);
    }
}

}  // namespace

size_t kv_attention_workspace_bytes(int format, int n_seqs, int kv_heads, int ratio, int head_dim, int64_t max_tokens,
                                    int64_t max_len) {
    const Plan p = plan_for(format, head_dim, n_seqs, kv_heads, ratio, max_tokens, max_len, true);
    return launchable(p, kv_heads) ? plan_bytes(p, n_seqs, kv_heads, head_dim) : 0;
}

awq_status launch_kv_attention(const KvAttentionArgs& a, void* workspace, hipStream_t stream) {
    if (a.format == AWQ_KV_INT4) return launch_kv4_attention(a, workspace, stream);
    const Plan p = plan_for(a.format, a.head_dim, a.n_seqs, a.c.heads, a.ratio, a.max_tokens, a.c.max_len, workspace != nullptr);
    if (!launchable(p, a.c.heads)) return AWQ_ERR_SHAPE;
    const Split sp = split_of(p, workspace);
    switch (a.head_dim) {
        case 64: launch_d<64>(a, p, sp, stream); break;
        case 96: launch_d<96>(a, p, sp, stream); break;
        case 128: launch_d<128>(a, p, sp, stream); break;
        case 192: launch_d<192>(a, p, sp, stream); break;
        case 256: launch_d<256>(a, p, sp, stream); break;
        default: return AWQ_ERR_CONFIG;
    }
    return last_launch_status();
}

}  // namespace awq
