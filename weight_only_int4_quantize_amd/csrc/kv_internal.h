// The paged 8-bit key / value cache: what its kernels share.
#pragma once

#include "awq_internal.h"

namespace awq {

typedef uint32_t kv_u32x4 __attribute__((ext_vector_type(4)));

// A cache and a batch as the kernels take them (see include/awq.h).
struct KvPages {
    uint8_t* k_codes;
    uint8_t* v_codes;
    float* k_scales;
    float* v_scales;
    const int32_t* table;
    const int32_t* cu;
    const int32_t* len;
    int64_t table_stride;
    int max_pages;
    int n_pages;
    int heads;          // of keys and values
    int log2_page;
    int n_tokens;       // rows of the token tensors
    int max_len;
};

// Longest sequence: whole splits of 1024 positions, and a tile past them, in
// 32 bits, so that one split can hold every position.
constexpr int64_t kKvMaxLen = (int64_t{1} << 31) - 1024;

constexpr float kInt8Top = 127.0f;
constexpr float kE4m3Top = 448.0f;
constexpr float kHalfMax = 65504.0f;

// One sequence of the batch: its rows in the token tensors (row0 and the
// n - 1 behind it), its tokens, the position of row row0. Whatever the arrays
// hold, rows stay in [0, n_tokens) and positions below max_pages pages, so no
// access leaves a tensor. Positions count from the sequence's last new token,
// whether the tensors have its row or not.
struct KvSeq {
    int row0, n, len, start;
    __device__ int end() const { return start + n; }    // position behind the last row's
};
__device__ inline KvSeq kv_seq(const KvPages& c, int b) {
    KvSeq s;
    s.row0 = min(max(c.cu[b], 0), c.n_tokens);
    const int rows_end = max(c.cu[b + 1], s.row0);
    s.n = min(rows_end, c.n_tokens) - s.row0;
    const int64_t held = static_cast<int64_t>(c.max_pages) << c.log2_page;
    s.len = min(max(c.len[b], 0), static_cast<int>(held < c.max_len ? held : c.max_len));
    s.start = s.len - (rows_end - s.row0);
    return s;
}

// A load that the whole wave shares, through the scalar cache: it neither
// waits for the vector loads in flight nor makes them wait. Only for tensors
// no kernel of this launch writes.
template <typename T>
__device__ inline T kv_shared_load(const T* p) {
#if defined(__HIP_DEVICE_COMPILE__)
    return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
#else
    return *p;
#endif
}

// Page number p of sequence b, or -1 when the cache does not hold it.
__device__ inline int kv_page(const KvPages& c, int b, int p) {
    const int id = c.table[static_cast<int64_t>(b) * c.table_stride + p];
    return id >= 0 && id < c.n_pages ? id : -1;
}

// kv_seq and kv_page for wave-uniform arguments (attention only: the write
// changes what it would read)
__device__ inline KvSeq kv_seq_shared(const KvPages& c, int b) {
    KvSeq s;
    s.row0 = min(max(kv_shared_load(c.cu + b), 0), c.n_tokens);
    const int rows_end = max(kv_shared_load(c.cu + b + 1), s.row0);
    s.n = min(rows_end, c.n_tokens) - s.row0;
    const int64_t held = static_cast<int64_t>(c.max_pages) << c.log2_page;
    s.len = min(max(kv_shared_load(c.len + b), 0), static_cast<int>(held < c.max_len ? held : c.max_len));
    s.start = s.len - (rows_end - s.row0);
    return s;
}
__device__ inline int kv_page_shared(const KvPages& c, int b, int p) {
    const int id = kv_shared_load(c.table + static_cast<int64_t>(b) * c.table_stride + p);
    return id >= 0 && id < c.n_pages ? id : -1;
}

// Four stored bytes -> their exact fp16 numbers, in order.
template <int FORMAT>
__device__ inline void kv_unpack4(uint32_t w, half2_t& lo, half2_t& hi) {
    if constexpr (FORMAT == AWQ_KV_INT8) {
        // a byte in the mantissa of 1024.0 is 1024 + byte; the code is byte - 128
        const half_t off = static_cast<half_t>(1152.0f);
        lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - half2_t{off, off};
        hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - half2_t{off, off};
    } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
    }
}
template <int FORMAT>
__device__ inline half8_t kv_unpack8(uint32_t w0, uint32_t w1) {
    half2_t a, b, c, d;
    kv_unpack4<FORMAT>(w0, a, b);
    kv_unpack4<FORMAT>(w1, c, d);
    return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Four scaled numbers (|v| up to the format's top) -> stored bytes.
template <int FORMAT>
__device__ inline uint32_t kv_pack4(float a, float b, float c, float d) {
    if constexpr (FORMAT == AWQ_KV_INT8) {
        auto byte = [](float v) {
            const float q = fminf(fmaxf(__builtin_rintf(v), -kInt8Top), kInt8Top);
            return static_cast<uint32_t>(static_cast<int>(q) + 128);
        };
        return byte(a) | (byte(b) << 8) | (byte(c) << 16) | (byte(d) << 24);
    } else {
        const auto top = [](float v) { return fminf(fmaxf(v, -kE4m3Top), kE4m3Top); };
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(top(a), top(b), 0, false);
        return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(top(c), top(d), w, true));
    }
}

// ---- launchers ----
struct KvWriteArgs {
    KvPages c;
    const half_t* k;
    const half_t* v;
    int64_t k_token, k_head, v_token, v_head;
    int head_dim, n_seqs, format;
    int64_t max_tokens;
};
awq_status launch_kv_write(const KvWriteArgs& a, hipStream_t stream);
struct KvReadArgs {
    KvPages c;
    half_t* k;
    half_t* v;
    int head_dim, n_seqs, format;
    int64_t max_tokens;
};
awq_status launch_kv_read(const KvReadArgs& a, hipStream_t stream);

struct KvAttentionArgs {
    KvPages c;
    const half_t* q;
    half_t* out;
    float* lse;
    int64_t q_token, q_head, out_token, out_head;
    int head_dim, n_seqs, format, ratio;   // ratio: query heads per kv head
    int64_t max_tokens;
    float scale_log2;                      // scale * log2(e)
    bool causal;
    int window;                            // 0: none
};
size_t kv_attention_workspace_bytes(int n_seqs, int kv_heads, int ratio, int head_dim, int64_t max_tokens,
                                    int64_t max_len);
awq_status launch_kv_attention(const KvAttentionArgs& a, void* workspace, hipStream_t stream);

}  // namespace awq
