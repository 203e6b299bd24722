// C ABI of the library (declared in include/awq.h): argument checks on the
// host, then kernels enqueued on the caller's stream.
#include <algorithm>
#include <cmath>
#include <limits>
#include <mutex>
#include <vector>

#include "kv_internal.h"

using namespace awq;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;      // any single extent
constexpr int64_t kMaxElems = int64_t(1) << 40;    // any product of extents

bool valid_group(int g) { return g == 32 || g == 64 || g == 128 || g == 256 || g == 512; }

awq_status check_dims(int64_t N, int64_t K, int group_size) {
    if (!valid_group(group_size)) return AWQ_ERR_CONFIG;
    if (N < 0 || K <= 0 || N > kMaxDim || K > kMaxDim) return AWQ_ERR_SHAPE;
    if (K % group_size != 0) return AWQ_ERR_SHAPE;
    return AWQ_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

struct Carve {
    char* base;
    size_t used = 0;
    explicit Carve(void* p) : base(static_cast<char*>(p)) {}
    template <class T>
    T* take(size_t count) {
        T* p = reinterpret_cast<T*>(base ? base + used : nullptr);
        used = round_up(used + count * sizeof(T), 256);
        return p;
    }
};

// Halves of the reference's tiled copy of W: whole 64-k steps take it, other
// K none (the reference then reads W in place).
size_t reference_tiled_halves(int64_t N, int64_t K) { return gemm_ref_tiled_ok(K) ? tiled_fp16_halves(N, K) : 0; }

// Lays out the scale-search workspace; with base == nullptr it only sizes it.
struct SearchLayout {
    double* m = nullptr;
    double* abs_partials = nullptr;
    float* s = nullptr;
    uint32_t* qweight = nullptr;
    half_t* scales = nullptr;
    half_t* zeros = nullptr;
    half_t* xs = nullptr;
    half_t* wt = nullptr;   // W in the reference's tiled order (whole 64-k steps only)
    float* yref = nullptr;
    double* tile_partials = nullptr;
    double* losses = nullptr;
    size_t bytes = 0;

    SearchLayout(void* base, int64_t N, int64_t K, int64_t T, int G, int n_alpha) {
        Carve c(base);
        m = c.take<double>(K);
        abs_partials = c.take<double>(absmean_workspace_bytes(T, K) / sizeof(double));
        s = c.take<float>(K);
        qweight = c.take<uint32_t>(tiled_qweight_words(N, K));   // tiled order or row-major
        scales = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        zeros = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        xs = c.take<half_t>(static_cast<size_t>(T) * K);
        wt = c.take<half_t>(reference_tiled_halves(N, K));
        yref = c.take<float>(static_cast<size_t>(ref_tiled_floats(T, N)));
        tile_partials = c.take<double>(gemm_tile_count(T, N) + kLossSumBlocks);
        losses = c.take<double>(n_alpha);
        bytes = c.used;
    }
};

// Lays out the salient-loss workspace; with base == nullptr it only sizes it.
struct SalientLayout {
    double* m = nullptr;
    double* abs_partials = nullptr;
    int* idx = nullptr;
    uint32_t* qweight = nullptr;
    half_t* scales = nullptr;
    half_t* zeros = nullptr;
    half_t* w_sal = nullptr;
    half_t* wt = nullptr;   // W in the reference's tiled order (whole 64-k steps only)
    float* yref = nullptr;
    double* tile_partials = nullptr;
    double* losses = nullptr;
    size_t bytes = 0;

    SalientLayout(void* base, int64_t N, int64_t K, int64_t T, int G, int n_sal) {
        Carve c(base);
        m = c.take<double>(K);
        abs_partials = c.take<double>(absmean_workspace_bytes(T, K) / sizeof(double));
        idx = c.take<int>(std::max(n_sal, 1));
        qweight = c.take<uint32_t>(static_cast<size_t>(N) * (K / 8));
        scales = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        zeros = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        w_sal = c.take<half_t>(static_cast<size_t>(std::max(n_sal, 1)) * N);
        wt = c.take<half_t>(reference_tiled_halves(N, K));
        yref = c.take<float>(static_cast<size_t>(ref_tiled_floats(T, N)));
        tile_partials = c.take<double>(gemm_tile_count(T, N) + kLossSumBlocks);
        losses = c.take<double>(2);
        bytes = c.used;
    }
};

// Channels the K^2 selection accepts (a few milliseconds at the largest).
constexpr int64_t kMaxSelectK = int64_t(1) << 17;

// Lays out the clip-search workspace; with base == nullptr it only sizes it.
struct ClipLayout {
    uint32_t* qweight = nullptr;
    half_t* scales = nullptr;
    half_t* zeros = nullptr;
    half_t* xs = nullptr;           // x / s, only with channel scales
    half_t* wt = nullptr;           // W in the reference's tiled order (whole 64-k steps only)
    float* yref = nullptr;
    double* tile_partials = nullptr;
    double* losses = nullptr;
    size_t bytes = 0;

    ClipLayout(void* base, int64_t N, int64_t K, int64_t T, int G, int n, bool scaled) {
        Carve c(base);
        qweight = c.take<uint32_t>(tiled_qweight_words(N, K));   // tiled order or row-major
        scales = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        zeros = c.take<half_t>(static_cast<size_t>(N) * (K / G));
        if (scaled) xs = c.take<half_t>(static_cast<size_t>(T) * K);
        wt = c.take<half_t>(reference_tiled_halves(N, K));
        yref = c.take<float>(static_cast<size_t>(ref_tiled_floats(T, N)));
        tile_partials = c.take<double>(gemm_tile_count(T, N) + kLossSumBlocks);
        losses = c.take<double>(n);
        bytes = c.used;
    }
};

// Y = x . W^T in fp32 (fp16 MFMA, fp32 accumulation), the unquantized
// reference of the searches, written in the tiled layout of ref_offset. With
// K whole 64-k steps W is first copied into wt in the GEMM's tiled B order
// (each wave's B of a step one contiguous piece); the products are the same.
awq_status reference_output(const half_t* x, const half_t* w, int64_t T, int64_t N, int64_t K, int G, float* y,
                            half_t* wt, hipStream_t s) {
    GemmArgs ref;
    ref.a = x;
    ref.w = w;
    ref.group_size = G;
    ref.M = T;
    ref.N = N;
    ref.K = K;
    ref.y32 = y;
    if (reference_tiled_halves(N, K) != 0 && T != 0 && N != 0) {
        const awq_status st = launch_tile_fp16_b(w, N, K, wt, s);
        if (st != AWQ_OK) return st;
        ref.w = wt;
        ref.b_tiled = true;
    }
    return launch_gemm(ref, GemmB::kF16, GemmOut::kF32, s);
}

// loss_out = || x' . dequant(Wq)^T - yref ||_F^2 (fused epilogue + fixed-order sum)
// tiled: qw holds the words in the tiled order (GemmArgs::b_tiled)
awq_status output_loss(const half_t* xa, const uint32_t* qw, const half_t* sc, const half_t* zr, int64_t T,
                       int64_t N, int64_t K, int G, const float* yref, double* partials, double* loss_out,
                       hipStream_t s, bool tiled = false) {
    GemmArgs q;
    q.a = xa;
    q.qweight = qw;
    q.scales = sc;
    q.zeros = zr;
    q.group_size = G;
    q.M = T;
    q.N = N;
    q.K = K;
    q.yref = yref;
    q.partials = partials;
    q.b_tiled = tiled;
    awq_status st = launch_gemm(q, GemmB::kInt4, GemmOut::kLoss, s);
    if (st != AWQ_OK) return st;
    return launch_sum_partials(partials, gemm_tile_count(T, N), loss_out, s);
}

// ---- the library-held scratch of awq_gemm_noalloc ----
// Callers that cannot allocate device memory (code under HIP graph capture,
// tight serving loops) get the skinny kernel's K-split partial tiles and
// tile counters from this array instead of a workspace. 49 MiB holds the
// split plan of every M <= 64 on a 256-CU device (4 KiB of counters + 768
// partial tiles of up to 64 KiB). Each device the library runs on holds its
// own copy until the process ends.
constexpr size_t kNoAllocScratchBytes = size_t(49) << 20;
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

__global__ void zero_words_kernel(uint32_t* p, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0u;
}

constexpr int kMaxDevices = 64;
struct ScratchSlot {
    std::once_flag once;
    void* ptr = nullptr;         // the device address of `scratch` on this device
    awq_status status = AWQ_OK;
};
ScratchSlot g_scratch[kMaxDevices];

// The current device's copy of `scratch` (its device address, taken once per
// device with that device current). The first call on a device also clears
// the tile counters (a fill kernel on `stream`, ahead of the call's own
// work); every split kernel leaves them at zero when it ends.
awq_status device_scratch(void** out, hipStream_t stream) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_HIP;
    ScratchSlot& slot = g_scratch[dev];
    std::call_once(slot.once, [&] {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) {
            slot.status = AWQ_ERR_HIP;
            return;
        }
        const int64_t words = static_cast<int64_t>(split_counter_bytes() / sizeof(uint32_t));
        hipLaunchKernelGGL(zero_words_kernel, dim3(static_cast<unsigned>(ceil_div(words, 256))), dim3(256), 0, stream,
                           static_cast<uint32_t*>(p), words);
        slot.status = last_launch_status();
        if (slot.status == AWQ_OK) slot.ptr = p;
    });
    if (slot.status != AWQ_OK) return slot.status;
    *out = slot.ptr;
    return AWQ_OK;
}

// The kernel a linear-layer call runs (1 GEMV, 2 GEMM, 3 skinny, 4 column
// tiles), or -1 when the requested path cannot take the shape. Automatic
// (path 0): the column tiles where they measured fastest; otherwise the GEMV
// up to 4 rows; the skinny kernel up to 64 rows (and below 5 rows where the
// GEMV's staged x does not fit the LDS), but below 9 rows only where it runs
// without K phases if the GEMV can run (the phased form, one block per
// column tile, is 2-3x slower than the GEMV there and 2-3x faster than the
// GEMM tile everywhere); else the GEMM.
int choose_path(int64_t M, int64_t N, int64_t K, int group_size, int path, bool have_workspace) {
    const bool gemv_ok = gemv_supported(M, N, K);
    bool skinny_phased = false;
    const bool skinny_ok = skinny_supported(M, N, K, group_size, have_workspace, &skinny_phased);
    switch (path) {
        case 1: return gemv_ok ? 1 : -1;
        case 2: return 2;
        case 3: return skinny_ok ? 3 : -1;
        case 4: return coltile_supported(M, N, K, group_size) ? 4 : -1;
        default: break;
    }
    // few-row layers with long rows: the GEMV's one-shot form beats the
    // column tiles up to 4 rows of x (512 x 11008 at M = 4: 7.9 against
    // 8.7 us; 1024 x 8192: 5.7 against 7.2 us)
    if (M >= 3 && gemv_ok && gemv_few_rows(M, N, K)) return 1;
    if (coltile_preferred(M, N, K, group_size, have_workspace)) return 4;
    if (skinny_ok && (M > 4 || !gemv_ok) && !(skinny_phased && gemv_ok)) return 3;
    return gemv_ok ? 1 : 2;
}

// The same behind an epilogue, whose GEMM has a tile for a few hundred rows
// that also beats the skinny kernel above 32 of them.
int choose_fused(int64_t M, int64_t N, int64_t K, int group_size, int path, bool have_workspace) {
    const int chosen = choose_path(M, N, K, group_size, path, have_workspace);
    if (path == 0 && chosen == 3 && M > kColTileMaxM && gemm_fused_mid(M, N, K, group_size, have_workspace)) return 2;
    return chosen;
}

// The W8 layer's kernel (1 GEMV, 2 GEMM), or -1. The MFMA form needs 32-bit
// byte offsets within a 256-row tile of x.
int choose_w8(int64_t M, int64_t N, int64_t K, int path) {
    const bool gemv_ok = gemv_supported(M, N, K, 8);
    if (path == 1) return gemv_ok ? 1 : -1;
    if (path == 0 && gemv_ok) return 1;
    return K * 256 * 2 < (int64_t(1) << 31) ? 2 : -1;
}

// The linear layer behind awq_gemm_ex and awq_gemm_noalloc: checks, then
// the kernel choice. workspace (may be NULL) feeds the skinny kernel's K
// splits and, when split_gemm is set, the GEMM's stream-K partials. With
// library_scratch the skinny kernel's splits take the device's `scratch`
// instead (set up only once every check has passed); the GEMM then runs
// unsplit.
awq_status gemm_dispatch(const void* x_f16, const uint32_t* qweight, const void* scales_f16, const void* zeros_f16,
                         int64_t M, int64_t N, int64_t K, int group_size, void* y_f16, int path, void* workspace,
                         size_t workspace_bytes, bool split_gemm, bool library_scratch, hipStream_t stream,
                         const Epilogue* epilogue = nullptr) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (path < 0 || path > 4) return AWQ_ERR_CONFIG;
    if (M < 0 || M > kMaxDim) return AWQ_ERR_SHAPE;
    // The MFMA kernel indexes with 32-bit row/column numbers and 64-bit offsets.
    if (M > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if (!x_f16 || !qweight || !scales_f16 || !zeros_f16 || !y_f16) return AWQ_ERR_NULL;
    if (!aligned16(x_f16) || !aligned16(qweight) || (reinterpret_cast<uintptr_t>(scales_f16) & 1) ||
        (reinterpret_cast<uintptr_t>(zeros_f16) & 1) || (reinterpret_cast<uintptr_t>(y_f16) & 1))
        return AWQ_ERR_ALIGN;
    const half_t* x = static_cast<const half_t*>(x_f16);
    const half_t* sc = static_cast<const half_t*>(scales_f16);
    const half_t* zr = static_cast<const half_t*>(zeros_f16);
    half_t* y = static_cast<half_t*>(y_f16);
    const int chosen = epilogue ? choose_fused(M, N, K, group_size, path, workspace != nullptr)
                                : choose_path(M, N, K, group_size, path, workspace != nullptr || library_scratch);
    if (chosen < 0) return AWQ_ERR_CONFIG;
    const bool use_skinny = chosen == 3;
    if (chosen == 4) return launch_coltile(x, qweight, sc, zr, M, N, K, group_size, y, stream, epilogue);
    if (chosen == 1) return launch_gemv(x, qweight, sc, zr, M, N, K, group_size, y, stream, 4, epilogue);
    if (!use_skinny && !split_gemm) workspace = nullptr;
    if (use_skinny && library_scratch) {
        if (skinny_workspace_bytes(M, N, K) > kNoAllocScratchBytes) return AWQ_ERR_WORKSPACE;
        if ((st = device_scratch(&workspace, stream)) != AWQ_OK) return st;
        workspace_bytes = kNoAllocScratchBytes;
    }
    if (workspace != nullptr) {
        if (reinterpret_cast<uintptr_t>(workspace) & 255) return AWQ_ERR_ALIGN;
        const size_t need = use_skinny ? skinny_workspace_bytes(M, N, K) : gemm_workspace_bytes(M, N);
        if (workspace_bytes < need) return AWQ_ERR_WORKSPACE;
    }
    if (use_skinny) return launch_skinny(x, qweight, sc, zr, M, N, K, group_size, y, workspace, stream, epilogue);
    GemmFusedArgs a;
    a.a = x;
    a.qweight = qweight;
    a.scales = sc;
    a.zeros = zr;
    a.group_size = group_size;
    a.M = M;
    a.N = N;
    a.K = K;
    a.y16 = y;
    if (epilogue) {
        a.epilogue = *epilogue;
        return launch_gemm_fused(a, GemmB::kInt4, stream, workspace);
    }
    return launch_gemm(a, GemmB::kInt4, GemmOut::kF16, stream, workspace);
}

// The W8 linear layer behind awq_gemm_w8 and awq_gemm_fused.
awq_status w8_dispatch(const void* x_f16, const uint32_t* qweight, const void* scales_f16, const void* zeros_f16,
                       int64_t M, int64_t N, int64_t K, int group_size, void* y_f16, int path, void* workspace,
                       size_t workspace_bytes, hipStream_t stream, const Epilogue* epilogue) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (group_size < 64) return AWQ_ERR_CONFIG;
    if (path < 0 || path > 2) return AWQ_ERR_CONFIG;
    if (M < 0 || M > kMaxDim) return AWQ_ERR_SHAPE;
    if (M > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0) return AWQ_OK;
    if (!x_f16 || !qweight || !scales_f16 || !zeros_f16 || !y_f16) return AWQ_ERR_NULL;
    if (!aligned16(x_f16) || !aligned16(qweight) || (reinterpret_cast<uintptr_t>(scales_f16) & 1) ||
        (reinterpret_cast<uintptr_t>(zeros_f16) & 1) || (reinterpret_cast<uintptr_t>(y_f16) & 1))
        return AWQ_ERR_ALIGN;
    const half_t* x = static_cast<const half_t*>(x_f16);
    const half_t* sc = static_cast<const half_t*>(scales_f16);
    const half_t* zr = static_cast<const half_t*>(zeros_f16);
    half_t* y = static_cast<half_t*>(y_f16);
    const int chosen = choose_w8(M, N, K, path);
    if (chosen < 0) return path == 0 ? AWQ_ERR_SHAPE : AWQ_ERR_CONFIG;
    if (chosen == 1) return launch_gemv(x, qweight, sc, zr, M, N, K, group_size, y, stream, 8, epilogue);
    if (workspace != nullptr) {
        if (reinterpret_cast<uintptr_t>(workspace) & 255) return AWQ_ERR_ALIGN;
        if (workspace_bytes < gemm_workspace_bytes(M, N)) return AWQ_ERR_WORKSPACE;
    }
    GemmFusedArgs a;
    a.a = x;
    a.qweight = qweight;
    a.scales = sc;
    a.zeros = zr;
    a.group_size = group_size;
    a.M = M;
    a.N = N;
    a.K = K;
    a.y16 = y;
    if (epilogue) {
        a.epilogue = *epilogue;
        return launch_gemm_fused(a, GemmB::kInt8, stream, workspace);
    }
    return launch_gemm(a, GemmB::kInt8, GemmOut::kF16, stream, workspace);
}

}  // namespace

extern "C" {

const char* awq_status_string(int status) {
    switch (status) {
        case AWQ_OK: return "AWQ_OK";
        case AWQ_ERR_NULL: return "AWQ_ERR_NULL: a required pointer is NULL";
        case AWQ_ERR_SHAPE: return "AWQ_ERR_SHAPE: invalid matrix sizes";
        case AWQ_ERR_ALIGN: return "AWQ_ERR_ALIGN: a device pointer is not 16-byte aligned";
        case AWQ_ERR_CONFIG: return "AWQ_ERR_CONFIG: unsupported configuration";
        case AWQ_ERR_WORKSPACE: return "AWQ_ERR_WORKSPACE: workspace too small";
        case AWQ_ERR_HIP: return "AWQ_ERR_HIP: HIP runtime error";
        default: return "unknown awq_status";
    }
}

int awq_version(void) { return 100; }

awq_status awq_quantize_ex(const void* w_f16, const float* channel_scale, int64_t N, int64_t K,
                           int group_size, int mode, double clip_fraction, uint32_t* qweight, void* scales_f16,
                           void* zeros_f16, void* stream) {
    if (mode != AWQ_QUANT_ASYMMETRIC && mode != AWQ_QUANT_SYMMETRIC) return AWQ_ERR_CONFIG;
    if (!clip_fraction_ok(clip_fraction)) return AWQ_ERR_CONFIG;
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (N * K > kMaxElems) return AWQ_ERR_SHAPE;
    if (N == 0) return AWQ_OK;
    if (!w_f16 || !qweight || !scales_f16 || !zeros_f16) return AWQ_ERR_NULL;
    if (!aligned16(w_f16) || !aligned16(qweight) || (channel_scale && !aligned16(channel_scale)))
        return AWQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(scales_f16) & 1) || (reinterpret_cast<uintptr_t>(zeros_f16) & 1))
        return AWQ_ERR_ALIGN;
    return launch_quantize(static_cast<const half_t*>(w_f16), channel_scale, N, K, group_size,
                           mode == AWQ_QUANT_SYMMETRIC, clip_fraction, qweight, static_cast<half_t*>(scales_f16),
                           static_cast<half_t*>(zeros_f16), as_stream(stream));
}

awq_status awq_quantize(const void* w_f16, const float* channel_scale, int64_t N, int64_t K,
                        int group_size, uint32_t* qweight, void* scales_f16, void* zeros_f16,
                        void* stream) {
    return awq_quantize_ex(w_f16, channel_scale, N, K, group_size, AWQ_QUANT_ASYMMETRIC, 0.0, qweight,
                           scales_f16, zeros_f16, stream);
}

size_t awq_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    return std::max(gemm_workspace_bytes(M, N), skinny_workspace_bytes(M, N, K));
}

awq_status awq_gemm_ex(const void* x_f16, const uint32_t* qweight, const void* scales_f16,
                       const void* zeros_f16, int64_t M, int64_t N, int64_t K, int group_size,
                       void* y_f16, int path, void* workspace, size_t workspace_bytes, void* stream) {
    return gemm_dispatch(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, workspace,
                         workspace_bytes, true, false, as_stream(stream));
}

awq_status awq_gemm_path(const void* x_f16, const uint32_t* qweight, const void* scales_f16,
                         const void* zeros_f16, int64_t M, int64_t N, int64_t K, int group_size,
                         void* y_f16, int path, void* stream) {
    return awq_gemm_ex(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, nullptr, 0,
                       stream);
}

int awq_gemm_kernel(int64_t M, int64_t N, int64_t K, int group_size, int path, int have_workspace) {
    if (check_dims(N, K, group_size) != AWQ_OK || path < 0 || path > 4) return -1;
    if (M < 1 || N < 1 || M > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return -1;
    return choose_path(M, N, K, group_size, path, have_workspace != 0);
}

int awq_gemm_fused_kernel(int64_t M, int64_t N, int64_t K, int group_size, int bits, int path, int have_workspace) {
    if (check_dims(N, K, group_size) != AWQ_OK || (bits != 4 && bits != 8) || path < 0 || path > (bits == 4 ? 4 : 2))
        return -1;
    if (M < 1 || N < 1 || M > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return -1;
    if (bits == 8 && group_size < 64) return -1;
    const int chosen = bits == 4 ? choose_fused(M, N, K, group_size, path, have_workspace != 0)
                                 : choose_w8(M, N, K, path);
    return chosen == 2 && gemm_fused_mid(M, N, K, group_size, have_workspace != 0) ? 5 : chosen;
}

awq_status awq_gemm_grouped(const void* x_f16, int n_layers, const uint32_t* const* qweight,
                            const void* const* scales_f16, const void* const* zeros_f16, const int64_t* N,
                            int64_t M, int64_t K, int group_size, void* const* y_f16, void* stream) {
    if (n_layers < 1 || n_layers > kGemvMaxLayers) return AWQ_ERR_CONFIG;
    if (!qweight || !scales_f16 || !zeros_f16 || !N || !y_f16) return AWQ_ERR_NULL;
    if (M < 0 || M > kMaxDim) return AWQ_ERR_SHAPE;
    int64_t total = 0;
    for (int i = 0; i < n_layers; ++i) {
        const awq_status st = check_dims(N[i], K, group_size);
        if (st != AWQ_OK) return st;
        total += N[i];
        if (M > 0 && N[i] > 0) {
            if (!x_f16 || !qweight[i] || !scales_f16[i] || !zeros_f16[i] || !y_f16[i]) return AWQ_ERR_NULL;
            if (!aligned16(x_f16) || !aligned16(qweight[i]) || (reinterpret_cast<uintptr_t>(scales_f16[i]) & 1) ||
                (reinterpret_cast<uintptr_t>(zeros_f16[i]) & 1) || (reinterpret_cast<uintptr_t>(y_f16[i]) & 1))
                return AWQ_ERR_ALIGN;
        }
    }
    if (total > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (M == 0 || total == 0) return AWQ_OK;
    const hipStream_t s = as_stream(stream);
    const int chosen = choose_path(M, total, K, group_size, 0, false);
    GemvLayers L{};
    int r = 0;
    for (int i = 0; i < n_layers; ++i) {
        if (N[i] == 0) continue;
        L.qweight[L.n] = qweight[i];
        L.scales[L.n] = static_cast<const half_t*>(scales_f16[i]);
        L.zeros[L.n] = static_cast<const half_t*>(zeros_f16[i]);
        L.y[L.n] = static_cast<half_t*>(y_f16[i]);
        L.row0[L.n] = r;
        r += static_cast<int>(N[i]);
        ++L.n;
    }
    L.row0[L.n] = r;
    for (int i = L.n + 1; i <= kGemvMaxLayers; ++i) L.row0[i] = INT32_MAX;
    const half_t* x = static_cast<const half_t*>(x_f16);
    if (chosen == 1 && M <= kGemvGroupedMaxM) return launch_gemv_grouped(x, L, M, K, group_size, s);
    // column tiles over the stacked layers where awq_gemm takes them, and at
    // 3-4 rows of x on few-row layers (which awq_gemm gives the GEMV one at a
    // time); the layers' own block counts must fit the launch
    if ((chosen == 4 || (chosen == 1 && M > kGemvGroupedMaxM)) && coltile_grouped_supported(M, L, K, group_size))
        return launch_coltile_grouped(x, L, M, K, group_size, s);
    for (int i = 0; i < n_layers; ++i) {
        const awq_status st = gemm_dispatch(x_f16, qweight[i], scales_f16[i], zeros_f16[i], M, N[i], K, group_size,
                                            y_f16[i], 0, nullptr, 0, false, false, s);
        if (st != AWQ_OK) return st;
    }
    return AWQ_OK;
}

awq_status awq_gemm_noalloc(const void* x_f16, const uint32_t* qweight, const void* scales_f16,
                            const void* zeros_f16, int64_t M, int64_t N, int64_t K, int group_size, void* y_f16,
                            int path, void* stream) {
    return gemm_dispatch(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, nullptr, 0,
                         false, true, as_stream(stream));
}

awq_status awq_gemm(const void* x_f16, const uint32_t* qweight, const void* scales_f16,
                    const void* zeros_f16, int64_t M, int64_t N, int64_t K, int group_size,
                    void* y_f16, void* stream) {
    return awq_gemm_path(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, 0, stream);
}

size_t awq_activation_absmean_workspace_bytes(int64_t T, int64_t K) {
    if (T <= 0 || K <= 0) return 0;
    return absmean_workspace_bytes(T, K);
}

awq_status awq_activation_absmean(const void* x_f16, int64_t T, int64_t K, double* m_f64,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (T <= 0 || K <= 0 || K % 8 != 0 || K > kMaxDim || T > (int64_t(1) << 24)) return AWQ_ERR_SHAPE;
    if (!x_f16 || !m_f64 || !workspace) return AWQ_ERR_NULL;
    if (!aligned16(x_f16) || (reinterpret_cast<uintptr_t>(m_f64) & 7) ||
        (reinterpret_cast<uintptr_t>(workspace) & 7))
        return AWQ_ERR_ALIGN;
    if (workspace_bytes < absmean_workspace_bytes(T, K)) return AWQ_ERR_WORKSPACE;
    return launch_absmean(static_cast<const half_t*>(x_f16), T, K, m_f64, static_cast<double*>(workspace),
                          as_stream(stream));
}

size_t awq_scale_search_workspace_bytes(int64_t N, int64_t K, int64_t T, int group_size, int n_alpha) {
    if (check_dims(N, K, group_size) != AWQ_OK || N <= 0 || T <= 0 || n_alpha < 1) return 0;
    return SearchLayout(nullptr, N, K, T, group_size, n_alpha).bytes;
}

awq_status awq_scale_search(const void* w_f16, const void* x_f16, int64_t N, int64_t K, int64_t T,
                            int group_size, const double* alphas, int n_alpha, void* workspace,
                            size_t workspace_bytes, double* losses, int* best_index, float* best_scales,
                            void* stream) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (N <= 0 || T <= 0 || T > (int64_t(1) << 24)) return AWQ_ERR_SHAPE;
    if (T > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (n_alpha < 1 || n_alpha > 64) return AWQ_ERR_CONFIG;
    if (!w_f16 || !x_f16 || !workspace || !losses || !best_index || !best_scales) return AWQ_ERR_NULL;
    // no grid given: alpha_i = i / n_alpha (n_alpha = 20: 0, 0.05, ..., 0.95)
    std::vector<double> grid(n_alpha);
    for (int i = 0; i < n_alpha; ++i) {
        grid[i] = alphas ? alphas[i] : static_cast<double>(i) / static_cast<double>(n_alpha);
        if (!std::isfinite(grid[i])) return AWQ_ERR_CONFIG;
    }
    if (!aligned16(w_f16) || !aligned16(x_f16) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(best_scales) & 3))
        return AWQ_ERR_ALIGN;
    SearchLayout L(workspace, N, K, T, group_size, n_alpha);
    if (workspace_bytes < L.bytes) return AWQ_ERR_WORKSPACE;
    hipStream_t s = as_stream(stream);
    const half_t* w = static_cast<const half_t*>(w_f16);
    const half_t* x = static_cast<const half_t*>(x_f16);

    // the loss GEMM reads the quantized words in the tiled order where its
    // direct form runs (one contiguous 1 KB piece per wave and K step)
    const bool tiled = gemm_tiled_ok(K, group_size);
    // m = mean |x| per input channel
    if ((st = launch_absmean(x, T, K, L.m, L.abs_partials, s)) != AWQ_OK) return st;
    // reference output W . x^T, once, in fp32
    if ((st = reference_output(x, w, T, N, K, group_size, L.yref, L.wt, s)) != AWQ_OK) return st;
    for (int i = 0; i < n_alpha; ++i) {
        if ((st = launch_pow_scales(L.m, K, grid[i], L.s, s)) != AWQ_OK) return st;
        if ((st = launch_quantize(w, L.s, N, K, group_size, false, 0.0, L.qweight, L.scales, L.zeros, s, 4,
                                  tiled)) != AWQ_OK)
            return st;
        // s = 1 exactly at alpha = 0, where x / s is x itself, bit for bit
        const bool identity = grid[i] == 0.0;
        if (!identity && (st = launch_divide_columns(x, L.s, T, K, L.xs, s)) != AWQ_OK) return st;
        if ((st = output_loss(identity ? x : L.xs, L.qweight, L.scales, L.zeros, T, N, K, group_size, L.yref,
                              L.tile_partials, L.losses + i, s, tiled)) != AWQ_OK)
            return st;
    }
    if (hipMemcpyAsync(losses, L.losses, sizeof(double) * n_alpha, hipMemcpyDeviceToHost, s) != hipSuccess)
        return AWQ_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return AWQ_ERR_HIP;
    int best = 0;
    for (int i = 1; i < n_alpha; ++i)
        if (losses[i] < losses[best]) best = i;   // strict: ties keep the smaller alpha
    *best_index = best;
    if ((st = launch_pow_scales(L.m, K, grid[best], best_scales, s)) != AWQ_OK) return st;
    return AWQ_OK;
}

size_t awq_clip_search_workspace_bytes(int64_t N, int64_t K, int64_t T, int group_size, int n_fractions,
                                        int scaled) {
    if (check_dims(N, K, group_size) != AWQ_OK || N <= 0 || T <= 0 || n_fractions < 1) return 0;
    return ClipLayout(nullptr, N, K, T, group_size, n_fractions, scaled != 0).bytes;
}

awq_status awq_clip_search(const void* w_f16, const void* x_f16, const float* channel_scale, int64_t N, int64_t K,
                           int64_t T, int group_size, int mode, const double* fractions, int n_fractions,
                           void* workspace, size_t workspace_bytes, double* losses, int* best_index,
                           void* stream) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (N <= 0 || T <= 0 || T > (int64_t(1) << 24)) return AWQ_ERR_SHAPE;
    if (T > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (mode != AWQ_QUANT_ASYMMETRIC && mode != AWQ_QUANT_SYMMETRIC) return AWQ_ERR_CONFIG;
    if (n_fractions < 1 || n_fractions > 64) return AWQ_ERR_CONFIG;
    if (!w_f16 || !x_f16 || !fractions || !workspace || !losses || !best_index) return AWQ_ERR_NULL;
    for (int i = 0; i < n_fractions; ++i)
        if (!clip_fraction_ok(fractions[i])) return AWQ_ERR_CONFIG;
    if (!aligned16(w_f16) || !aligned16(x_f16) || !aligned16(workspace) ||
        (channel_scale && !aligned16(channel_scale)))
        return AWQ_ERR_ALIGN;
    ClipLayout L(workspace, N, K, T, group_size, n_fractions, channel_scale != nullptr);
    if (workspace_bytes < L.bytes) return AWQ_ERR_WORKSPACE;
    hipStream_t s = as_stream(stream);
    const half_t* w = static_cast<const half_t*>(w_f16);
    const half_t* x = static_cast<const half_t*>(x_f16);

    if ((st = reference_output(x, w, T, N, K, group_size, L.yref, L.wt, s)) != AWQ_OK) return st;
    const half_t* xa = x;
    if (channel_scale != nullptr) {
        if ((st = launch_divide_columns(x, channel_scale, T, K, L.xs, s)) != AWQ_OK) return st;
        xa = L.xs;
    }
    const bool tiled = gemm_tiled_ok(K, group_size);   // as in the scale search
    for (int i = 0; i < n_fractions; ++i) {
        if ((st = launch_quantize(w, channel_scale, N, K, group_size, mode == AWQ_QUANT_SYMMETRIC, fractions[i],
                                  L.qweight, L.scales, L.zeros, s, 4, tiled)) != AWQ_OK)
            return st;
        if ((st = output_loss(xa, L.qweight, L.scales, L.zeros, T, N, K, group_size, L.yref, L.tile_partials,
                              L.losses + i, s, tiled)) != AWQ_OK)
            return st;
    }
    if (hipMemcpyAsync(losses, L.losses, sizeof(double) * n_fractions, hipMemcpyDeviceToHost, s) != hipSuccess)
        return AWQ_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return AWQ_ERR_HIP;
    int best = 0;
    for (int i = 1; i < n_fractions; ++i)
        if (losses[i] < losses[best]) best = i;   // strict: ties keep the earlier fraction
    *best_index = best;
    return AWQ_OK;
}

awq_status awq_select_salient(const double* m_f64, int64_t K, int n_salient, int* idx, void* stream) {
    if (K <= 0 || K > kMaxSelectK || n_salient < 0 || n_salient > K) return AWQ_ERR_SHAPE;
    if (n_salient == 0) return AWQ_OK;
    if (!m_f64 || !idx) return AWQ_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(m_f64) & 7) || (reinterpret_cast<uintptr_t>(idx) & 3)) return AWQ_ERR_ALIGN;
    return launch_select_salient(m_f64, K, n_salient, idx, as_stream(stream));
}

awq_status awq_quantize_salient(const void* w_f16, int64_t N, int64_t K, int group_size, int mode, const int* idx,
                                int n_salient, uint32_t* qweight, void* scales_f16, void* zeros_f16,
                                void* w_salient_f16, void* stream) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (N * K > kMaxElems || n_salient < 0 || n_salient > K) return AWQ_ERR_SHAPE;
    if (mode != AWQ_QUANT_ASYMMETRIC && mode != AWQ_QUANT_SYMMETRIC) return AWQ_ERR_CONFIG;
    if (N == 0) return AWQ_OK;
    if (!w_f16 || !qweight || !scales_f16 || !zeros_f16 || (n_salient > 0 && (!idx || !w_salient_f16)))
        return AWQ_ERR_NULL;
    if (!aligned16(w_f16) || !aligned16(qweight) || (reinterpret_cast<uintptr_t>(scales_f16) & 1) ||
        (reinterpret_cast<uintptr_t>(zeros_f16) & 1) || (reinterpret_cast<uintptr_t>(idx) & 3) ||
        (reinterpret_cast<uintptr_t>(w_salient_f16) & 1))
        return AWQ_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    const half_t* w = static_cast<const half_t*>(w_f16);
    if ((st = launch_quantize(w, nullptr, N, K, group_size, mode == AWQ_QUANT_SYMMETRIC, 0.0, qweight,
                              static_cast<half_t*>(scales_f16), static_cast<half_t*>(zeros_f16), s)) != AWQ_OK)
        return st;
    return launch_salient_fix(w, N, K, group_size, idx, n_salient, qweight, static_cast<const half_t*>(zeros_f16),
                              static_cast<half_t*>(w_salient_f16), s);
}

awq_status awq_salient_apply(const void* x_f16, const int* idx, const void* w_salient_f16, int64_t M, int64_t N,
                             int64_t K, int n_salient, void* y_f16, void* stream) {
    if (M < 0 || N < 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim || n_salient < 0 || n_salient > K)
        return AWQ_ERR_SHAPE;
    if (M == 0 || N == 0 || n_salient == 0) return AWQ_OK;
    if (!x_f16 || !idx || !w_salient_f16 || !y_f16) return AWQ_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(x_f16) & 1) || (reinterpret_cast<uintptr_t>(idx) & 3) ||
        (reinterpret_cast<uintptr_t>(w_salient_f16) & 1) || (reinterpret_cast<uintptr_t>(y_f16) & 1))
        return AWQ_ERR_ALIGN;
    return launch_salient_apply(static_cast<const half_t*>(x_f16), idx, static_cast<const half_t*>(w_salient_f16), M,
                                N, K, n_salient, static_cast<half_t*>(y_f16), as_stream(stream));
}

int64_t awq_salient_count(int64_t K) {
    if (K <= 0) return 0;
    // round(K / 100), ties to even (the default rounding mode)
    return static_cast<int64_t>(std::nearbyint(0.01 * static_cast<double>(K)));
}

size_t awq_salient_loss_workspace_bytes(int64_t N, int64_t K, int64_t T, int group_size, int n_salient) {
    if (n_salient < 0) n_salient = static_cast<int>(awq_salient_count(K));
    if (check_dims(N, K, group_size) != AWQ_OK || N <= 0 || T <= 0 || n_salient > K) return 0;
    return SalientLayout(nullptr, N, K, T, group_size, n_salient).bytes;
}

awq_status awq_salient_loss(const void* w_f16, const void* x_f16, int64_t N, int64_t K, int64_t T, int group_size,
                            int mode, int n_salient, void* workspace, size_t workspace_bytes, double* loss_rtn,
                            double* loss_salient, int* idx_out, void* stream) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (N <= 0 || T <= 0 || T > (int64_t(1) << 24) || K % 8 != 0) return AWQ_ERR_SHAPE;
    if (T > (int64_t(1) << 31) - 256 || N > (int64_t(1) << 31) - 256) return AWQ_ERR_SHAPE;
    if (n_salient < 0 && K <= kMaxSelectK) n_salient = static_cast<int>(awq_salient_count(K));
    if (K > kMaxSelectK || n_salient < 0 || n_salient > K) return AWQ_ERR_SHAPE;
    if (mode != AWQ_QUANT_ASYMMETRIC && mode != AWQ_QUANT_SYMMETRIC) return AWQ_ERR_CONFIG;
    if (!w_f16 || !x_f16 || !workspace || !loss_rtn || !loss_salient) return AWQ_ERR_NULL;
    if (!aligned16(w_f16) || !aligned16(x_f16) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(idx_out) & 3))
        return AWQ_ERR_ALIGN;
    SalientLayout L(workspace, N, K, T, group_size, n_salient);
    if (workspace_bytes < L.bytes) return AWQ_ERR_WORKSPACE;
    hipStream_t s = as_stream(stream);
    const half_t* w = static_cast<const half_t*>(w_f16);
    const half_t* x = static_cast<const half_t*>(x_f16);
    const bool sym = mode == AWQ_QUANT_SYMMETRIC;

    // salient channels from m = mean |x|
    if ((st = launch_absmean(x, T, K, L.m, L.abs_partials, s)) != AWQ_OK) return st;
    if ((st = launch_select_salient(L.m, K, n_salient, L.idx, s)) != AWQ_OK) return st;
    // reference W . x^T; the plain quantizer's loss
    if ((st = reference_output(x, w, T, N, K, group_size, L.yref, L.wt, s)) != AWQ_OK) return st;
    if ((st = launch_quantize(w, nullptr, N, K, group_size, sym, 0.0, L.qweight, L.scales, L.zeros, s)) != AWQ_OK)
        return st;
    if ((st = output_loss(x, L.qweight, L.scales, L.zeros, T, N, K, group_size, L.yref, L.tile_partials, L.losses,
                          s)) != AWQ_OK)
        return st;
    // mixed layer: INT4 part with the salient codes at the zero-point, fp16
    // side part moved to the reference: || x Q0^T - (W x^T - x_S W_S^T) ||^2
    if ((st = launch_salient_fix(w, N, K, group_size, L.idx, n_salient, L.qweight, L.zeros, L.w_sal, s)) != AWQ_OK)
        return st;
    if ((st = launch_salient_subtract(x, L.idx, L.w_sal, T, N, K, n_salient, L.yref, s)) != AWQ_OK) return st;
    if ((st = output_loss(x, L.qweight, L.scales, L.zeros, T, N, K, group_size, L.yref, L.tile_partials,
                          L.losses + 1, s)) != AWQ_OK)
        return st;
    if (idx_out && n_salient > 0 &&
        hipMemcpyAsync(idx_out, L.idx, sizeof(int) * n_salient, hipMemcpyDeviceToDevice, s) != hipSuccess)
        return AWQ_ERR_HIP;
    double host[2];
    if (hipMemcpyAsync(host, L.losses, sizeof(host), hipMemcpyDeviceToHost, s) != hipSuccess) return AWQ_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return AWQ_ERR_HIP;
    *loss_rtn = host[0];
    *loss_salient = host[1];
    return AWQ_OK;
}

awq_status awq_quantize_w8(const void* w_f16, const float* channel_scale, int64_t N, int64_t K, int group_size,
                           int mode, uint32_t* qweight, void* scales_f16, void* zeros_f16, void* stream) {
    awq_status st = check_dims(N, K, group_size);
    if (st != AWQ_OK) return st;
    if (group_size < 64) return AWQ_ERR_CONFIG;
    if (N * K > kMaxElems) return AWQ_ERR_SHAPE;
    if (mode != AWQ_QUANT_ASYMMETRIC && mode != AWQ_QUANT_SYMMETRIC) return AWQ_ERR_CONFIG;
    if (N == 0) return AWQ_OK;
    if (!w_f16 || !qweight || !scales_f16 || !zeros_f16) return AWQ_ERR_NULL;
    if (!aligned16(w_f16) || !aligned16(qweight) || (channel_scale && !aligned16(channel_scale)) ||
        (reinterpret_cast<uintptr_t>(scales_f16) & 1) || (reinterpret_cast<uintptr_t>(zeros_f16) & 1))
        return AWQ_ERR_ALIGN;
    return launch_quantize(static_cast<const half_t*>(w_f16), channel_scale, N, K, group_size,
                           mode == AWQ_QUANT_SYMMETRIC, 0.0, qweight, static_cast<half_t*>(scales_f16),
                           static_cast<half_t*>(zeros_f16), as_stream(stream), 8);
}

awq_status awq_gemm_w8(const void* x_f16, const uint32_t* qweight, const void* scales_f16, const void* zeros_f16,
                       int64_t M, int64_t N, int64_t K, int group_size, void* y_f16, int path, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return w8_dispatch(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, workspace,
                       workspace_bytes, as_stream(stream), nullptr);
}

awq_status awq_gemm_fused(const void* x_f16, const uint32_t* qweight, const void* scales_f16, const void* zeros_f16,
                          int64_t M, int64_t N, int64_t K, int group_size, int bits, const void* bias_f16,
                          int activation, const void* mul_f16, int64_t mul_stride, const void* residual_f16,
                          int64_t residual_stride, void* y_f16, int path, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (bits != 4 && bits != 8) return AWQ_ERR_CONFIG;
    if (activation < AWQ_ACT_NONE || activation > AWQ_ACT_GELU_TANH) return AWQ_ERR_CONFIG;
    if ((mul_f16 && (mul_stride < N || mul_stride > kMaxDim)) ||
        (residual_f16 && (residual_stride < N || residual_stride > kMaxDim)))
        return AWQ_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(bias_f16) & 1) || (reinterpret_cast<uintptr_t>(mul_f16) & 1) ||
        (reinterpret_cast<uintptr_t>(residual_f16) & 1))
        return AWQ_ERR_ALIGN;
    Epilogue e;
    e.bias = static_cast<const half_t*>(bias_f16);
    e.mul = static_cast<const half_t*>(mul_f16);
    e.residual = static_cast<const half_t*>(residual_f16);
    e.mul_stride = mul_stride;
    e.residual_stride = residual_stride;
    e.act = activation;
    e.vectors = N % 8 == 0 && aligned16(y_f16) && aligned16(bias_f16) && aligned16(mul_f16) &&
                aligned16(residual_f16) && (!mul_f16 || mul_stride % 8 == 0) &&
                (!residual_f16 || residual_stride % 8 == 0);
    // nothing to fuse: the plain kernels
    const bool plain = !bias_f16 && !mul_f16 && !residual_f16 && activation == AWQ_ACT_NONE;
    const Epilogue* epilogue = plain ? nullptr : &e;
    if (bits == 8)
        return w8_dispatch(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, workspace,
                           workspace_bytes, as_stream(stream), epilogue);
    return gemm_dispatch(x_f16, qweight, scales_f16, zeros_f16, M, N, K, group_size, y_f16, path, workspace,
                         workspace_bytes, true, false, as_stream(stream), epilogue);
}

}  // extern "C"

// ---- the paged cache ----
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks a cache and a batch and lays them out for the kernels. *empty is set
// when there is nothing to do (no sequence, no token).
awq_status kv_pages(const awq_kv_cache* cache, const awq_kv_seqs* seqs, int64_t n_tokens, KvPages* out, bool* empty) {
    if (!cache || !seqs) return AWQ_ERR_NULL;
    const bool int4 = cache->format == AWQ_KV_INT4;
    if (cache->format != AWQ_KV_INT8 && cache->format != AWQ_KV_E4M3 && !int4) return AWQ_ERR_CONFIG;
    const int page = cache->page_size, dim = cache->head_dim;
    if (page != 32 && page != 64 && page != 128 && page != 256) return AWQ_ERR_CONFIG;
    if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return AWQ_ERR_CONFIG;
    if (cache->n_pages < 1 || cache->n_pages > INT32_MAX || cache->n_kv_heads < 1 || cache->n_kv_heads > 65535)
        return AWQ_ERR_SHAPE;
    if (seqs->n_seqs < 0 || seqs->n_seqs > 32767 || seqs->max_pages < 0 || seqs->table_stride < seqs->max_pages ||
        seqs->max_tokens < 0 || seqs->max_tokens > INT32_MAX || seqs->max_len < 0 || seqs->max_len > kKvMaxLen ||
        n_tokens < 0 || n_tokens > INT32_MAX)
        return AWQ_ERR_SHAPE;
    *empty = seqs->n_seqs == 0 || seqs->max_tokens == 0 || n_tokens == 0;
    if (*empty) return AWQ_OK;
    if (!cache->k_codes || !cache->v_codes || !cache->k_scales || !cache->v_scales || !seqs->cu_tokens ||
        !seqs->kv_len || (seqs->max_pages > 0 && !seqs->block_table))
        return AWQ_ERR_NULL;
    if (!aligned16(cache->k_codes) || !aligned16(cache->v_codes) || !aligned4(cache->k_scales) ||
        !aligned4(cache->v_scales) || !aligned4(seqs->block_table) || !aligned4(seqs->cu_tokens) ||
        !aligned4(seqs->kv_len) || (int4 && (!aligned16(cache->k_scales) || !aligned16(cache->v_scales))))
        return AWQ_ERR_ALIGN;
    out->k_codes = static_cast<uint8_t*>(cache->k_codes);
    out->v_codes = static_cast<uint8_t*>(cache->v_codes);
    out->k_scales = static_cast<float*>(cache->k_scales);     // fp16 pairs behind them with AWQ_KV_INT4
    out->v_scales = static_cast<float*>(cache->v_scales);
    out->table = seqs->block_table;
    out->cu = seqs->cu_tokens;
    out->len = seqs->kv_len;
    out->table_stride = seqs->table_stride;
    out->max_pages = seqs->max_pages;
    out->n_pages = static_cast<int>(cache->n_pages);
    out->heads = cache->n_kv_heads;
    out->log2_page = 31 - __builtin_clz(static_cast<unsigned>(page));
    out->n_tokens = static_cast<int>(n_tokens);
    out->max_len = static_cast<int>(seqs->max_len);
    return AWQ_OK;
}

// strides of a token tensor: whole 16-byte pieces, not negative
bool strides_ok(int64_t token, int64_t head) {
    return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= kMaxDim && head <= kMaxDim;
}

}  // namespace

extern "C" {

awq_status awq_kv_write(const awq_kv_cache* cache, const awq_kv_seqs* seqs, const void* k_f16, int64_t k_token_stride,
                        int64_t k_head_stride, const void* v_f16, int64_t v_token_stride, int64_t v_head_stride,
                        int64_t n_tokens, void* stream) {
    KvWriteArgs a{};
    bool empty = false;
    const awq_status st = kv_pages(cache, seqs, n_tokens, &a.c, &empty);
    if (st != AWQ_OK) return st;
    if (!strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride)) return AWQ_ERR_SHAPE;
    if (empty || seqs->max_pages == 0) return AWQ_OK;
    if (!k_f16 || !v_f16) return AWQ_ERR_NULL;
    if (!aligned16(k_f16) || !aligned16(v_f16)) return AWQ_ERR_ALIGN;
    a.k = static_cast<const half_t*>(k_f16);
    a.v = static_cast<const half_t*>(v_f16);
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.head_dim = cache->head_dim;
    a.n_seqs = seqs->n_seqs;
    a.format = cache->format;
    a.max_tokens = std::min(seqs->max_tokens, n_tokens);
    return launch_kv_write(a, as_stream(stream));
}

awq_status awq_kv_read(const awq_kv_cache* cache, const awq_kv_seqs* seqs, void* k_f16, void* v_f16, int64_t n_tokens,
                       void* stream) {
    KvReadArgs a{};
    bool empty = false;
    const awq_status st = kv_pages(cache, seqs, n_tokens, &a.c, &empty);
    if (st != AWQ_OK) return st;
    if (empty || (!k_f16 && !v_f16)) return AWQ_OK;
    if (!aligned16(k_f16) || !aligned16(v_f16)) return AWQ_ERR_ALIGN;
    a.k = static_cast<half_t*>(k_f16);
    a.v = static_cast<half_t*>(v_f16);
    a.head_dim = cache->head_dim;
    a.n_seqs = seqs->n_seqs;
    a.format = cache->format;
    a.max_tokens = std::min(seqs->max_tokens, n_tokens);
    return launch_kv_read(a, as_stream(stream));
}

size_t awq_kv_attention_workspace_bytes(const awq_kv_cache* cache, const awq_kv_seqs* seqs, int n_heads) {
    KvPages c{};
    bool empty = false;
    if (kv_pages(cache, seqs, 1, &c, &empty) != AWQ_OK) return 0;
    if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 ||
        seqs->max_tokens * (n_heads / cache->n_kv_heads) > INT32_MAX - 256)
        return 0;
    if (empty) return 256;
    return kv_attention_workspace_bytes(cache->format, seqs->n_seqs, cache->n_kv_heads, n_heads / cache->n_kv_heads,
                                        cache->head_dim, seqs->max_tokens, seqs->max_len);
}

awq_status awq_kv_attention(const awq_kv_cache* cache, const awq_kv_seqs* seqs, const void* q_f16,
                            int64_t q_token_stride, int64_t q_head_stride, int64_t n_tokens, int n_heads, float scale,
                            int causal, int64_t window, void* out_f16, int64_t out_token_stride,
                            int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
    KvAttentionArgs a{};
    bool empty = false;
    const awq_status st = kv_pages(cache, seqs, n_tokens, &a.c, &empty);
    if (st != AWQ_OK) return st;
    if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 || n_tokens * n_heads > INT32_MAX ||
        seqs->max_tokens * (n_heads / cache->n_kv_heads) > INT32_MAX - 256)
        return AWQ_ERR_SHAPE;
    if (!strides_ok(q_token_stride, q_head_stride) || !strides_ok(out_token_stride, out_head_stride))
        return AWQ_ERR_SHAPE;
    // rows of the output that share memory would be written by several blocks
    if ((n_tokens > 1 && out_token_stride < cache->head_dim) || (n_heads > 1 && out_head_stride < cache->head_dim))
        return AWQ_ERR_SHAPE;
    if (n_tokens > 1 && n_heads > 1 && out_token_stride < (n_heads - 1) * out_head_stride + cache->head_dim &&
        out_head_stride < (n_tokens - 1) * out_token_stride + cache->head_dim)
        return AWQ_ERR_SHAPE;
    if (!std::isfinite(scale) || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal))
        return AWQ_ERR_CONFIG;
    if (empty) return AWQ_OK;
    if (!q_f16 || !out_f16) return AWQ_ERR_NULL;
    if (!aligned16(q_f16) || !aligned16(out_f16) || !aligned4(lse)) return AWQ_ERR_ALIGN;
    a.q = static_cast<const half_t*>(q_f16);
    a.out = static_cast<half_t*>(out_f16);
    a.lse = lse;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.head_dim = cache->head_dim;
    a.n_seqs = seqs->n_seqs;
    a.format = cache->format;
    a.ratio = n_heads / cache->n_kv_heads;
    a.by_ratio = KvDivisor(static_cast<uint32_t>(a.ratio));
    a.max_tokens = seqs->max_tokens;        // as the workspace query counts
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.causal = causal != 0;
    a.window = static_cast<int>(std::min<int64_t>(window, INT32_MAX));
    if (workspace) {
        if (reinterpret_cast<uintptr_t>(workspace) & 255) return AWQ_ERR_ALIGN;
        if (workspace_bytes < kv_attention_workspace_bytes(a.format, a.n_seqs, a.c.heads, a.ratio, a.head_dim,
                                                           a.max_tokens, a.c.max_len))
            return AWQ_ERR_WORKSPACE;
    }
    return launch_kv_attention(a, workspace, as_stream(stream));
}

}  // extern "C"

// ---- the norm and the rotary positions ----
namespace {

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

constexpr int64_t kMaxStride = int64_t{1} << 40;
bool stride_ok(int64_t stride, int64_t least) { return stride >= least && stride < kMaxStride; }

// a tensor of rotary positions: AWQ_OK and *out filled
awq_status rope_heads(const awq_rope_heads* t, int head_dim, int64_t n_tokens, RopeHeads* out) {
    *out = RopeHeads{};
    if (t == nullptr || t->heads == 0) return AWQ_OK;
    if (t->heads < 0 || t->heads > 65535) return AWQ_ERR_SHAPE;
    if (!stride_ok(t->in_token_stride, 0) || !stride_ok(t->in_head_stride, 0)) return AWQ_ERR_SHAPE;
    const bool tokens = n_tokens > 1, heads = t->heads > 1;
    if (!stride_ok(t->out_token_stride, tokens ? head_dim : 0) || !stride_ok(t->out_head_stride, heads ? head_dim : 0))
        return AWQ_ERR_SHAPE;
    // (2^24 tokens times a stride of 2^40 pass 64 bits)
    if (tokens && heads && t->out_token_stride < (t->heads - 1) * t->out_head_stride + head_dim &&
        t->out_head_stride < static_cast<__int128>(n_tokens - 1) * t->out_token_stride + head_dim)
        return AWQ_ERR_SHAPE;
    if (t->in == t->out && ((tokens && t->in_token_stride != t->out_token_stride) ||
                            (heads && t->in_head_stride != t->out_head_stride)))
        return AWQ_ERR_SHAPE;
    if (n_tokens > 0 && (!t->in || !t->out)) return AWQ_ERR_NULL;
    if (!aligned2(t->in) || !aligned2(t->out)) return AWQ_ERR_ALIGN;
    out->in = static_cast<const half_t*>(t->in);
    out->out = static_cast<half_t*>(t->out);
    out->in_token = t->in_token_stride;
    out->in_head = t->in_head_stride;
    out->out_token = t->out_token_stride;
    out->out_head = t->out_head_stride;
    out->heads = t->heads;
    return AWQ_OK;
}

}  // namespace

extern "C" {

awq_status awq_rmsnorm(const void* x_f16, int64_t x_stride, const void* residual_f16, int64_t residual_stride,
                       void* residual_out_f16, int64_t residual_out_stride, const void* weight_f16,
                       float weight_offset, float eps, int64_t rows, int64_t width, int format, int group_size,
                       void* out, int64_t out_stride, float* scales, void* stream) {
    if (format != AWQ_NORM_F16 && format != AWQ_NORM_INT8 && format != AWQ_NORM_E4M3) return AWQ_ERR_CONFIG;
    if (group_size != 0 && (format == AWQ_NORM_F16 || (group_size != 32 && group_size != 64 && group_size != 128 &&
                                                       group_size != 256 && group_size != 512)))
        return AWQ_ERR_CONFIG;
    // (an offset as large as the largest weight keeps the unscaled products in fp32)
    if (!(std::fabs(weight_offset) <= kHalfMax) || !std::isfinite(eps) || eps < 0.f) return AWQ_ERR_CONFIG;
    if (rows < 0 || rows >= int64_t{1} << 31 || width < 1 || width > int64_t{1} << 24 ||
        (group_size != 0 && width % group_size != 0))
        return AWQ_ERR_SHAPE;
    const int64_t least = rows > 1 ? width : 0;
    if (!stride_ok(x_stride, 0) || !stride_ok(out_stride, least) || (residual_f16 && !stride_ok(residual_stride, 0)) ||
        (residual_out_f16 && !stride_ok(residual_out_stride, least)))
        return AWQ_ERR_SHAPE;
    const auto same = [&](const void* o, int64_t os, const void* i, int64_t is) {
        return o && o == i && rows > 1 && os != is;
    };
    if (same(residual_out_f16, residual_out_stride, x_f16, x_stride) ||
        same(residual_out_f16, residual_out_stride, residual_f16, residual_stride) ||
        (format == AWQ_NORM_F16 &&
         (same(out, out_stride, x_f16, x_stride) || same(out, out_stride, residual_f16, residual_stride))))
        return AWQ_ERR_SHAPE;
    if (rows == 0) return AWQ_OK;
    if (!x_f16 || !out || (format != AWQ_NORM_F16 && !scales)) return AWQ_ERR_NULL;
    if (out == residual_out_f16) return AWQ_ERR_SHAPE;
    // 8-bit rows written over fp16 ones would overtake them
    if (format != AWQ_NORM_F16 && (out == x_f16 || out == residual_f16)) return AWQ_ERR_SHAPE;
    if (!aligned2(x_f16) || !aligned2(residual_f16) || !aligned2(residual_out_f16) || !aligned2(weight_f16) ||
        (format == AWQ_NORM_F16 && !aligned2(out)) || (format != AWQ_NORM_F16 && !aligned4(scales)))
        return AWQ_ERR_ALIGN;
    NormArgs a{};
    a.x = static_cast<const half_t*>(x_f16);
    a.residual = static_cast<const half_t*>(residual_f16);
    a.sum = static_cast<half_t*>(residual_out_f16);
    a.weight = static_cast<const half_t*>(weight_f16);
    a.out = out;
    a.scales = scales;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.sum_stride = residual_out_stride;
    a.out_stride = out_stride;
    a.rows = rows;
    a.width = width;
    a.offset = weight_offset;
    // The kernel's reciprocal root takes a subnormal number as 0, and a row of zeros
    // would be 0 / 0. The mean square of any other row is 2^-72 or more, beside
    // which no such eps shows.
    a.eps = eps > 0.f ? std::max(eps, std::numeric_limits<float>::min()) : eps;
    a.per_width = static_cast<float>(1.0 / static_cast<double>(width));
    a.format = format;
    a.group = group_size;
    return launch_rmsnorm(a, as_stream(stream));
}

awq_status awq_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double trained_len, double low,
                                double high, double* freqs, double* amplitude) {
    if (!freqs || !amplitude) return AWQ_ERR_NULL;
    if (rotary_dim < 2 || rotary_dim > 4096 || rotary_dim % 2 != 0) return AWQ_ERR_SHAPE;
    if (scaling < AWQ_ROPE_NONE || scaling > AWQ_ROPE_WAVELENGTH || !(base > 1.0) || !std::isfinite(base))
        return AWQ_ERR_CONFIG;
    const bool ramp = scaling == AWQ_ROPE_YARN || scaling == AWQ_ROPE_WAVELENGTH;
    if (scaling != AWQ_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return AWQ_ERR_CONFIG;
    if (ramp && (!(trained_len > 0.0) || !std::isfinite(trained_len) || !(low > 0.0) || !(high > low) ||
                 !std::isfinite(high)))
        return AWQ_ERR_CONFIG;
    if (scaling == AWQ_ROPE_NTK && rotary_dim == 2) return AWQ_ERR_CONFIG;
    constexpr double kTurn = 6.283185307179586;
    const double R = rotary_dim;
    const double b = scaling == AWQ_ROPE_NTK ? base * std::pow(factor, R / (R - 2.0)) : base;
    double first = 0.0, last = 0.0;
    if (scaling == AWQ_ROPE_YARN) {
        const auto pair = [&](double turns) { return R * std::log(trained_len / (kTurn * turns)) / (2.0 * std::log(base)); };
        first = std::max(std::floor(pair(high)), 0.0);
        last = std::min(std::ceil(pair(low)), R - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(b, -2.0 * i / R);
        double keep = 1.0;      // of the frequency that stays
        if (scaling == AWQ_ROPE_LINEAR) keep = 0.0;
        if (scaling == AWQ_ROPE_YARN)
            keep = 1.0 - std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
        if (scaling == AWQ_ROPE_WAVELENGTH)
            keep = std::min(std::max((trained_len * f / kTurn - low) / (high - low), 0.0), 1.0);
        freqs[i] = f * keep + f / factor * (1.0 - keep);
        if (keep == 1.0) freqs[i] = f;
    }
    *amplitude = scaling == AWQ_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return AWQ_OK;
}

awq_status awq_rope(const awq_rope_table* rope, const int32_t* positions, const awq_kv_seqs* seqs,
                    const awq_rope_heads* q, const awq_rope_heads* k, int head_dim, int64_t n_tokens, void* stream) {
    if (!rope) return AWQ_ERR_NULL;
    if (rope->layout != AWQ_ROPE_HALF && rope->layout != AWQ_ROPE_INTERLEAVED) return AWQ_ERR_CONFIG;
    if (!std::isfinite(rope->amplitude)) return AWQ_ERR_CONFIG;
    if (head_dim < 2 || head_dim > 4096 || rope->rotary_dim < 2 || rope->rotary_dim > head_dim ||
        rope->rotary_dim % 2 != 0 || n_tokens < 0 || n_tokens >= int64_t{1} << 24)
        return AWQ_ERR_SHAPE;
    if ((positions == nullptr) == (seqs == nullptr) && n_tokens > 0) return AWQ_ERR_NULL;
    if (seqs && (seqs->n_seqs < 0 || seqs->n_seqs > 32767 || seqs->max_tokens < 0 || seqs->max_tokens > INT32_MAX ||
                 seqs->max_len < 0 || seqs->max_len > kKvMaxLen))
        return AWQ_ERR_SHAPE;
    RopeArgs a{};
    awq_status st = rope_heads(q, head_dim, n_tokens, &a.q);
    if (st == AWQ_OK) st = rope_heads(k, head_dim, n_tokens, &a.k);
    if (st != AWQ_OK) return st;
    if (n_tokens == 0 || a.q.heads + a.k.heads == 0 || (seqs && (seqs->n_seqs == 0 || seqs->max_tokens == 0)))
        return AWQ_OK;
    if (!rope->freqs || (seqs && (!seqs->cu_tokens || !seqs->kv_len))) return AWQ_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(rope->freqs) & 7u) != 0 || !aligned4(positions) ||
        (seqs && (!aligned4(seqs->cu_tokens) || !aligned4(seqs->kv_len))))
        return AWQ_ERR_ALIGN;
    a.freqs = rope->freqs;
    a.positions = positions;
    a.n_tokens = static_cast<int>(n_tokens);
    a.dim = head_dim;
    a.rotary = rope->rotary_dim;
    a.amplitude = rope->amplitude;
    a.interleaved = rope->layout == AWQ_ROPE_INTERLEAVED;
    if (seqs) {
        a.cu = seqs->cu_tokens;
        a.len = seqs->kv_len;
        a.max_len = static_cast<int>(seqs->max_len);
    }
    return launch_rope(a, seqs ? std::min(seqs->max_tokens, n_tokens) : n_tokens, seqs ? seqs->n_seqs : 1,
                       as_stream(stream));
}

}  // extern "C"
