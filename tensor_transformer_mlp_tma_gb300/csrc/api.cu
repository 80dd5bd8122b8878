// The C ABI of libtpmlp.so (declared in include/tpmlp.h): argument validation,
// workspace layout, the launch sequence of the forward and backward passes, the
// device status word and per-kernel timing.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "kernels.h"
#include "tpmlp.h"

namespace tpmlp {

thread_local char g_last_error[512] = "";

void set_last_error(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
}

}  // namespace tpmlp

namespace {
std::atomic<uint64_t> g_launches{0};
}

void tpmlp::add_launches(uint64_t n) { g_launches.fetch_add(n); }

namespace {

using tpmlp::Epi;
using tpmlp::GemmArgs;

std::atomic<uint64_t> g_wait_ns{2000000000ull};

// ---- per-kernel timing --------------------------------------------------------
struct PendingTiming {
    std::string name;
    cudaEvent_t e0, e1;
};
struct TimingTotal {
    int64_t launches = 0;
    double ms = 0.0;
};
std::mutex g_prof_mu;
bool g_prof_on = false;
std::vector<PendingTiming> g_pending;
std::vector<cudaEvent_t> g_event_pool;
std::vector<std::pair<std::string, TimingTotal>> g_totals;

cudaEvent_t get_event() {
    if (!g_event_pool.empty()) {
        cudaEvent_t e = g_event_pool.back();
        g_event_pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
}

// Brackets one launch with events on its stream when timing is on.
struct Timed {
    const char *name;
    cudaStream_t st;
    cudaEvent_t e0 = nullptr, e1 = nullptr;
    Timed(const char *n, cudaStream_t s) : name(n), st(s) {
        std::lock_guard<std::mutex> lk(g_prof_mu);
        if (!g_prof_on) return;
        e0 = get_event();
        e1 = get_event();
        if (e0 && e1) cudaEventRecord(e0, st);
    }
    ~Timed() {
        if (!e0 || !e1) return;
        cudaEventRecord(e1, st);
        std::lock_guard<std::mutex> lk(g_prof_mu);
        g_pending.push_back({name, e0, e1});
    }
};

// ---- device properties -----------------------------------------------------------
int num_sms_current() {
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0) {
        int n = 0, major = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return 0;
        int minor = 0;
        if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return 0;
        cache[dev] = (major == 10 && minor == 3) ? n : -1;  // the kernels are built for sm_103a only
    }
    return cache[dev];
}

// ---- shapes and workspace --------------------------------------------------------------
// The GEMM kernels count output tiles (128 x 256 at the smallest, times the
// problem count) in 32-bit integers.
bool tiles_fit(int64_t M, int64_t N, int64_t batch = 1) {
    const int64_t t = ((M + 127) / 128) * ((N + 255) / 256);
    return t <= (int64_t{1} << 31) / 2 && batch <= (int64_t{1} << 31) / 2 / (t > 0 ? t : 1);
}

bool shape_valid(const tpmlp_shape *s) {
    if (!s) return false;
    if (s->tokens < 0 || s->hidden <= 0 || s->ffn <= 0) return false;
    if (s->t < 1 || s->t > 16 || s->ffn % s->t != 0) return false;
    if (s->dtype != TPMLP_F32 && s->dtype != TPMLP_BF16) return false;
    if (s->algo != TPMLP_ALGO_DEFAULT && s->algo != TPMLP_ALGO_SIMT) return false;
    if ((s->flags & ~(TPMLP_FLAG_RECOMPUTE | TPMLP_FLAG_LAYERNORM)) != 0) return false;
    // int32 tile and grid arithmetic inside the kernels
    if (s->tokens > (1LL << 30) || s->hidden > (1LL << 30) || s->ffn > (1LL << 30)) return false;
    const int64_t T = s->tokens, h = s->hidden, F = s->ffn;
    // the six GEMMs: T x F (fc1, dY), T x h (fc2, dX), F x h (dB), h x F (dA)
    if (!tiles_fit(T, F) || !tiles_fit(T, h) || !tiles_fit(F + 256, h) || !tiles_fit(h, F)) return false;
    return true;
}

size_t elt(const tpmlp_shape *s) { return s->dtype == TPMLP_BF16 ? 2 : 4; }

bool use_tc(const tpmlp_shape *s) { return s->dtype == TPMLP_BF16 && s->algo == TPMLP_ALGO_DEFAULT; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr size_t STATUS_BYTES = 1024;

// fp32 column-sum partials: the two-pass column sums of db (and of da on the
// FFMA path), or the per-32-row-block da partials written by the tensor-core
// GeLU' epilogue.  They are used one after the other, so they share one region.
size_t partials_bytes(const tpmlp_shape *s) {
    const int64_t T = s->tokens, h = s->hidden, F = s->ffn;
    int64_t n = tpmlp::colsum_chunks(T, h) * h;
    const int64_t p2 = tpmlp::colsum_chunks(T, F) * F;
    const int64_t p3 = (T + 31) / 32 * F;
    const int64_t p4 = (s->flags & TPMLP_FLAG_LAYERNORM) ? tpmlp::ln_partial_floats(T, h) : 0;
    n = n > p2 ? n : p2;
    n = n > p3 ? n : p3;
    n = n > p4 ? n : p4;
    return align_up(static_cast<size_t>(n) * sizeof(float), 1024);
}

size_t dy_offset(const tpmlp_shape *s) { return STATUS_BYTES + partials_bytes(s); }

size_t dy_bytes(const tpmlp_shape *s) {
    return align_up(static_cast<size_t>(s->tokens) * static_cast<size_t>(s->ffn) * elt(s), 1024);
}

bool recompute(const tpmlp_shape *s) { return (s->flags & TPMLP_FLAG_RECOMPUTE) != 0; }

size_t y_offset(const tpmlp_shape *s) { return dy_offset(s) + dy_bytes(s); }

size_t y_bytes(const tpmlp_shape *s) { return recompute(s) ? dy_bytes(s) : 0; }

bool layernorm(const tpmlp_shape *s) { return (s->flags & TPMLP_FLAG_LAYERNORM) != 0; }

size_t dxn_offset(const tpmlp_shape *s) { return y_offset(s) + y_bytes(s); }

size_t dxn_bytes(const tpmlp_shape *s) {
    return layernorm(s) ? align_up(static_cast<size_t>(s->tokens) * static_cast<size_t>(s->hidden) * elt(s), 1024)
                        : 0;
}

// 64 x 64 bf16 ones: the A operand of the bias-gradient tile of dB = Y^T dZ.
constexpr size_t ONES_BYTES = 64 * 64 * 2;

size_t ones_offset(const tpmlp_shape *s) { return dxn_offset(s) + dxn_bytes(s); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_elt(const void *p, size_t e) { return (reinterpret_cast<uintptr_t>(p) % e) == 0; }

// Checks common to forward and backward.  Returns OK, INVALID_ARG or UNSUPPORTED.
tpmlp_status check_ptrs(const tpmlp_shape *s, std::initializer_list<const void *> required,
                        std::initializer_list<const void *> optional) {
    for (const void *p : required)
        if (!p) return TPMLP_ERR_INVALID_ARG;
    const size_t e = elt(s);
    for (const void *p : required)
        if (!aligned_elt(p, e)) return TPMLP_ERR_UNSUPPORTED;
    for (const void *p : optional)
        if (p && !aligned_elt(p, e)) return TPMLP_ERR_UNSUPPORTED;
    if (use_tc(s)) {
        // TMA: 16-byte aligned bases and row pitches; shard boundaries on 64-element k-blocks.
        for (const void *p : required)
            if (!aligned16(p)) return TPMLP_ERR_UNSUPPORTED;
        for (const void *p : optional)
            if (p && !aligned16(p)) return TPMLP_ERR_UNSUPPORTED;
        if (s->hidden % 8 != 0 || s->ffn % 8 != 0) return TPMLP_ERR_UNSUPPORTED;
        if (s->t > 1 && (s->ffn / s->t) % 64 != 0) return TPMLP_ERR_UNSUPPORTED;
    }
    return TPMLP_OK;
}

tpmlp_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return TPMLP_OK;
    if (tpmlp::g_last_error[0] == '\0') tpmlp::set_last_error("%s", cudaGetErrorString(e));
    return TPMLP_ERR_CUDA;
}

tpmlp_status invalid(const char *why) {
    tpmlp::set_last_error("%s", why);
    return TPMLP_ERR_INVALID_ARG;
}

// One GEMM launch on the selected path.
cudaError_t gemm(const tpmlp_shape *s, const char *name, Epi epi, const GemmArgs &g, int sms,
                 cudaStream_t st) {
    Timed timed(name, st);
    cudaError_t e;
    if (use_tc(s))
        e = tpmlp::launch_tc_gemm(epi, g, sms, st);
    else
        e = tpmlp::launch_simt_gemm(epi, s->dtype == TPMLP_BF16, g, st);
    if (e == cudaSuccess && g.M > 0 && g.N > 0) g_launches.fetch_add(1);
    return e;
}

cudaError_t colsum(const tpmlp_shape *s, const char *name, const void *x, int64_t rows, int64_t cols,
                   float *partials, void *out, cudaStream_t st) {
    Timed timed(name, st);
    int n = 0;
    cudaError_t e = tpmlp::launch_colsum(s->dtype == TPMLP_BF16, x, rows, cols, partials, out, st, &n);
    g_launches.fetch_add(static_cast<uint64_t>(n));
    return e;
}

GemmArgs base_args(uint32_t *status) {
    GemmArgs g;
    std::memset(&g, 0, sizeof(g));
    g.nshards = 1;
    g.status = status;
    g.wait_ns = g_wait_ns.load();
    g.group = 1;
    g.raster_n = false;
    // CTA pairs (256 x 256 tiles) by default; TPMLP_CTA_PAIR=0 selects single-CTA
    // 128 x 256 tiles (a tuning knob, read per call).
    const char *pair = std::getenv("TPMLP_CTA_PAIR");
    g.cta_pair = !(pair && pair[0] == '0');
    return g;
}

// Raster order of the tensor-core GEMM tiles (256 x 256, 256 x 512 or 128 x 256).  Tiles are walked in
// super-rows of G tiles along M (or N); the G operand panels of the grouped
// dimension (each spans all of K) are re-read while the super-row lasts, so
// they should stay in L2, and each panel of the other operand is read once per
// super-row.  DRAM traffic is about  A + B * ceil(m_tiles / G)  (groups along M)
// or  B + A * ceil(n_tiles / G)  (along N); G is the largest group whose panels
// fit in the L2 budget, and the cheaper direction wins.
// TPMLP_RASTER=m:G or n:G overrides the choice (a tuning knob, read per call).
void pick_raster(GemmArgs &g, Epi epi = tpmlp::EPI_FOLD) {
    const int64_t tile_m = g.cta_pair ? 256 : 128;
    const int64_t tile_n = tpmlp::tc_wide_tile(epi, g) ? 512 : 256;
    const int64_t m_tiles = (g.M + tile_m - 1) / tile_m, n_tiles = (g.N + tile_n - 1) / tile_n;
    const char *env = std::getenv("TPMLP_RASTER");
    if (env && (env[0] == 'm' || env[0] == 'n') && env[1] == ':') {
        g.raster_n = env[0] == 'n';
        g.group = std::atoi(env + 2);
        return;
    }
    // At most 32 M-tiles (M is the token count or the hidden size in every GEMM
    // of the MLP and attention blocks at these sizes): walk up to 16 of them,
    // all where there are 16 or fewer, down each group of N columns.  Per GEMM
    // at h8192 (ncu, one kernel per capture) this order read 8-25% fewer DRAM
    // bytes than the panel-budget rule below and ran up to 2% faster alone.
    if (g.batch <= 1 && m_tiles <= 32) {
        g.raster_n = false;
        g.group = static_cast<int>(m_tiles < 16 ? m_tiles : 16);
        return;
    }
    const char *bud = std::getenv("TPMLP_L2_PANEL_MB");
    const double budget = (bud ? std::atof(bud) : 24.0) * 1048576.0;
    const double a_panel = static_cast<double>(tile_m) * g.K * 2, b_panel = static_cast<double>(tile_n) * g.K * 2;
    const double a_total = static_cast<double>(g.M) * g.K * 2, b_total = static_cast<double>(g.N) * g.K * 2;
    int64_t gm = static_cast<int64_t>(budget / a_panel), gn = static_cast<int64_t>(budget / b_panel);
    // Very long K makes panels too big for the budget; tiles that run in the same
    // wave still share panels while they walk K together, so keep the wave
    // roughly square: G between 8 and 24 tiles (measured best on GB300).
    gm = gm < 8 ? 8 : (gm > 24 ? 24 : gm);
    gn = gn < 8 ? 8 : (gn > 24 ? 24 : gn);
    gm = gm > m_tiles ? m_tiles : gm;
    gn = gn > n_tiles ? n_tiles : gn;
    const double tm = a_total + b_total * static_cast<double>((m_tiles + gm - 1) / gm);
    const double tn = b_total + a_total * static_cast<double>((n_tiles + gn - 1) / gn);
    g.raster_n = tn < tm;
    g.group = static_cast<int>(g.raster_n ? gn : gm);
}

}  // namespace

extern "C" {

const char *tpmlp_status_string(tpmlp_status s) {
    switch (s) {
        case TPMLP_OK: return "ok";
        case TPMLP_ERR_INVALID_ARG: return "invalid argument";
        case TPMLP_ERR_UNSUPPORTED: return "unsupported argument (alignment or shard size)";
        case TPMLP_ERR_CUDA: return "CUDA error";
        case TPMLP_ERR_TIMEOUT: return "device-side wait timed out";
        case TPMLP_ERR_DEVICE: return "no usable sm_100-family device";
    }
    return "unknown status";
}

int tpmlp_version(void) { return 100; }

const char *tpmlp_last_error(void) { return tpmlp::g_last_error; }

size_t tpmlp_saved_bytes(const tpmlp_shape *s) {
    if (!shape_valid(s)) return 0;
    return (recompute(s) ? 1 : 2) * static_cast<size_t>(s->tokens) * static_cast<size_t>(s->ffn) * elt(s);
}

size_t tpmlp_workspace_bytes(const tpmlp_shape *s) {
    if (!shape_valid(s)) return 0;
    return ones_offset(s) + ONES_BYTES;
}

size_t tpmlp_workspace_offset(const tpmlp_shape *s, int region) {
    if (!shape_valid(s)) return static_cast<size_t>(-1);
    switch (region) {
        case TPMLP_WS_STATUS: return 0;
        case TPMLP_WS_PARTIALS: return STATUS_BYTES;
        case TPMLP_WS_DY: return dy_offset(s);
        case TPMLP_WS_Y: return y_offset(s);
        case TPMLP_WS_DXN: return dxn_offset(s);
    }
    return static_cast<size_t>(-1);
}

}  // extern "C"

namespace {

tpmlp_status validate_forward(const tpmlp_shape *s, const void *X, const void *A, const void *a, const void *B,
                              const void *b, const void *Z, const tpmlp_saved *saved, const void *workspace) {
    if (!shape_valid(s)) return invalid("tpmlp_forward: invalid shape");
    if (!workspace) return invalid("tpmlp_forward: workspace is NULL");
    if (!aligned16(workspace)) return TPMLP_ERR_UNSUPPORTED;
    // Inference (saved == NULL): nothing is kept; Y goes to the workspace.
    if (!saved)
        return s->tokens == 0 ? check_ptrs(s, {A, a, B, b}, {X, Z}) : check_ptrs(s, {X, A, a, B, b, Z}, {});
    // With no tokens the [T, .] tensors are empty and may have NULL data pointers.
    // Under recomputation H is the saved activation and Y lives in the workspace.
    const bool rec = recompute(s);
    return s->tokens == 0 ? check_ptrs(s, {A, a, B, b}, {X, Z, saved->Y, saved->H})
           : rec          ? check_ptrs(s, {X, A, a, B, b, Z, saved->H}, {saved->Y})
                          : check_ptrs(s, {X, A, a, B, b, Z, saved->Y}, {saved->H});
}

tpmlp_status validate_backward(const tpmlp_shape *s, const void *dZ, const tpmlp_saved *saved, const void *dX,
                               const void *dA, const void *da, const void *dB, const void *db,
                               const void *workspace) {
    if (!shape_valid(s)) return invalid("tpmlp_backward: invalid shape");
    if (!saved || !workspace) return invalid("tpmlp_backward: saved or workspace is NULL");
    if (!aligned16(workspace)) return TPMLP_ERR_UNSUPPORTED;
    const bool rec = recompute(s);
    return s->tokens == 0
               ? check_ptrs(s, {saved->A, saved->B, dA, da, dB, db}, {dZ, saved->X, saved->H, saved->Y, dX})
           : rec ? check_ptrs(s, {dZ, saved->X, saved->A, saved->B, saved->H, dX, dA, da, dB, db}, {saved->Y})
                 : check_ptrs(s, {dZ, saved->X, saved->A, saved->B, saved->H, saved->Y, dX, dA, da, dB, db}, {});
}

}  // namespace

extern "C" {

tpmlp_status tpmlp_forward(const tpmlp_shape *s, const void *X, const void *A, const void *a,
                           const void *B, const void *b, void *Z, tpmlp_saved *saved,
                           void *workspace, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    tpmlp_status rc = validate_forward(s, X, A, a, B, b, Z, saved, workspace);
    if (rc != TPMLP_OK) return rc;
    const bool rec = recompute(s);
    if (saved) {
        saved->X = X;
        saved->A = A;
        saved->B = B;
    }
    const int64_t T = s->tokens, h = s->hidden, F = s->ffn;
    if (T == 0) return TPMLP_OK;
    const int sms = num_sms_current();
    if (sms == 0) return TPMLP_ERR_CUDA;
    if (use_tc(s) && sms < 0) return TPMLP_ERR_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t *status = static_cast<uint32_t *>(workspace);
    // Y: the caller's buffer; under recomputation the workspace's Y region; for
    // inference (saved == NULL) the workspace's dY region, which only the
    // backward pass uses.
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    void *Y = !saved ? static_cast<void *>(ws + dy_offset(s)) : (rec ? static_cast<void *>(ws + y_offset(s)) : saved->Y);

    // Column-parallel GEMM of all shards, bias and GeLU fused: H = X A + a, Y = GeLU(H).
    GemmArgs g1 = base_args(status);
    g1.a = X, g1.a_mn = false;  // X[T,h]: K-major
    g1.b = A, g1.b_mn = true;   // A[h,F]: N contiguous, MN-major
    g1.M = T, g1.N = F, g1.K = h, g1.kshard = h;
    g1.out0 = saved ? saved->H : nullptr, g1.out1 = Y, g1.bias = a;
    pick_raster(g1, tpmlp::EPI_BIAS_GELU);
    cudaError_t e = gemm(s, "fc1_bias_gelu", tpmlp::EPI_BIAS_GELU, g1, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // Row-parallel GEMM, one accumulation per shard, shard partials folded in order, + b.
    GemmArgs g2 = base_args(status);
    g2.a = Y, g2.a_mn = false;  // Y[T,F]: K-major
    g2.b = B, g2.b_mn = true;          // B[F,h]: MN-major
    g2.M = T, g2.N = h, g2.K = F;
    g2.nshards = s->t, g2.kshard = F / s->t;
    g2.out0 = Z, g2.bias = b;
    pick_raster(g2);
    e = gemm(s, "fc2_shard_fold", tpmlp::EPI_FOLD_BIAS, g2, sms, st);
    return from_cuda(e);
}

tpmlp_status tpmlp_backward(const tpmlp_shape *s, const void *dZ, const tpmlp_saved *saved, void *dX,
                            void *dA, void *da, void *dB, void *db, void *workspace, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    tpmlp_status rc = validate_backward(s, dZ, saved, dX, dA, da, dB, db, workspace);
    if (rc != TPMLP_OK) return rc;
    const bool rec = recompute(s);
    const int64_t T = s->tokens, h = s->hidden, F = s->ffn;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // Empty batch: the weight and bias gradients are sums over no tokens.
        cudaError_t e = cudaMemsetAsync(dA, 0, static_cast<size_t>(h) * F * elt(s), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, static_cast<size_t>(F) * h * elt(s), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(da, 0, static_cast<size_t>(F) * elt(s), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(db, 0, static_cast<size_t>(h) * elt(s), st);
        return from_cuda(e);
    }
    const int sms = num_sms_current();
    if (sms == 0) return TPMLP_ERR_CUDA;
    if (use_tc(s) && sms < 0) return TPMLP_ERR_DEVICE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);
    float *partials = reinterpret_cast<float *>(ws + STATUS_BYTES);
    void *dY = ws + dy_offset(s);
    // Under recomputation the GeLU' epilogue rebuilds Y = GeLU(H) into the workspace.
    void *Y = rec ? static_cast<void *>(ws + y_offset(s)) : saved->Y;

    // db = column sums of dZ: on tensor cores from the dB GEMM's ones tile (below,
    // its block of ones is filled by the da pass), on the FFMA path a two-pass
    // column sum.
    void *ones = ws + ones_offset(s);
    cudaError_t e = cudaSuccess;
    if (!use_tc(s)) {
        e = colsum(s, "colsum_db", dZ, T, h, partials, db, st);
        if (e != cudaSuccess) return from_cuda(e);
    }

    // dY = (dZ B^T) * GeLU'(H)
    GemmArgs g3 = base_args(status);
    g3.a = dZ, g3.a_mn = false;        // dZ[T,h]: K-major
    g3.b = saved->B, g3.b_mn = false;  // B[F,h] as [N=F, K=h]: K-major
    g3.M = T, g3.N = F, g3.K = h, g3.kshard = h;
    g3.out0 = dY, g3.aux = saved->H;
    g3.out1 = rec ? Y : nullptr;
    // On tensor cores the epilogue also sums dY's columns per 32-row block.
    g3.colsum_part = use_tc(s) ? partials : nullptr;
    pick_raster(g3, tpmlp::EPI_DGELU);
    e = gemm(s, "bwd_dY_dgelu", tpmlp::EPI_DGELU, g3, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // da = column sums of dY: the in-order sum of those block partials, or a
    // two-pass column sum of dY on the FFMA path.
    if (use_tc(s)) {
        Timed timed("da_block_sum", st);
        e = tpmlp::launch_colsum_final(true, partials, (T + 31) / 32, F, da, st, ones);
        if (e == cudaSuccess) g_launches.fetch_add(1);
    } else {
        e = colsum(s, "colsum_da", dY, T, F, partials, da, st);
    }
    if (e != cudaSuccess) return from_cuda(e);

    // dB = Y^T dZ
    GemmArgs g4 = base_args(status);
    g4.a = Y, g4.a_mn = true;  // Y[T,F] as [K=T, M=F]: MN-major
    g4.b = dZ, g4.b_mn = true;        // dZ[T,h] as [K=T, N=h]: MN-major
    g4.M = F, g4.N = h, g4.K = T, g4.kshard = T;
    g4.out0 = dB;
    if (use_tc(s)) g4.ones = ones, g4.bias_grad = db;  // db = 1^T dZ from an extra ones tile
    pick_raster(g4, tpmlp::EPI_STORE);
    e = gemm(s, "bwd_dB", tpmlp::EPI_STORE, g4, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dA = X^T dY
    GemmArgs g5 = base_args(status);
    g5.a = saved->X, g5.a_mn = true;  // X[T,h] as [K=T, M=h]: MN-major
    g5.b = dY, g5.b_mn = true;        // dY[T,F] as [K=T, N=F]: MN-major
    g5.M = h, g5.N = F, g5.K = T, g5.kshard = T;
    g5.out0 = dA;
    pick_raster(g5, tpmlp::EPI_STORE);
    e = gemm(s, "bwd_dA", tpmlp::EPI_STORE, g5, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dX = sum_i dY_i A_i^T, shard partials folded in order (the backward all-reduce)
    GemmArgs g6 = base_args(status);
    g6.a = dY, g6.a_mn = false;        // dY[T,F]: K-major
    g6.b = saved->A, g6.b_mn = false;  // A[h,F] as [N=h, K=F]: K-major
    g6.M = T, g6.N = h, g6.K = F;
    g6.nshards = s->t, g6.kshard = F / s->t;
    g6.out0 = dX;
    pick_raster(g6);
    e = gemm(s, "bwd_dX_shard_fold", tpmlp::EPI_FOLD, g6, sms, st);
    return from_cuda(e);
}

tpmlp_status tpmlp_ln_forward(const tpmlp_shape *s, tpmlp_layernorm *ln, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    if (!shape_valid(s) || !ln) return invalid("tpmlp_ln_forward: invalid shape or NULL layernorm");
    if (!(ln->eps >= 0.0f)) return invalid("tpmlp_ln_forward: eps must be >= 0");
    const int64_t T = s->tokens;
    tpmlp_status rc = T > 0 ? check_ptrs(s, {ln->X_in, ln->gamma, ln->beta, ln->Xn}, {})
                            : check_ptrs(s, {ln->gamma, ln->beta}, {ln->X_in, ln->Xn});
    if (rc != TPMLP_OK) return rc;
    if (T > 0 && (!ln->mean || !ln->rstd)) return invalid("tpmlp_ln_forward: NULL mean or rstd");
    if (T == 0) return TPMLP_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    tpmlp::LnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = T, a.h = s->hidden, a.eps = ln->eps;
    a.x = ln->X_in, a.gamma = ln->gamma, a.beta = ln->beta, a.y = ln->Xn, a.mean = ln->mean, a.rstd = ln->rstd;
    Timed timed("ln_forward", st);
    cudaError_t e = tpmlp::launch_ln_forward(s->dtype == TPMLP_BF16, a, st);
    if (e == cudaSuccess) g_launches.fetch_add(1);
    return from_cuda(e);
}

tpmlp_status tpmlp_ln_backward(const tpmlp_shape *s, const tpmlp_layernorm *ln, const void *dXn, void *dX_in,
                               void *dgamma, void *dbeta, void *workspace, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    if (!shape_valid(s) || !ln || !workspace) return invalid("tpmlp_ln_backward: invalid shape or NULL argument");
    if (!layernorm(s)) return invalid("tpmlp_ln_backward: the shape needs TPMLP_FLAG_LAYERNORM (workspace size)");
    const int64_t T = s->tokens;
    tpmlp_status rc = T > 0 ? check_ptrs(s, {dXn, ln->X_in, ln->gamma, dX_in, dgamma, dbeta}, {})
                            : check_ptrs(s, {ln->gamma, dgamma, dbeta}, {dXn, ln->X_in, dX_in});
    if (rc != TPMLP_OK) return rc;
    if (T > 0 && (!ln->mean || !ln->rstd)) return invalid("tpmlp_ln_backward: NULL mean or rstd");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    tpmlp::LnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = T, a.h = s->hidden, a.eps = ln->eps;
    a.x = ln->X_in, a.gamma = ln->gamma, a.mean = ln->mean, a.rstd = ln->rstd;
    a.dy = dXn, a.dx = dX_in, a.dgamma = dgamma, a.dbeta = dbeta;
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + STATUS_BYTES);
    Timed timed("ln_backward", st);
    int n = 0;
    cudaError_t e = tpmlp::launch_ln_backward(s->dtype == TPMLP_BF16, a, st, &n);
    g_launches.fetch_add(static_cast<uint64_t>(n));
    return from_cuda(e);
}

tpmlp_status tpmlp_sp_forward(const tpmlp_shape *s, tpmlp_layernorm *ln, const void *A, const void *a,
                              const void *B, const void *b, void *Z, tpmlp_saved *saved, void *workspace,
                              void *stream) {
    if (!shape_valid(s) || !ln) return invalid("tpmlp_sp_forward: invalid shape or NULL layernorm");
    if (!layernorm(s)) return invalid("tpmlp_sp_forward: the shape needs TPMLP_FLAG_LAYERNORM");
    // Validate the whole call before the first launch.
    tpmlp_status rc = validate_forward(s, ln->Xn, A, a, B, b, Z, saved, workspace);
    if (rc != TPMLP_OK) return rc;
    if (s->tokens > 0 && (!ln->X_in || !ln->mean || !ln->rstd)) return invalid("tpmlp_sp_forward: NULL layernorm buffer");
    rc = tpmlp_ln_forward(s, ln, stream);
    if (rc != TPMLP_OK) return rc;
    return tpmlp_forward(s, ln->Xn, A, a, B, b, Z, saved, workspace, stream);
}

tpmlp_status tpmlp_sp_backward(const tpmlp_shape *s, const tpmlp_layernorm *ln, const void *dZ,
                               const tpmlp_saved *saved, void *dX_in, void *dgamma, void *dbeta, void *dA,
                               void *da, void *dB, void *db, void *workspace, void *stream) {
    if (!shape_valid(s) || !ln || !workspace) return invalid("tpmlp_sp_backward: invalid shape or NULL argument");
    if (!layernorm(s)) return invalid("tpmlp_sp_backward: the shape needs TPMLP_FLAG_LAYERNORM");
    void *dXn = static_cast<uint8_t *>(workspace) + dxn_offset(s);
    void *dXn_or_null = s->tokens > 0 ? dXn : nullptr;
    // Validate the whole call before the first launch.
    tpmlp_status rc = validate_backward(s, dZ, saved, dXn_or_null, dA, da, dB, db, workspace);
    if (rc != TPMLP_OK) return rc;
    rc = s->tokens > 0 ? check_ptrs(s, {ln->X_in, ln->gamma, dX_in, dgamma, dbeta}, {})
                       : check_ptrs(s, {ln->gamma, dgamma, dbeta}, {ln->X_in, dX_in});
    if (rc != TPMLP_OK) return rc;
    if (s->tokens > 0 && (!ln->mean || !ln->rstd)) return invalid("tpmlp_sp_backward: NULL mean or rstd");
    rc = tpmlp_backward(s, dZ, saved, dXn_or_null, dA, da, dB, db, workspace, stream);
    if (rc != TPMLP_OK) return rc;
    return tpmlp_ln_backward(s, ln, dXn, dX_in, dgamma, dbeta, workspace, stream);
}

tpmlp_status tpmlp_check_device_status(void *workspace, void *stream) {
    if (!workspace) return TPMLP_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t words[2] = {0, 0};
    cudaError_t e = cudaMemcpyAsync(words, workspace, sizeof(words), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return TPMLP_ERR_CUDA;
    if (words[0] != 0) {
        e = cudaMemsetAsync(workspace, 0, sizeof(words), st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
        if (e != cudaSuccess) return TPMLP_ERR_CUDA;
    }
    if (words[0] > TPMLP_ERR_DEVICE) return TPMLP_ERR_DEVICE;
    return static_cast<tpmlp_status>(words[0]);
}

void tpmlp_set_wait_limit_ns(uint64_t ns) { g_wait_ns.store(ns == 0 ? 1 : ns); }

tpmlp_status tpmlp_debug_timeout_probe(void *workspace, uint64_t wait_ns, void *stream) {
    if (!workspace) return TPMLP_ERR_INVALID_ARG;
    if (wait_ns > 10000000000ull) return TPMLP_ERR_INVALID_ARG;  // at most 10 s
    const int sms = num_sms_current();
    if (sms == 0) return TPMLP_ERR_CUDA;
    if (sms < 0) return TPMLP_ERR_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Timed timed("timeout_probe", st);
    cudaError_t e = tpmlp::launch_timeout_probe(static_cast<uint32_t *>(workspace), wait_ns, st);
    if (e == cudaSuccess) g_launches.fetch_add(1);
    return from_cuda(e);
}

uint64_t tpmlp_launch_count(void) { return g_launches.load(); }

void tpmlp_profile_enable(int on) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_on = on != 0;
}

void tpmlp_profile_reset(void) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    for (auto &p : g_pending) {
        g_event_pool.push_back(p.e0);
        g_event_pool.push_back(p.e1);
    }
    g_pending.clear();
    g_totals.clear();
}

tpmlp_status tpmlp_profile_collect(void) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    tpmlp_status rc = TPMLP_OK;
    for (auto &p : g_pending) {
        float ms = 0.0f;
        if (cudaEventSynchronize(p.e1) != cudaSuccess || cudaEventElapsedTime(&ms, p.e0, p.e1) != cudaSuccess) {
            rc = TPMLP_ERR_CUDA;
        } else {
            bool found = false;
            for (auto &t : g_totals)
                if (t.first == p.name) {
                    t.second.launches += 1;
                    t.second.ms += ms;
                    found = true;
                    break;
                }
            if (!found) {
                TimingTotal tt;
                tt.launches = 1;
                tt.ms = ms;
                g_totals.emplace_back(p.name, tt);
            }
        }
        g_event_pool.push_back(p.e0);
        g_event_pool.push_back(p.e1);
    }
    g_pending.clear();
    return rc;
}

int tpmlp_profile_count(void) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    return static_cast<int>(g_totals.size());
}

int tpmlp_profile_entry(int i, char *name, int name_len, int64_t *launches, double *total_ms) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (i < 0 || i >= static_cast<int>(g_totals.size())) return -1;
    const auto &t = g_totals[static_cast<size_t>(i)];
    if (name && name_len > 0) {
        std::strncpy(name, t.first.c_str(), static_cast<size_t>(name_len - 1));
        name[name_len - 1] = '\0';
    }
    if (launches) *launches = t.second.launches;
    if (total_ms) *total_ms = t.second.ms;
    return 0;
}

}  // extern "C"

// ---- tensor-parallel self-attention block ------------------------------------------------
namespace {

bool attn_shape_valid(const tpmlp_attn_shape *s) {
    if (!s) return false;
    if (s->batch < 0 || s->seq <= 0 || s->hidden <= 0 || s->heads <= 0) return false;
    if (s->t < 1 || s->t > 16 || s->heads % s->t != 0 || s->hidden % s->heads != 0) return false;
    if ((s->flags & ~TPMLP_ATTN_P_UPPER_ZERO) != 0) return false;
    // int32 tile and grid arithmetic inside the kernels
    if (s->hidden > (1LL << 28) || s->seq > (1LL << 20) || s->batch * s->seq > (1LL << 30)) return false;
    if (static_cast<int64_t>(s->batch) * s->heads > (1LL << 24)) return false;
    // tile counts of the projections and the per-head products; the scores
    // ([batch*heads][seq][seq]) must be addressable
    const int64_t T = s->batch * s->seq, h = s->hidden, nz = s->batch * s->heads;
    if (!tiles_fit(T, 3 * h) || !tiles_fit(h + 256, 3 * h) || !tiles_fit(s->seq, s->seq, nz)) return false;
    if (static_cast<double>(nz) * s->seq * s->seq > static_cast<double>(1LL << 48)) return false;
    return true;
}

// Device workspace of the attention block, 1 KB-aligned regions:
//   status | D [batch*heads*seq] fp32 | dO [T,h] bf16 | dQKV [T,3h] bf16 |
//   scores [batch*heads][seq][seq] fp16 (the backward reuses it for dS in bf16) |
//   a 64 x 64 bf16 block of ones (bias-gradient tiles).
// The per-head GEMMs address Q, K, V, O, dO, dQ, dK, dV in place inside the
// token-major QKV, O, dO and dQKV arrays (4-D and 5-D tensor maps).
struct AttnLayout {
    size_t D, dO, dQKV, scores, ones, total;
};

AttnLayout attn_layout(const tpmlp_attn_shape *s) {
    const int64_t T = s->batch * s->seq, h = s->hidden;
    AttnLayout L;
    size_t off = STATUS_BYTES;
    L.D = off;
    off += align_up(static_cast<size_t>(T) * s->heads * 4, 1024);
    const size_t th = align_up(static_cast<size_t>(T) * h * 2, 1024);
    L.dO = off;
    off += th;
    L.dQKV = off;
    off += 3 * th;
    L.scores = off;
    off += align_up(static_cast<size_t>(s->batch) * s->heads * s->seq * s->seq * 2, 1024);
    L.ones = off;
    off += ONES_BYTES;
    L.total = off;
    return L;
}

// The MLP shape that routes the attention GEMMs and column sums to the bf16
// tensor-core path.
tpmlp_shape attn_route(const tpmlp_attn_shape *s) {
    tpmlp_shape m;
    std::memset(&m, 0, sizeof(m));
    m.tokens = s->batch * s->seq;
    m.hidden = s->hidden;
    m.ffn = 3 * s->hidden;
    m.t = s->t;
    m.dtype = TPMLP_BF16;
    m.algo = TPMLP_ALGO_DEFAULT;
    return m;
}

tpmlp::HeadLayout head_layout(const tpmlp_attn_shape *s) {
    tpmlp::HeadLayout L;
    L.nb = s->batch;
    L.S = s->seq;
    L.h = s->hidden;
    L.heads = s->heads;
    L.d = s->hidden / s->heads;
    return L;
}

// Head g's Q (which = 0), K (1) or V (2) columns inside a token-major [T, 3h]
// array with shard-major columns (QKV, dQKV), as a rank-5 view; its base is the
// array plus which * h/t elements.
tpmlp::HeadView qkv_view(const tpmlp_attn_shape *s) {
    tpmlp::HeadView v;
    v.rank = 5;
    v.S = s->seq;
    v.nb = s->batch;
    v.heads = s->heads;
    v.hpt = s->heads / s->t;
    v.d = s->hidden / s->heads;
    v.ld = 3 * s->hidden;
    v.coli = 3 * s->hidden / s->t;
    return v;
}

// Head g's columns [g*d, (g+1)*d) of a token-major [T, h] array (O, dO), rank 4.
tpmlp::HeadView tok_view(const tpmlp_attn_shape *s) {
    tpmlp::HeadView v;
    v.rank = 4;
    v.S = s->seq;
    v.nb = s->batch;
    v.heads = s->heads;
    v.hpt = s->heads / s->t;
    v.d = s->hidden / s->heads;
    v.ld = s->hidden;
    v.coli = 0;
    return v;
}

const void *qkv_part(const void *base, const tpmlp_attn_shape *s, int which) {
    return static_cast<const uint8_t *>(base) + static_cast<size_t>(which) * (s->hidden / s->t) * 2;
}

tpmlp_status attn_check(const tpmlp_attn_shape *s, const char *who, std::initializer_list<const void *> required,
                        std::initializer_list<const void *> token_ptrs, const void *workspace) {
    if (!attn_shape_valid(s)) {
        tpmlp::set_last_error("%s: invalid shape", who);
        return TPMLP_ERR_INVALID_ARG;
    }
    if (!workspace) {
        tpmlp::set_last_error("%s: workspace is NULL", who);
        return TPMLP_ERR_INVALID_ARG;
    }
    const bool empty = s->batch == 0;
    for (const void *p : required)
        if (!p) {
            tpmlp::set_last_error("%s: NULL pointer", who);
            return TPMLP_ERR_INVALID_ARG;
        }
    for (const void *p : token_ptrs)
        if (!p && !empty) {
            tpmlp::set_last_error("%s: NULL pointer", who);
            return TPMLP_ERR_INVALID_ARG;
        }
    if (s->dtype != TPMLP_BF16) {
        tpmlp::set_last_error("%s: the attention block runs in bf16 only", who);
        return TPMLP_ERR_UNSUPPORTED;
    }
    const int64_t d = s->hidden / s->heads;
    if (d % 64 != 0 || s->seq % 8 != 0) {
        tpmlp::set_last_error("%s: head size %lld must be a multiple of 64 and seq %lld of 8", who,
                              static_cast<long long>(d), static_cast<long long>(s->seq));
        return TPMLP_ERR_UNSUPPORTED;
    }
    if (!aligned16(workspace)) return TPMLP_ERR_UNSUPPORTED;
    for (const void *p : required)
        if (!aligned16(p)) return TPMLP_ERR_UNSUPPORTED;
    for (const void *p : token_ptrs)
        if (p && !aligned16(p)) return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

// One batched GEMM of the per-head products.
GemmArgs head_gemm(uint32_t *status, const void *a, bool a_mn, const void *b, bool b_mn, int64_t M, int64_t N,
                   int64_t K, int64_t batch, void *out) {
    GemmArgs g = base_args(status);
    g.a = a, g.a_mn = a_mn;
    g.b = b, g.b_mn = b_mn;
    g.M = M, g.N = N, g.K = K, g.kshard = K;
    g.batch = batch;
    g.out0 = out;
    pick_raster(g);
    return g;
}

}  // namespace

extern "C" {

size_t tpmlp_attn_saved_bytes(const tpmlp_attn_shape *s) {
    if (!attn_shape_valid(s)) return 0;
    const size_t T = static_cast<size_t>(s->batch * s->seq), h = static_cast<size_t>(s->hidden);
    return 2 * (T * 3 * h + T * h + static_cast<size_t>(s->batch) * s->heads * s->seq * s->seq);
}

size_t tpmlp_attn_workspace_bytes(const tpmlp_attn_shape *s) {
    if (!attn_shape_valid(s)) return 0;
    return attn_layout(s).total;
}

tpmlp_status tpmlp_attn_forward(const tpmlp_attn_shape *s, const void *X, const void *Wqkv, const void *bqkv,
                                const void *Wo, const void *bo, void *Z, tpmlp_attn_saved *saved, void *workspace,
                                void *stream) {
    tpmlp::g_last_error[0] = '\0';
    if (!saved) return invalid("tpmlp_attn_forward: saved is NULL");
    tpmlp_status rc = attn_check(s, "tpmlp_attn_forward", {Wqkv, bqkv, Wo, bo},
                                 {X, Z, saved->QKV, saved->P, saved->O}, workspace);
    if (rc != TPMLP_OK) return rc;
    saved->X = X;
    saved->Wqkv = Wqkv;
    saved->Wo = Wo;
    if (s->batch == 0) return TPMLP_OK;
    const int sms = num_sms_current();
    if (sms == 0) return TPMLP_ERR_CUDA;
    if (sms < 0) return TPMLP_ERR_DEVICE;
    const tpmlp_shape ms = attn_route(s);
    const AttnLayout L = attn_layout(s);
    const int64_t T = s->batch * s->seq, h = s->hidden, S = s->seq, d = h / s->heads;
    const int64_t nz = s->batch * s->heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);
    void *scores = ws + L.scores;
    const tpmlp::HeadView qv = qkv_view(s), tv = tok_view(s);
    const void *Qp = qkv_part(saved->QKV, s, 0), *Kp = qkv_part(saved->QKV, s, 1), *Vp = qkv_part(saved->QKV, s, 2);

    // Column-parallel projection of all shards: QKV = X Wqkv + bqkv (the bias
    // epilogue without an activation, on 256 x 512 tiles).
    GemmArgs g1 = base_args(status);
    g1.a = X, g1.a_mn = false;     // X[T,h]: K-major
    g1.b = Wqkv, g1.b_mn = true;   // Wqkv[h,3h]: MN-major
    g1.M = T, g1.N = 3 * h, g1.K = h, g1.kshard = h;
    g1.out0 = saved->QKV, g1.out1 = nullptr, g1.bias = bqkv;
    pick_raster(g1, tpmlp::EPI_BIAS_GELU);
    cudaError_t e = gemm(&ms, "attn_qkv_proj", tpmlp::EPI_BIAS_GELU, g1, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // Scores of every head: scale * Q K^T, causal; Q and K read in place in QKV.
    GemmArgs g2 = head_gemm(status, Qp, false, Kp, false, S, S, d, nz, scores);
    g2.heads_layout = true, g2.a_view = qv, g2.b_view = qv;
    g2.scale = 1.0f / std::sqrt(static_cast<float>(d));
    g2.causal = true;
    g2.skip_upper = true;  // never read: the softmax stops at the diagonal
    e = gemm(&ms, "attn_scores", tpmlp::EPI_ATTN_SCORE, g2, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    {
        Timed timed("attn_softmax", st);
        // With TPMLP_ATTN_P_UPPER_ZERO the 256 x 256 tiles of P wholly above the
        // diagonal (never read: P V and dS K stop at the tile's keys, P^T dO starts
        // at its queries, dS skips them) already hold zeros and are not written.
        const int64_t wtile = (s->flags & TPMLP_ATTN_P_UPPER_ZERO) ? 256 : 0;
        e = tpmlp::launch_softmax(scores, saved->P, nz * S, S, true, wtile, st);
        if (e != cudaSuccess) return from_cuda(e);
        g_launches.fetch_add(1);
    }

    // O_head = P V, V read in place in QKV, O_head written in place in O[T,h].
    GemmArgs g3 = head_gemm(status, saved->P, false, Vp, true, S, d, S, nz, saved->O);
    g3.causal_k = 1;  // P is zero past each row's last key
    g3.heads_layout = true, g3.b_view = qv, g3.o_view = tv;
    e = gemm(&ms, "attn_pv", tpmlp::EPI_STORE, g3, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // Row-parallel output projection: shard partials O_i Wo_i folded in order, + bo.
    GemmArgs g4 = base_args(status);
    g4.a = saved->O, g4.a_mn = false;  // O[T,h]: K-major
    g4.b = Wo, g4.b_mn = true;         // Wo[h,h]: MN-major
    g4.M = T, g4.N = h, g4.K = h;
    g4.nshards = s->t, g4.kshard = h / s->t;
    g4.out0 = Z, g4.bias = bo;
    pick_raster(g4);
    e = gemm(&ms, "attn_out_proj_fold", tpmlp::EPI_FOLD_BIAS, g4, sms, st);
    return from_cuda(e);
}

tpmlp_status tpmlp_attn_backward(const tpmlp_attn_shape *s, const void *dZ, const tpmlp_attn_saved *saved,
                                 void *dX, void *dWqkv, void *dbqkv, void *dWo, void *dbo, void *workspace,
                                 void *stream) {
    tpmlp::g_last_error[0] = '\0';
    if (!saved) return invalid("tpmlp_attn_backward: saved is NULL");
    tpmlp_status rc = attn_check(s, "tpmlp_attn_backward", {saved->Wqkv, saved->Wo, dWqkv, dbqkv, dWo, dbo},
                                 {dZ, saved->X, saved->QKV, saved->P, saved->O, dX}, workspace);
    if (rc != TPMLP_OK) return rc;
    const int64_t T = s->batch * s->seq, h = s->hidden, S = s->seq, d = h / s->heads;
    const int64_t nz = s->batch * s->heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // Empty batch: the weight and bias gradients are sums over no tokens.
        cudaError_t e = cudaMemsetAsync(dWqkv, 0, static_cast<size_t>(h) * 3 * h * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dbqkv, 0, static_cast<size_t>(3 * h) * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dWo, 0, static_cast<size_t>(h) * h * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dbo, 0, static_cast<size_t>(h) * 2, st);
        return from_cuda(e);
    }
    const int sms = num_sms_current();
    if (sms == 0) return TPMLP_ERR_CUDA;
    if (sms < 0) return TPMLP_ERR_DEVICE;
    const tpmlp_shape ms = attn_route(s);
    const AttnLayout L = attn_layout(s);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);
    float *D = reinterpret_cast<float *>(ws + L.D);
    void *dO = ws + L.dO, *dQKV = ws + L.dQKV;
    // Per-head Q, K, V (in the saved QKV), dO (in dO[T,h]) and dQ, dK, dV (in
    // dQKV) are addressed in place through rank-5 and rank-4 views.
    const tpmlp::HeadView qv = qkv_view(s), tv = tok_view(s);
    const void *Qp = qkv_part(saved->QKV, s, 0), *Kp = qkv_part(saved->QKV, s, 1), *Vp = qkv_part(saved->QKV, s, 2);
    void *dQp = const_cast<void *>(qkv_part(dQKV, s, 0)), *dKp = const_cast<void *>(qkv_part(dQKV, s, 1)),
         *dVp = const_cast<void *>(qkv_part(dQKV, s, 2));
    void *dS = ws + L.scores;  // bf16 [nz][S][S] over the dead fp16 scores
    const float scale = 1.0f / std::sqrt(static_cast<float>(d));

    // dbo = 1^T dZ and dbqkv = 1^T dQKV come from the ones tiles of the dWo and
    // dWqkv GEMMs; the row-dot pass, which runs before both, fills the ones.
    void *ones = ws + L.ones;
    cudaError_t e;

    // dO = dZ Wo^T (every shard's columns at once; no fold needed)
    GemmArgs g1 = base_args(status);
    g1.a = dZ, g1.a_mn = false;         // dZ[T,h]: K-major
    g1.b = saved->Wo, g1.b_mn = false;  // Wo[h,h] as [N, K]: K-major
    g1.M = T, g1.N = h, g1.K = h, g1.kshard = h;
    g1.out0 = dO;
    pick_raster(g1, tpmlp::EPI_STORE);
    e = gemm(&ms, "attn_bwd_dO", tpmlp::EPI_STORE, g1, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // D = rowsum(dO * O) per head (and the block of ones)
    {
        Timed timed("attn_bwd_rowdot", st);
        e = tpmlp::launch_rowdot(head_layout(s), dO, saved->O, D, st, ones);
        if (e != cudaSuccess) return from_cuda(e);
        g_launches.fetch_add(1);
    }

    // dWo = O^T dZ
    GemmArgs g2 = base_args(status);
    g2.a = saved->O, g2.a_mn = true;  // O[T,h] as [K=T, M=h]: MN-major
    g2.b = dZ, g2.b_mn = true;        // dZ[T,h] as [K=T, N=h]: MN-major
    g2.M = h, g2.N = h, g2.K = T, g2.kshard = T;
    g2.out0 = dWo;
    g2.ones = ones, g2.bias_grad = dbo;
    pick_raster(g2, tpmlp::EPI_STORE);
    e = gemm(&ms, "attn_bwd_dWo", tpmlp::EPI_STORE, g2, sms, st);
    if (e != cudaSuccess) return from_cuda(e);


    // dV_head = P^T dO_head
    GemmArgs g3 = head_gemm(status, saved->P, true, dO, true, S, d, S, nz, dVp);
    g3.causal_k = 2;  // key j only gets gradient from queries i >= j
    g3.heads_layout = true, g3.b_view = tv, g3.o_view = qv;
    e = gemm(&ms, "attn_bwd_dV", tpmlp::EPI_STORE, g3, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dS = P * (dO V^T - D) * scale
    GemmArgs g4 = head_gemm(status, dO, false, Vp, false, S, S, d, nz, dS);
    g4.heads_layout = true, g4.a_view = tv, g4.b_view = qv;
    g4.aux = saved->P;
    g4.rowvec = D;
    g4.scale = scale;
    g4.skip_upper = true;  // dS is zero above the diagonal; dQ and dK below never read those tiles
    e = gemm(&ms, "attn_bwd_dS", tpmlp::EPI_ATTN_DS, g4, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dQ_head = dS K_head,  dK_head = dS^T Q_head
    GemmArgs g5 = head_gemm(status, dS, false, Kp, true, S, d, S, nz, dQp);
    g5.causal_k = 1;
    g5.heads_layout = true, g5.b_view = qv, g5.o_view = qv;
    e = gemm(&ms, "attn_bwd_dQ", tpmlp::EPI_STORE, g5, sms, st);
    if (e != cudaSuccess) return from_cuda(e);
    GemmArgs g6 = head_gemm(status, dS, true, Qp, true, S, d, S, nz, dKp);
    g6.causal_k = 2;
    g6.heads_layout = true, g6.b_view = qv, g6.o_view = qv;
    e = gemm(&ms, "attn_bwd_dK", tpmlp::EPI_STORE, g6, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dWqkv = X^T dQKV
    GemmArgs g7 = base_args(status);
    g7.a = saved->X, g7.a_mn = true;  // X[T,h] as [K=T, M=h]: MN-major
    g7.b = dQKV, g7.b_mn = true;      // dQKV[T,3h] as [K=T, N=3h]: MN-major
    g7.M = h, g7.N = 3 * h, g7.K = T, g7.kshard = T;
    g7.out0 = dWqkv;
    g7.ones = ones, g7.bias_grad = dbqkv;
    pick_raster(g7, tpmlp::EPI_STORE);
    e = gemm(&ms, "attn_bwd_dWqkv", tpmlp::EPI_STORE, g7, sms, st);
    if (e != cudaSuccess) return from_cuda(e);

    // dX = sum_i dQKV_i Wqkv_i^T, shard partials folded in order (the backward all-reduce)
    GemmArgs g8 = base_args(status);
    g8.a = dQKV, g8.a_mn = false;         // dQKV[T,3h]: K-major
    g8.b = saved->Wqkv, g8.b_mn = false;  // Wqkv[h,3h] as [N=h, K=3h]: K-major
    g8.M = T, g8.N = h, g8.K = 3 * h;
    g8.nshards = s->t, g8.kshard = 3 * h / s->t;
    g8.out0 = dX;
    pick_raster(g8);
    e = gemm(&ms, "attn_bwd_dX_shard_fold", tpmlp::EPI_FOLD, g8, sms, st);
    return from_cuda(e);
}

}  // extern "C"

// ---- vocabulary cross entropy -------------------------------------------------------

namespace {

bool xent_valid(const tpmlp_xent_shape *s) {
    if (!s) return false;
    if (s->tokens < 0 || s->hidden <= 0 || s->vocab <= 0 || s->piece < 0) return false;
    if (s->dtype != TPMLP_F32 && s->dtype != TPMLP_BF16) return false;
    if (s->algo != TPMLP_ALGO_DEFAULT && s->algo != TPMLP_ALGO_SIMT) return false;
    if (s->piece % 8 != 0) return false;
    if (s->tokens > (1LL << 30) || s->hidden > (1LL << 30) || s->vocab > (1LL << 30)) return false;
    const int64_t T = s->tokens, h = s->hidden, V = s->vocab;
    return tiles_fit(T, V) && tiles_fit(T, h) && tiles_fit(V + 256, h);
}

// Tensor cores for both types: fp32 operands as the sum of three bf16 matrices each.
bool xent_tc(const tpmlp_xent_shape *s) { return s->algo == TPMLP_ALGO_DEFAULT; }

// Vocabulary rows per piece.  The backward pass holds one piece of dS [T, piece] (and the
// FFMA path its fp32 logits).  Each further piece costs one more addition to the fp32
// dX [T, h], so pieces are as large as 256 MiB allow, equal in size, in whole wide
// tiles (512 columns).
int64_t xent_piece(const tpmlp_xent_shape *s) {
    const int64_t V = s->vocab, T = s->tokens < 1 ? 1 : s->tokens;
    if (s->piece > 0) return s->piece < V ? s->piece : (V + 7) / 8 * 8;
    const int64_t esz = s->dtype == TPMLP_F32 && xent_tc(s) ? 6 : (xent_tc(s) ? 2 : 4);
    int64_t most = (int64_t{256} << 20) / (T * esz) / 512 * 512;
    if (most < 2048) most = 2048;
    const int64_t n = (V + most - 1) / most;
    const int64_t even = ((V + n - 1) / n + 511) / 512 * 512;
    return even < V ? even : (V + 7) / 8 * 8;
}

// How many K ranges a product of M x N outputs is split into, and their length.  An
// output of few tiles leaves most CTA pairs idle (76 of them take 256 x 512 tiles or
// halves of such): S ranges run at once, each into an fp32 matrix of its own, which
// sum_splits adds up.  The model counts waves of half tiles at the rate of a pair's
// share of the tensor rate, and 8 bytes written and read per split output at the copy
// rate.
// Measured: dX of T = 1001, h = 1000, V = 30011 (16 tiles of 256 x 256) 173 us in one range,
// 54 + 8 us split.
// fp32 operands also take each split in `ranges` ranges of at most 512, which the epilogue adds up
// in fp32, however long K is (see xent_stats_tile): T = 2100, h = 8192, V = 2000, dX and dW to 6e-7
// of themselves (the FFMA path 8e-7) in 1010 us, in ranges of 256 3.5e-7 in 1064, of 1024 1.2e-6 in 981.
struct Split {
    int n;
    int64_t len;  // of a split: ranges * range
    int ranges;
    int64_t range;
    void apply(GemmArgs &g) const {
        if (n > 1)
            g.ksplit = n, g.nshards = ranges, g.kshard = range;
        else if (ranges > 1)  // of what there is: the last piece of a vocabulary may be short
            g.nshards = static_cast<int>((g.K + range - 1) / range), g.kshard = range;
    }
};
Split xent_split(int64_t M, int64_t N, int64_t K, bool f32) {
    const double pair_rate = 24e12 / (f32 ? 6 : 1), bytes_rate = 6e12;
    const int64_t halves = (M + 255) / 256 * ((N + 255) / 256), units = 76;
    Split best{1, 0, 1, 0};
    double best_t = 0.0;
    for (int64_t n = 1; n <= (f32 ? 80 : 16); ++n) {
        int64_t len = ((K + n - 1) / n + 63) / 64 * 64;
        if (n > 1 && len < 256) break;
        const int64_t ranges = f32 ? (len + 511) / 512 : 1, range = ((len + ranges - 1) / ranges + 63) / 64 * 64;
        len = ranges * range;
        const double waves = static_cast<double>((halves * n + units - 1) / units);
        const double t = waves * (static_cast<double>(len) * 2 * 256 * 256 / pair_rate + 1e-6) +
                         (n > 1 ? static_cast<double>(n) * M * N * 8 / bytes_rate + 4e-6 : 0.0);
        if (best_t == 0.0 || t < best_t)
            best_t = t, best = {static_cast<int>((K + len - 1) / len), len, static_cast<int>(ranges), range};
    }
    return best;
}

// The forward product's tiles.  512: 256 x 512 with the whole K in one accumulator.
// Otherwise 256 (or 128) x tile_n with K in ranges that the epilogue adds up in fp32: the tensor
// core cuts the accumulator off (towards zero, it does not round) at every step of 16 products,
// which takes 2^-26 of a logit a step with independent terms, and up to 2^-24 a step with all
// terms of one sign.  Relative error of the loss (T = 300 to 8192, V = 2500 to 50000, X
// towards the target's row): 6e-8 in ranges of 256, 1.2e-7 of 512, 2.4 to 3.4e-7 of 1024, 5.0 to
// 5.9e-7 of 2048, 1.0e-6 of 4096, 2.6e-6 of 8192; the plain fp32 form's is 2e-7.
// Wide tiles take a quarter less from L2 per product, which bounds short products at full
// clock (T = 333, h = 2048, V = 50021: 72 us against 81 in ranges of 1024), so that up to 2048
// products go into one accumulation; longer rows go in ranges of 1024 (T = 8192, h = 4096,
// V = 65536: 2.53 ms, ranges of 2048 2.50, one of 4096 on wide tiles 2.39).  Where there are few
// tiles the ranges cost nothing, and narrower tiles divide the vocabulary evenly among the units;
// fp32 operands want the precision and take ranges of 256 always (T = 512, h = 1024, V = 16384:
// 8.4e-8 in 116 us, ranges of 512 1.8e-7 in 107).
// Up to 128 bf16 tokens fill a single CTA's tile: pairs would multiply 128 empty rows, at which
// rate W comes no faster than 6 TB/s (h = 4096, V = 32768: T = 64 62.0 against 54.3 us; T = 100,
// h = 8192: 112 against 98.7; T = 128, h = 1536, V = 50000: 42.6 against 38.6; T = 16, h = 2048,
// V = 50021, unevenly divided: 60.0 against 61.2).  fp32 stays on pairs (T = 20, h = 1024,
// V = 16000: 79 against 96 us), and so do more tokens (T = 256: 64.4 against 74.0 us).
struct StatsTile {
    int tile_n;  // 0: a pass over W without tiles, for few tokens
    int64_t ranges, range;  // of K, in both passes: lse and the recomputed logits come from the same sums
    bool pair;  // on CTA pairs
};
StatsTile xent_stats_tile(const tpmlp_xent_shape *s) {
    const int64_t T = std::max<int64_t>(1, s->tokens), V = s->vocab, h = s->hidden;
    const bool f32 = s->dtype == TPMLP_F32, pair = f32 || T > 128;
    const int64_t units = pair ? 76 : 152, tile_m = pair ? 256 : 128;
    const int64_t m = (T + tile_m - 1) / tile_m, tiles = m * ((V + 255) / 256);
    const bool few = m == 1 || tiles <= 4 * units;
    if (!f32 && !few && h <= 2048) return {512, 1, h, true};
    int64_t tile_n = 256;
    if (few) {  // as many waves as 256-wide tiles need, evenly filled
        const int64_t waves = (tiles + units - 1) / units, per = std::max<int64_t>(1, waves * units / m);
        tile_n = std::min<int64_t>(256, ((V + per - 1) / per + 31) / 32 * 32);
    }
    const int64_t longest = f32 ? 256 : 1024;
    const int64_t ranges = (h + longest - 1) / longest, range = ((h + ranges - 1) / ranges + 63) / 64 * 64;
    if (tpmlp::xent_few(!f32, T, h)) tile_n = 0;
    return {static_cast<int>(tile_n), ranges, range, pair};
}

struct XentLayout {
    int64_t piece, pieces, groups, hp, ldo;
    StatsTile stats;
    Split dx, dw;
    size_t unit, part, target_logit, xp, wp, ds, logits, acc, dwacc, total;
    size_t forward;  // what the forward pass alone uses, from the start
};

// Workspace, 1 KB-aligned regions: status | the unit of dS | statistics | the targets' logits | three bf16
// parts of X and W (fp32) | dS of one piece | fp32 logits of one piece (FFMA path) | fp32
// dX, per split | fp32 dW of one piece, per split.
XentLayout xent_layout(const tpmlp_xent_shape *s) {
    XentLayout L;
    const size_t T = static_cast<size_t>(s->tokens);
    const size_t V = static_cast<size_t>(s->vocab);
    const bool tc = xent_tc(s), f32 = s->dtype == TPMLP_F32;
    L.piece = xent_piece(s);
    L.pieces = (s->vocab + L.piece - 1) / L.piece;
    L.stats = xent_stats_tile(s);
    // stored groups, and those of them that hold columns
    const size_t stored = static_cast<size_t>(!tc                     ? L.pieces
                                              : L.stats.tile_n == 0 ? tpmlp::xent_few_groups(s->vocab)
                                                                    : tpmlp::xent_groups(s->vocab, L.stats.tile_n));
    L.groups = tc && L.stats.tile_n == 512 ? (s->vocab + 127) / 128 : static_cast<int64_t>(stored);
    L.hp = (s->hidden + 63) / 64 * 64;
    L.ldo = (s->hidden + 3) / 4 * 4;
    L.dx = L.dw = {1, 0, 1, 0};
    if (tc && s->tokens > 0) {
        L.dx = xent_split(s->tokens, s->hidden, L.piece, f32);
        L.dw = xent_split(L.piece, s->hidden, s->tokens, f32);
    }
    size_t off = STATUS_BYTES;
    auto region = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 1024);
        return at;
    };
    const size_t piece = static_cast<size_t>(L.piece), hp = static_cast<size_t>(L.hp), ldo = static_cast<size_t>(L.ldo);
    L.unit = region(sizeof(float));
    L.part = region(stored * T * sizeof(float2));
    L.target_logit = region(T * 4);
    L.forward = off;  // the statistics alone: bf16, and few tokens of either type
    L.xp = region(tc && f32 ? 3 * T * hp * 2 : 0);
    L.wp = region(tc && f32 ? 3 * V * hp * 2 : 0);
    if (tc && f32 && L.stats.tile_n != 0) L.forward = off;
    L.ds = region(T * piece * (tc ? (f32 ? 6 : 2) : (f32 ? 4 : 2)));
    // FFMA path: in fp32 dS takes the place of the logits
    L.logits = tc || f32 ? L.ds : region(T * piece * 4);
    if (!tc) L.forward = off;
    // dX and dW pass through fp32 where they are summed, or (fp32) cannot be stored by TMA
    const bool odd = f32 && s->hidden % 4 != 0;
    const bool dx_direct = tc ? L.dx.n == 1 && (f32 ? !odd : L.pieces == 1) : f32 || L.pieces == 1;
    L.acc = region(dx_direct && !f32 ? 0 : static_cast<size_t>(L.dx.n) * T * ldo * 4);
    L.dwacc = region(tc && (L.dw.n > 1 || f32) ? static_cast<size_t>(L.dw.n) * piece * ldo * 4 : 0);
    L.total = off;
    return L;
}

tpmlp_status xent_check(const tpmlp_xent_shape *s, const char *who, std::initializer_list<const void *> token_ptrs,
                        std::initializer_list<const void *> matrices, std::initializer_list<const void *> rows,
                        const void *workspace) {
    if (!xent_valid(s)) {
        tpmlp::set_last_error("%s: invalid shape", who);
        return TPMLP_ERR_INVALID_ARG;
    }
    bool null = !workspace;
    for (const void *p : token_ptrs) null = null || (!p && s->tokens > 0);
    for (const void *p : rows) null = null || (!p && s->tokens > 0);
    if (null) {
        tpmlp::set_last_error("%s: NULL pointer", who);
        return TPMLP_ERR_INVALID_ARG;
    }
    // bf16: TMA bases and row pitches on 16 bytes; fp32: elements
    const size_t al = s->dtype == TPMLP_BF16 ? 16 : 4;
    bool bad = !aligned16(workspace) || (s->dtype == TPMLP_BF16 && s->hidden % 8 != 0);
    for (const void *p : matrices) bad = bad || (p && !aligned_elt(p, al));
    for (const void *p : rows) bad = bad || (p && !aligned_elt(p, 4));
    if (bad) {
        tpmlp::set_last_error("%s: bf16 needs h a multiple of 8 and 16-byte aligned matrices, the workspace 16 bytes",
                              who);
        return TPMLP_ERR_UNSUPPORTED;
    }
    if (s->algo == TPMLP_ALGO_SIMT && (s->tokens > 65535LL * 64 || s->vocab > 65535LL * 64)) {
        tpmlp::set_last_error("%s: the FFMA path takes at most 65535 * 64 tokens and vocabulary rows", who);
        return TPMLP_ERR_UNSUPPORTED;
    }
    return TPMLP_OK;
}

struct Buffer {
    const void *p;
    int64_t bytes;
};
// Whether an output's bytes are also an input's, or another output's.
bool outputs_overlap(std::initializer_list<Buffer> outputs, std::initializer_list<Buffer> inputs) {
    const auto shared = [](const Buffer &x, const Buffer &y) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
        return a && b && a < b + static_cast<uintptr_t>(y.bytes) && b < a + static_cast<uintptr_t>(x.bytes);
    };
    for (const Buffer *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Buffer &i : inputs)
            if (shared(*o, i)) return true;
        for (const Buffer *q = o + 1; q != outputs.end(); ++q)
            if (shared(*o, *q)) return true;
    }
    return false;
}

// SMs of the current device, or the error to return.
tpmlp_status device_ready(int &sms) {
    sms = num_sms_current();
    return sms == 0 ? TPMLP_ERR_CUDA : (sms < 0 ? TPMLP_ERR_DEVICE : TPMLP_OK);
}

struct XentCall {
    const tpmlp_xent_shape *s;
    XentLayout L;
    uint8_t *ws;
    int sms;
    cudaStream_t st;
    tpmlp::RowArgs rows;
    XentCall(const tpmlp_xent_shape *s_, const int64_t *target, void *workspace, int sms_, void *stream)
        : s(s_), L(xent_layout(s_)), ws(static_cast<uint8_t *>(workspace)), sms(sms_),
          st(static_cast<cudaStream_t>(stream)) {
        rows.tokens = s->tokens, rows.vocab = s->vocab, rows.ignore_index = s->ignore_index;
        rows.target = target;
        rows.part = reinterpret_cast<float2 *>(ws + L.part);
        rows.groups = L.groups;
        rows.target_logit = reinterpret_cast<float *>(ws + L.target_logit);
        rows.status = reinterpret_cast<uint32_t *>(ws);
    }
    size_t esz() const { return s->dtype == TPMLP_BF16 ? 2 : 4; }
    // fp32 on tensor cores: the three bf16 parts of X [3][T][hp] and W [3][V][hp].
    bool parts() const { return xent_tc(s) && s->dtype == TPMLP_F32; }
    const uint16_t *xp() const { return reinterpret_cast<const uint16_t *>(ws + L.xp); }
    const uint16_t *wp(int64_t v0) const { return reinterpret_cast<const uint16_t *>(ws + L.wp) + v0 * L.hp; }
    static void set_parts(GemmArgs &g, int64_t a_part, int64_t b_part) {
        g.parts = 3, g.a_part = a_part, g.b_part = b_part;
    }
    cudaError_t split_operands(const void *X, const void *W) const {
        if (!parts()) return cudaSuccess;
        const tpmlp::Split3 x = {static_cast<const float *>(X), s->tokens, s->hidden, L.hp, ws + L.xp};
        const tpmlp::Split3 w = {static_cast<const float *>(W), s->vocab, s->hidden, L.hp, ws + L.wp};
        return kernel("xent_split", [&] { return tpmlp::launch_split3(x, w, st); });
    }
    const void *w_rows(const void *W, int64_t v0) const {
        return static_cast<const uint8_t *>(W) + static_cast<size_t>(v0) * s->hidden * esz();
    }
    // X W_p^T over vocabulary rows v0 .. v0 + n - 1.
    GemmArgs logits(const void *X, const void *W, int64_t v0, int64_t n) const {
        GemmArgs g = base_args(rows.status);
        g.a = X, g.a_mn = false;
        g.b = w_rows(W, v0), g.b_mn = false;
        g.M = s->tokens, g.N = n, g.K = s->hidden;
        g.nshards = xent_tc(s) ? static_cast<int>(L.stats.ranges) : 1;
        g.kshard = xent_tc(s) ? L.stats.range : s->hidden;
        if (parts()) {
            g.a = xp(), g.lda = L.hp;
            g.b = wp(v0), g.ldb = L.hp;
            set_parts(g, s->tokens * L.hp, s->vocab * L.hp);
        }
        g.target = rows.target, g.ignore_index = s->ignore_index, g.col0 = v0;
        return g;
    }
    cudaError_t launch(const char *name, Epi epi, GemmArgs &g) const {
        const bool tc = xent_tc(s);
        // Products of no more 128 x 128 tiles than there are SMs are bound by latency (T = 95, h = 840,
        // V = 81: a step 35 against 31 us); with two waves of them the operands' bytes
        // count again (T = 1001, h = 1000, V = 30011, dX: 90 against 55 us).
        g.small_tile = epi != tpmlp::EPI_XENT_STATS && epi != tpmlp::EPI_XENT_FOLD &&
                       (g.M + 127) / 128 * ((g.N + 127) / 128) * std::max(1, g.ksplit) <= 152;
        if (g.small_tile) g.cta_pair = false;
        if (tc) pick_raster(g, epi);
        Timed timed(name, st);
        const cudaError_t e = tc ? tpmlp::launch_tc_gemm(epi, g, sms, st)
                                 : tpmlp::launch_simt_gemm(epi, s->dtype == TPMLP_BF16, g, st);
        if (e == cudaSuccess) g_launches.fetch_add(1);
        return e;
    }
    template <typename F>
    cudaError_t kernel(const char *name, F f) const {
        Timed timed(name, st);
        const cudaError_t e = f();
        if (e == cudaSuccess) g_launches.fetch_add(1);
        return e;
    }
};

}  // namespace

extern "C" {

size_t tpmlp_xent_workspace_bytes(const tpmlp_xent_shape *s) { return xent_valid(s) ? xent_layout(s).total : 0; }

size_t tpmlp_xent_forward_workspace_bytes(const tpmlp_xent_shape *s) {
    return xent_valid(s) ? xent_layout(s).forward : 0;
}

tpmlp_status tpmlp_xent_forward(const tpmlp_xent_shape *s, const void *X, const void *W, const int64_t *target,
                                float *loss, float *lse, void *workspace, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    tpmlp_status rc = xent_check(s, "tpmlp_xent_forward", {X}, {X, W}, {loss, lse}, workspace);
    if (rc != TPMLP_OK) return rc;
    if (!W || (!target && s->tokens > 0)) return invalid("tpmlp_xent_forward: NULL pointer");
    if (!aligned_elt(target, 8)) return TPMLP_ERR_UNSUPPORTED;
    if (s->tokens == 0) return TPMLP_OK;
    const int64_t T = s->tokens, esz = s->dtype == TPMLP_BF16 ? 2 : 4;
    if (outputs_overlap({{loss, 4 * T}, {lse, 4 * T}},
                        {{X, T * s->hidden * esz}, {W, s->vocab * s->hidden * esz}, {target, 8 * T}}))
        return invalid("tpmlp_xent_forward: an output overlaps an input or the other output");
    int sms;
    if ((rc = device_ready(sms)) != TPMLP_OK) return rc;
    const XentCall c(s, target, workspace, sms, stream);
    cudaError_t e = cudaSuccess;
    if (xent_tc(s) && c.L.stats.tile_n == 0) {
        float2 *part = reinterpret_cast<float2 *>(c.ws + c.L.part);
        e = c.kernel("xent_few", [&] {
            return tpmlp::launch_xent_few(s->dtype == TPMLP_BF16, c.rows, X, W, s->hidden, part, loss, lse, c.st);
        });
        return from_cuda(e);
    } else if (xent_tc(s)) {
        e = c.split_operands(X, W);
        if (e != cudaSuccess) return from_cuda(e);
        GemmArgs g = c.logits(X, W, 0, s->vocab);
        g.part = reinterpret_cast<float2 *>(c.ws + c.L.part);
        g.target_logit = c.rows.target_logit;
        const StatsTile &t = c.L.stats;
        if (t.tile_n < 512) g.tile_n = t.tile_n, g.cta_pair = t.pair;
        e = c.launch("xent_stats", t.tile_n < 512 ? tpmlp::EPI_XENT_FOLD : tpmlp::EPI_XENT_STATS, g);
        if (e != cudaSuccess) return from_cuda(e);
    } else {
        float *logits = reinterpret_cast<float *>(c.ws + c.L.logits);
        for (int64_t k = 0; k < c.L.pieces; ++k) {
            const int64_t v0 = k * c.L.piece, n = std::min(c.L.piece, s->vocab - v0);
            GemmArgs g = c.logits(X, W, v0, n);
            g.out0 = logits;
            e = c.launch("xent_logits", tpmlp::EPI_ACC32, g);
            if (e != cudaSuccess) return from_cuda(e);
            float2 *part = reinterpret_cast<float2 *>(c.ws + c.L.part) + k * s->tokens;
            e = c.kernel("xent_piece_stats",
                         [&] { return tpmlp::launch_xent_piece_stats(c.rows, logits, n, v0, part, c.st); });
            if (e != cudaSuccess) return from_cuda(e);
        }
    }
    return from_cuda(c.kernel("xent_combine", [&] { return tpmlp::launch_xent_combine(c.rows, loss, lse, c.st); }));
}

tpmlp_status tpmlp_xent_backward(const tpmlp_xent_shape *s, const void *X, const void *W, const int64_t *target,
                                 const float *lse, const float *dloss, void *dX, void *dW, void *workspace,
                                 void *stream) {
    tpmlp::g_last_error[0] = '\0';
    tpmlp_status rc = xent_check(s, "tpmlp_xent_backward", {X}, {X, W, dX, dW}, {lse, dloss}, workspace);
    if (rc != TPMLP_OK) return rc;
    if (!W || (!target && s->tokens > 0)) return invalid("tpmlp_xent_backward: NULL pointer");
    if (!aligned_elt(target, 8)) return TPMLP_ERR_UNSUPPORTED;
    const int64_t T = s->tokens, h = s->hidden, esz = s->dtype == TPMLP_BF16 ? 2 : 4;
    if (T > 0 && outputs_overlap({{dX, T * h * esz}, {dW, s->vocab * h * esz}},
                                 {{X, T * h * esz}, {W, s->vocab * h * esz}, {target, 8 * T}, {lse, 4 * T}, {dloss, 4 * T}}))
        return invalid("tpmlp_xent_backward: an output overlaps an input or the other output");
    if (!dX && !dW) return TPMLP_OK;
    int sms;
    if ((rc = device_ready(sms)) != TPMLP_OK) return rc;
    cudaError_t e;
    if (s->tokens == 0) {
        if (!dW) return TPMLP_OK;
        return from_cuda(cudaMemsetAsync(dW, 0, static_cast<size_t>(s->vocab * h * esz), static_cast<cudaStream_t>(stream)));
    }
    const XentCall c(s, target, workspace, sms, stream);
    const bool tc = xent_tc(s), f32 = s->dtype == TPMLP_F32;
    if ((e = c.split_operands(X, W)) != cudaSuccess) return from_cuda(e);
    uint8_t *ds = c.ws + c.L.ds;
    // dX is summed over the pieces (and the splits of each) in fp32: in place for fp32,
    // in the workspace for bf16, and not at all when one piece and one range hold it all.
    const bool stores = !f32 || (h % 4 == 0 && aligned16(dX));  // fp32 rows that TMA can store
    const bool one = !f32 && c.L.pieces == 1 && c.L.dx.n == 1;
    const bool dx_in_place = tc ? (f32 ? c.L.dx.n == 1 && stores : one) : f32 || c.L.pieces == 1;
    float *acc = reinterpret_cast<float *>(c.ws + c.L.acc), *unit = reinterpret_cast<float *>(c.ws + c.L.unit);
    for (int64_t k = 0; k < c.L.pieces; ++k) {
        const int64_t v0 = k * c.L.piece, n = std::min(c.L.piece, s->vocab - v0);
        GemmArgs g = c.logits(X, W, v0, n);
        const int64_t ld = tc ? c.L.piece : n;  // row pitch of dS, and between its parts
        const int64_t ds_part = T * ld;
        if (tc && c.L.stats.tile_n == 0) {  // few tokens: the logits of the forward pass's kernel
            tpmlp::RowArgs rows = c.rows;
            rows.vocab = n;
            const tpmlp::FewGrad d = {lse, dloss, unit, ds, ld, ds_part, v0, s->vocab};
            e = c.kernel("xent_few_ds", [&] {
                return tpmlp::launch_xent_few_grad(!f32, rows, X, c.w_rows(W, v0), h, d, c.st);
            });
        } else if (tc) {
            g.out0 = ds, g.ldo = ld;
            g.row_lse = lse, g.dloss = dloss, g.vocab = s->vocab, g.unit = unit;
            e = c.launch("xent_ds", f32 ? tpmlp::EPI_XENT_GRAD3 : tpmlp::EPI_XENT_GRAD, g);
        } else {
            float *logits = reinterpret_cast<float *>(c.ws + c.L.logits);
            g.out0 = logits;
            e = c.launch("xent_logits", tpmlp::EPI_ACC32, g);
            if (e == cudaSuccess)
                e = c.kernel("xent_piece_grad", [&] {
                    return tpmlp::launch_xent_piece_grad(!f32, c.rows, logits, n, v0, lse, dloss, ds, c.st);
                });
        }
        if (e != cudaSuccess) return from_cuda(e);
        if (dW) {  // rows v0 .. of dW = dS_p^T X
            void *out = const_cast<void *>(c.w_rows(dW, v0));
            GemmArgs w = base_args(c.rows.status);
            w.a = ds, w.a_mn = true, w.lda = ld;
            w.b = X, w.b_mn = true;
            w.M = n, w.N = h, w.K = T, w.kshard = T;
            w.out0 = out;
            bool in_place = true;
            if (tc) {
                in_place = c.L.dw.n == 1 && (!f32 || (h % 4 == 0 && aligned16(out)));
                c.L.dw.apply(w);
                if (!in_place) w.out0 = c.ws + c.L.dwacc, w.ldo = c.L.ldo;
                if (f32) {
                    w.b = c.xp(), w.ldb = c.L.hp;
                    XentCall::set_parts(w, ds_part, T * c.L.hp);
                }
            }
            w.unit = unit;
            e = c.launch("xent_dw", !tc         ? tpmlp::EPI_STORE
                                    : f32       ? tpmlp::EPI_FOLD32
                                    : !in_place ? tpmlp::EPI_ACC32
                                                : tpmlp::EPI_STORE_UNIT, w);
            if (e == cudaSuccess && !in_place)
                e = c.kernel("xent_dw_sum", [&] {
                    return tpmlp::launch_sum_splits(!f32, reinterpret_cast<float *>(c.ws + c.L.dwacc), c.L.dw.n, n, h,
                                                    c.L.ldo, f32 ? nullptr : unit, out, c.st);
                });
            if (e != cudaSuccess) return from_cuda(e);
        }
        if (dX) {  // dX (+)= dS_p W_p
            GemmArgs x = base_args(c.rows.status);
            x.a = ds, x.a_mn = false, x.lda = ld;
            x.b = c.w_rows(W, v0), x.b_mn = true;
            x.M = T, x.N = h, x.K = n, x.kshard = n;
            x.out0 = dx_in_place ? dX : static_cast<void *>(acc);
            x.accumulate = k > 0;
            if (tc) {
                c.L.dx.apply(x);
                if (!dx_in_place) x.ldo = c.L.ldo;
                if (f32) {
                    x.b = c.wp(v0), x.ldb = c.L.hp;
                    XentCall::set_parts(x, ds_part, s->vocab * c.L.hp);
                }
            }
            const bool rounds = dx_in_place && !f32;  // one product gives the bf16 result
            x.unit = unit;
            e = c.launch("xent_dx", tc && f32 ? tpmlp::EPI_FOLD32
                                    : !rounds ? tpmlp::EPI_ACC32
                                              : (tc ? tpmlp::EPI_STORE_UNIT : tpmlp::EPI_STORE), x);
            if (e != cudaSuccess) return from_cuda(e);
        }
    }
    if (dX && !dx_in_place)
        e = c.kernel("xent_dx_sum", [&] {
            return tpmlp::launch_sum_splits(!f32, acc, tc ? c.L.dx.n : 1, T, h, tc ? c.L.ldo : h,
                                            tc && !f32 ? unit : nullptr, dX, c.st);
        });
    return from_cuda(e);
}

}  // extern "C"

// ---- Newton-Schulz orthogonalisation ------------------------------------------------

namespace {

// Powers of two that the fp16 iterates are stored with, so that both their largest
// values (|X| < 2, |A| < 3.6, |C| < 7.5, see ortho_range_ok) and the small entries of
// a large matrix's first step (about 1/(p sqrt(p)) off A's diagonal) are normal
// fp16 numbers.
constexpr float kScaleX = 8192.0f, kScaleA = 16384.0f, kScaleC = 8192.0f;

// X' = aX + CX with C = bA + cA^2 is computed as (a - d) X + (C + dI) X: near the end A is
// close to I and C to (b + c) I, about -2.7, so that d = 2 leaves C + dI small and its
// rounding with it.  d is the power of two next to a/2.
float ortho_shift(float a) { return a > 0.0f ? std::exp2(std::round(std::log2(0.5f * a))) : 0.0f; }

// Follows the largest singular value through the steps: starting from the interval
// [0, 1] (the Frobenius norm bounds it), the image of [0, r] under x -> x f(x^2), f(l) =
// a + b l + c l^2; every iterate must stay inside the fp16 scales above.  Extremes lie
// at the ends and where a derivative vanishes.
// q_bound: a bound of the product of the steps' factors f(l).
bool ortho_range_ok(const tpmlp_ortho_shape *s, double &q_bound) {
    const double a = s->a, b = s->b, c = s->c, d = ortho_shift(s->a);
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    if (std::fabs(a - d) > 64.0) return false;
    const auto f = [&](double l) { return a + b * l + c * l * l; };
    const double disc = 9.0 * b * b - 20.0 * a * c;  // (x f(x^2))' = a + 3 b l + 5 c l^2
    const double root = disc > 0.0 ? std::sqrt(disc) : 0.0;
    const double at[3] = {c != 0.0 ? (-3.0 * b + root) / (10.0 * c) : (b != 0.0 ? -a / (3.0 * b) : -1.0),
                          c != 0.0 ? (-3.0 * b - root) / (10.0 * c) : -1.0, c != 0.0 ? -b / (2.0 * c) : -1.0};
    double r = 1.0;
    q_bound = 1.0;
    for (int k = 0; k < s->steps; ++k) {
        double next = 0.0, factor = 0.0;
        const auto see = [&](double l) {
            factor = std::max(factor, std::max(std::fabs(f(l)), std::fabs(f(l) - (a - d))));
            next = std::max(next, std::sqrt(l) * std::fabs(f(l)));
        };
        see(0.0);
        see(r * r);
        for (double l : at)
            if (l > 0.0 && l < r * r) see(l);
        if (!(factor <= 7.5)) return false;
        q_bound *= factor * 1.01;
        r = next * 1.01;  // rounding
        if (!(r <= 1.9)) return false;
    }
    return true;
}

bool ortho_valid(const tpmlp_ortho_shape *s) {
    if (!s) return false;
    if (s->batch < 0 || s->batch > 65535 || s->rows <= 0 || s->cols <= 0) return false;
    if (s->rows > (1LL << 20) || s->cols > (1LL << 20)) return false;
    if (s->steps < 1 || s->steps > 32) return false;
    if (s->dtype != TPMLP_F32 && s->dtype != TPMLP_BF16) return false;
    if (!(s->eps >= 0.0f) || !std::isfinite(s->eps)) return false;
    // 32-bit counts of 16-byte pieces
    if ((s->rows + 64) * (s->cols + 64) >= (1LL << 34)) return false;
    return tiles_fit(s->rows + 64, s->cols + 64, s->batch);
}

// K elements per accumulation of the Gram product that the chain starts from.  The tensor
// core cuts its accumulator off at every step of 16 (three times for two parts): a relative
// error of A_0 of about 2^-25 per step, which counts against the smallest eigenvalue's share
// of the largest.  With 1024 at once, matrices with one singular value 200 times the others
// came out with errors of 5e-3 to 8e-3; the ranges' sums are added in fp32.
int64_t gram_range(const tpmlp_ortho_shape *s) { return s->dtype == TPMLP_F32 ? 128 : 256; }

struct OrthoLayout {
    int64_t P, Q, p;
    bool wide;   // rows <= cols: A = X X^T, else A = X^T X
    bool chain;  // the steps on the Gram matrix alone (ns_chain.cu)
    int splits;  // K ranges of the Gram product, and their length
    int64_t split_len;
    float q_scale;
    size_t norm, hi[2], lo[2], rest, gram, A, C, total;
};

// Workspace, 1 KB-aligned regions: status | block sums of the norm | X's high and low parts
// (without the chain two of each, used in turn; with it only once, and a padded output
// where TMA cannot store the unpadded one) | A | C (chain: the splits' A in fp32 | Q).
OrthoLayout ortho_layout(const tpmlp_ortho_shape *s) {
    OrthoLayout L;
    L.P = (s->rows + 63) / 64 * 64, L.Q = (s->cols + 63) / 64 * 64;
    L.wide = s->rows <= s->cols;
    L.p = L.wide ? L.P : L.Q;
    // The chain holds A_0 to about 2^-23 of its largest eigenvalue, and the steps multiply what they
    // do to the small ones by up to Q^2: errors (on matrices with some strong directions) of 3e-9 Q^2,
    // 2e-3 in all up to Q = 485 (five steps of the usual coefficients), 3e-3 at 535, 4e-3 to 9e-3 at
    // 1670 (six), 5e-2 at 5753.  Steps on X itself do not lose that (2e-3 to 4e-3 at 12 steps).
    double q_bound = 0.0;
    L.chain = L.p <= tpmlp::NS_CHAIN_P && ortho_range_ok(s, q_bound) && q_bound <= 600.0;
    L.q_scale = L.chain ? static_cast<float>(std::exp2(std::floor(std::log2(30000.0 / std::max(q_bound, 1.0))))) : 1.0f;
    size_t off = STATUS_BYTES;
    auto region = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 1024);
        return at;
    };
    const size_t n = static_cast<size_t>(s->batch);
    L.norm = region(n * static_cast<size_t>(tpmlp::ortho_norm_blocks(s->batch, s->rows * s->cols)) * 12);
    const size_t x = n * static_cast<size_t>(L.P) * L.Q * 2, a = n * static_cast<size_t>(L.p) * L.p * 2;
    if (L.chain) {
        // one tile per matrix: split K until the SMs have one each, 256 or more at a time
        const int64_t K = L.wide ? L.Q : L.P, range = gram_range(s);
        const int64_t want = std::min<int64_t>(152 / std::max<int64_t>(1, s->batch), (K + 255) / 256);
        L.split_len = (K / std::max<int64_t>(1, want) + range - 1) / range * range;
        L.splits = static_cast<int>((K + L.split_len - 1) / L.split_len);
        const bool f32 = s->dtype == TPMLP_F32;  // bf16 values need no low part (see OrthoStart::rest)
        L.hi[0] = region(f32 ? 2 * x : x);
        L.lo[0] = f32 ? L.hi[0] + x : 0;
        L.rest = region(n * 4);
        L.hi[1] = region(s->cols % 8 ? x : 0);
        L.lo[1] = 0;
        L.A = region(2 * a * static_cast<size_t>(L.splits));
        L.C = region(2 * a);
    } else {
        // A long K over few tiles: K ranges of 512 or more on the idle SMs, added up by a launch of
        // their own (about 6 us against 0.3 us per 64 of K; 700 x 8000: A 42 us at 21 tiles).
        const int64_t K = L.wide ? L.Q : L.P, t = (L.p + 127) / 128, tiles = t * (t + 1) / 2 * s->batch;
        const int64_t want = std::min<int64_t>(152 / std::max<int64_t>(1, tiles), K / 512);
        L.splits = 1, L.split_len = K;
        if (want > 1 && K - K / want >= 2048) {
            L.split_len = (K / want + 63) / 64 * 64;
            L.splits = static_cast<int>((K + L.split_len - 1) / L.split_len);
        }
        L.gram = region(L.splits > 1 ? 2 * a * static_cast<size_t>(L.splits) : 0);
        for (int i = 0; i < 2; ++i) L.hi[i] = region(x), L.lo[i] = region(x);
        L.A = region(a);
        L.C = region(a);
    }
    L.total = off;
    return L;
}

}  // namespace

extern "C" {

size_t tpmlp_ortho_workspace_bytes(const tpmlp_ortho_shape *s) {
    return ortho_valid(s) && s->batch >= 0 ? ortho_layout(s).total : 0;
}

tpmlp_status tpmlp_orthogonalize(const tpmlp_ortho_shape *s, const void *G, void *O, void *workspace, void *stream) {
    tpmlp::g_last_error[0] = '\0';
    if (!ortho_valid(s)) return invalid("tpmlp_orthogonalize: invalid shape");
    if (!workspace || (s->batch > 0 && (!G || !O))) return invalid("tpmlp_orthogonalize: NULL pointer");
    const size_t e_in = s->dtype == TPMLP_BF16 ? 2 : 4;
    // whole rows of 16 bytes are stored by TMA, which wants the base on 16 bytes too
    const bool tma_out = s->cols % 8 == 0;
    if (!aligned16(workspace) || !aligned_elt(G, e_in) || !aligned_elt(O, tma_out ? 16 : 2)) {
        tpmlp::set_last_error("tpmlp_orthogonalize: misaligned pointer (workspace 16 bytes, O 16 where cols is a "
                              "multiple of 8, else 2)");
        return TPMLP_ERR_UNSUPPORTED;
    }
    double q_bound;
    if (!ortho_range_ok(s, q_bound)) {
        tpmlp::set_last_error("tpmlp_orthogonalize: the coefficients let the iterates leave the fp16 range");
        return TPMLP_ERR_UNSUPPORTED;
    }
    if (s->batch == 0) return TPMLP_OK;
    int sms;
    const tpmlp_status rc = device_ready(sms);
    if (rc != TPMLP_OK) return rc;
    const OrthoLayout L = ortho_layout(s);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);

    tpmlp::OrthoStart a;
    a.G = G;
    a.batch = s->batch, a.rows = s->rows, a.cols = s->cols, a.P = L.P, a.Q = L.Q;
    a.eps = s->eps, a.scale = kScaleX;
    a.part = ws + L.norm;
    a.hi = ws + L.hi[0], a.lo = ws + L.lo[0];
    a.lo_scale = L.chain ? 1.0f : 2048.0f;
    a.rest = nullptr;
    const bool single = L.chain && s->dtype == TPMLP_BF16;
    if (L.chain) a.rest = reinterpret_cast<float *>(ws + L.rest);
    if (single) a.lo = nullptr;
    auto timed_launch = [&](const char *name, auto f) {
        Timed timed(name, st);
        const cudaError_t r = f();
        if (r == cudaSuccess) g_launches.fetch_add(1);
        return r;
    };
    const bool bf16 = s->dtype == TPMLP_BF16;
    cudaError_t e = timed_launch("ortho_norm", [&] { return tpmlp::launch_ortho_norm(bf16, a, st); });
    if (e != cudaSuccess) return from_cuda(e);
    e = timed_launch("ortho_scale", [&] { return tpmlp::launch_ortho_scale(bf16, a, st); });
    if (e != cudaSuccess) return from_cuda(e);

    auto product = [&](const void *x, bool x_mn, const void *y, bool y_mn, int64_t M,
                       int64_t N, int64_t K, void *out) {
        GemmArgs g = base_args(status);
        g.a = x, g.a_mn = x_mn;
        g.b = y, g.b_mn = y_mn;
        g.M = M, g.N = N, g.K = K, g.kshard = K;
        g.batch = s->batch;
        g.out0 = out;
        return g;
    };
    auto launch = [&](const char *name, Epi epi, GemmArgs &g) {
        // Products of few tiles are bound by their latency, which 128 x 128 tiles on single CTAs
        // keep shorter than 256 x 256 tiles on CTA pairs, up to about two waves of them
        // (256 x 1024: 148 against 109 us, 700 x 8000: 393 against 365 us, six of 515 x 1003: 204
        // against 183 us; 4096 x 4096, beyond it, the same with either).
        const int64_t mt = (g.M + 127) / 128, nt = (g.N + 127) / 128;
        const bool sym = epi == tpmlp::EPI_NS_GRAM || epi == tpmlp::EPI_NS_POLY;
        g.cta_pair = (sym ? mt * (mt + 1) / 2 : mt * nt) * s->batch > 400;
        pick_raster(g, epi);
        return timed_launch(name, [&] { return tpmlp::launch_tc_gemm(epi, g, sms, st); });
    };
    if (L.chain) {
        GemmArgs g = product(ws + L.hi[0], !L.wide, ws + L.hi[0], !L.wide, L.p, L.p, L.wide ? L.Q : L.P, ws + L.A);
        g.ksplit = L.splits, g.kshard = gram_range(s);
        g.nshards = static_cast<int>(L.split_len / g.kshard);
        g.x_single = single;
        e = launch("ortho_gram32", tpmlp::EPI_NS_GRAM32, g);
        if (e != cudaSuccess) return from_cuda(e);
        tpmlp::NsChain c;
        c.matrices = s->batch, c.P = L.p;
        c.size = static_cast<int>(std::min(s->rows, s->cols) + 15) / 16 * 16;
        c.gram = reinterpret_cast<const float *>(ws + L.A), c.splits = L.splits;
        c.unit = 1.0f / (kScaleX * kScaleX), c.rest = a.rest;
        c.steps = s->steps, c.a = s->a, c.b = s->b, c.c = s->c, c.q_scale = L.q_scale;
        c.Q = ws + L.C;
        c.status = status, c.wait_ns = g_wait_ns.load();
        e = timed_launch("ortho_chain", [&] { return tpmlp::launch_ns_chain(c, st); });
        if (e != cudaSuccess) return from_cuda(e);
        void *out = tma_out ? O : ws + L.hi[1];
        GemmArgs u = L.wide ? product(c.Q, false, ws + L.hi[0], true, L.P, L.Q, L.p, out)
                            : product(ws + L.hi[0], false, c.Q, false, L.P, L.Q, L.p, out);
        u.scale = 1.0f / (kScaleX * L.q_scale);
        u.x_single = single;
        u.out_rows = tma_out ? s->rows : L.P, u.out_cols = tma_out ? s->cols : L.Q;
        e = launch("ortho_final", tpmlp::EPI_NS_FINAL, u);
        if (e == cudaSuccess && !tma_out)
            e = timed_launch("ortho_unpad", [&] {
                return tpmlp::launch_ortho_unpad(out, s->batch, s->rows, s->cols, L.P, L.Q, O, st);
            });
        return from_cuda(e);
    }

    const float shift = ortho_shift(s->a);
    void *A = ws + L.A, *C = ws + L.C;
    for (int k = 0; k < s->steps; ++k) {
        const bool last = k == s->steps - 1;
        void *hi = ws + L.hi[k & 1], *lo = ws + L.lo[k & 1];
        const int64_t inner = L.wide ? L.Q : L.P;
        GemmArgs g = product(hi, !L.wide, hi, !L.wide, L.p, L.p, inner, A);
        g.scale = kScaleA / (kScaleX * kScaleX);
        if (L.splits > 1) {
            g.out0 = ws + L.gram;
            g.ksplit = L.splits, g.kshard = L.split_len;
            e = launch("ortho_gram", tpmlp::EPI_NS_GRAMS, g);
            if (e == cudaSuccess)
                e = timed_launch("ortho_gram_sum", [&] {
                    return tpmlp::launch_ortho_gram_sum(reinterpret_cast<const float *>(ws + L.gram), L.splits,
                                                        s->batch, L.p, g.scale, A, st);
                });
        } else {
            e = launch("ortho_gram", tpmlp::EPI_NS_GRAM, g);
        }
        if (e != cudaSuccess) return from_cuda(e);

        GemmArgs c = product(A, false, A, false, L.p, L.p, L.p, C);
        c.aux = A;
        c.alpha = s->b * (kScaleC / kScaleA);
        c.scale = s->c * (kScaleC / (kScaleA * kScaleA));
        c.diag = shift * kScaleC;
        e = launch("ortho_poly", tpmlp::EPI_NS_POLY, c);
        if (e != cudaSuccess) return from_cuda(e);

        // X' = (a - d) hi + a lo + (C + dI) hi, hi and lo as stored (scale kScaleX, lo 2^11 times too large)
        const Epi epi = last ? tpmlp::EPI_NS_LAST : tpmlp::EPI_NS_UPDATE;
        void *hi2 = ws + L.hi[~k & 1], *lo2 = ws + L.lo[~k & 1];
        void *out = last && tma_out ? O : hi2;
        GemmArgs u = L.wide ? product(C, false, hi, true, L.P, L.Q, L.p, out)
                            : product(hi, false, C, false, L.P, L.Q, L.p, out);
        const float unit = last ? 1.0f / kScaleX : 1.0f;
        u.aux = hi, u.aux2 = lo;
        u.alpha = (s->a - shift) * unit;
        u.beta = s->a / 2048.0f * unit;
        u.scale = unit / kScaleC;
        u.out1 = lo2;
        u.out_rows = tma_out ? s->rows : L.P, u.out_cols = tma_out ? s->cols : L.Q;
        e = launch(last ? "ortho_last" : "ortho_update", epi, u);
        if (e != cudaSuccess) return from_cuda(e);
        if (last && !tma_out)
            e = timed_launch("ortho_unpad", [&] {
                return tpmlp::launch_ortho_unpad(hi2, s->batch, s->rows, s->cols, L.P, L.Q, O, st);
            });
    }
    return from_cuda(e);
}

}  // extern "C"
