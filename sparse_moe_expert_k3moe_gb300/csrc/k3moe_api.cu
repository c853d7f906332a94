// k3moe_api.cu -- the C ABI entry points: argument validation, workspace
// layout, path choice, launch accounting and timing.  Kernels live in the other
// files; nothing here computes on the host beyond bookkeeping.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <type_traits>
#include <utility>
#include <vector>

#include "k3moe_internal.cuh"

namespace k3moe {

// ----------------------------------------------------------------------------------- accounting
static std::atomic<int64_t> g_launches{0};
static std::atomic<int> g_timing_on{0};

struct TimingEntry {
    int64_t launches = 0;
    double ms = 0.0;
    std::vector<std::pair<cudaEvent_t, cudaEvent_t>> pending;
    cudaEvent_t open = nullptr;
};
static std::mutex g_tmu;
static std::map<std::string, TimingEntry> g_timing;
static std::vector<cudaEvent_t> g_event_pool;

static cudaEvent_t take_event()
{
    if (!g_event_pool.empty()) {
        cudaEvent_t e = g_event_pool.back();
        g_event_pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
}

void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

static std::atomic<int> g_prefill_gemm{0};
int prefill_gemm_setting() { return g_prefill_gemm.load(std::memory_order_relaxed); }
// The default (setting 0) is the block-scaled GEMM: measured faster on the K3 shape at
// T = 4096 (routed gate/up 3.73 against 4.67 ms) and T = 16384.
bool prefill_gemm_block_scaled(const k3moe_config &c, int T)
{
    (void)c;
    (void)T;
    return prefill_gemm_setting() != 1;
}

void timing_begin(const char *name, cudaStream_t s)
{
    if (!g_timing_on.load(std::memory_order_relaxed)) return;
    std::lock_guard<std::mutex> lk(g_tmu);
    TimingEntry &t = g_timing[name];
    t.open = take_event();
    cudaEventRecord(t.open, s);
}

void timing_end(const char *name, cudaStream_t s)
{
    if (!g_timing_on.load(std::memory_order_relaxed)) return;
    std::lock_guard<std::mutex> lk(g_tmu);
    TimingEntry &t = g_timing[name];
    if (!t.open) return;
    cudaEvent_t e = take_event();
    cudaEventRecord(e, s);
    t.pending.emplace_back(t.open, e);
    t.open = nullptr;
    t.launches++;
}

// ----------------------------------------------------------------------------------- results still being written
// A mixer's call (k3moe_linear, k3moe_delta_rule) lets the next kernel launch when its own
// has begun, before it has written its result.  Every kernel of the library waits before it reads,
// but for the forward's mat-vec path, which converts x ahead of that wait.  So the streams whose
// latest call is a mixer's are kept here, apart for each capture, and the forward does not read
// ahead on them.  What is not known counts as pending, as does a new stream with the handle of one
// that is gone: the forward then starts a little later, never too early.
struct StreamKey {
    const void *stream;
    unsigned long long capture;                          // its id; 0: launched, not captured
    bool operator==(const StreamKey &o) const { return stream == o.stream && capture == o.capture; }
};
constexpr size_t kMaxPending = 1024;
static std::mutex g_pmu;
static std::vector<StreamKey> g_pending;
static std::atomic<bool> g_any_pending{false}, g_all_pending{false};     // some; more than are kept

static bool stream_key(cudaStream_t s, StreamKey *key)
{
    static thread_local char own;                        // stands for this thread's default stream
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(s, &cap, &id) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    key->stream = s == cudaStreamLegacy ? nullptr : s == cudaStreamPerThread ? (const void *)&own : (const void *)s;
    key->capture = cap == cudaStreamCaptureStatusNone ? 0 : id;
    return true;
}

void result_pending_begin(cudaStream_t s)
{
    StreamKey key;
    const bool known = stream_key(s, &key);
    std::lock_guard<std::mutex> lk(g_pmu);
    if (!known || (g_pending.size() >= kMaxPending && std::find(g_pending.begin(), g_pending.end(), key) == g_pending.end()))
        g_all_pending = true;
    else if (std::find(g_pending.begin(), g_pending.end(), key) == g_pending.end())
        g_pending.push_back(key);
    g_any_pending = true;
}

void result_pending_end(cudaStream_t s)
{
    StreamKey key;
    if (!g_any_pending || !stream_key(s, &key)) return;
    std::lock_guard<std::mutex> lk(g_pmu);
    const auto at = std::find(g_pending.begin(), g_pending.end(), key);
    if (at != g_pending.end()) {
        *at = g_pending.back();
        g_pending.pop_back();
    }
    g_any_pending = g_all_pending || !g_pending.empty();
}

bool result_pending(cudaStream_t s)
{
    StreamKey key;
    if (!g_any_pending) return false;
    if (g_all_pending || !stream_key(s, &key)) return true;
    std::lock_guard<std::mutex> lk(g_pmu);
    return std::find(g_pending.begin(), g_pending.end(), key) != g_pending.end();
}

// The end of a call whose first kernel waits before it lets the next one launch.
static k3moe_status waited(cudaError_t e, cudaStream_t s)
{
    if (e != cudaSuccess) return K3MOE_ECUDA;
    result_pending_end(s);
    return K3MOE_OK;
}

// ----------------------------------------------------------------------------------- validation
static bool finite_pos(float v) { return std::isfinite(v) && v > 0.0f; }

static k3moe_status check_config(const k3moe_config *c)
{
    if (!c) return K3MOE_EINVAL;
    if (c->d <= 0 || c->f <= 0 || c->n_experts <= 0 || c->top_k <= 0 || c->group <= 0 ||
        c->n_shared < 0)
        return K3MOE_EINVAL;
    if (c->group != kGroup) return K3MOE_EINVAL;
    if (!finite_pos(c->situ_b1) || !finite_pos(c->situ_b2)) return K3MOE_EINVAL;
    if (c->renorm != 0 && c->renorm != 1) return K3MOE_EINVAL;
    if (!std::isfinite(c->routed_scale)) return K3MOE_EINVAL;
    if (c->top_k > c->n_experts) return K3MOE_EINVAL;
    if (c->d % kTileK || c->f % kTileK || c->d > kMaxWidth || c->f > kMaxWidth) return K3MOE_ESHAPE;
    if (c->n_experts > kMaxExperts || c->top_k > kMaxTopK || c->n_shared > kMaxShared)
        return K3MOE_ESHAPE;
    return K3MOE_OK;
}

static bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The largest workspace any 0 <= T <= T_max needs.  Sizes grow with T within each
// forward path, with two exceptions: a single token on the mat-vec path also holds the
// split shared-expert partials, and the first T of the tensor-core path can need less
// than the last T of the mat-vec path.  So the maximum is at T = 1, at the last mat-vec
// T, or at T_max.  total(T) is the layout size of one call with T tokens.
template <typename Total>
static size_t max_total(const k3moe_config &c, int32_t T_max, Total total)
{
    size_t m = total(T_max);
    if (T_max >= 1) m = std::max(m, total(1));
    const int64_t first_gemm = std::max<int64_t>(32, (8LL * c.n_experts + c.top_k - 1) / c.top_k);
    const int64_t last_gemv = std::min<int64_t>(T_max, first_gemm - 1);
    if (last_gemv >= 1) m = std::max(m, total((int32_t)last_gemv));
    return m;
}

// The index check of k3moe_check_bounds: the guard the kernels use, with no access.
__global__ void check_bounds_kernel(int32_t *status, int32_t index, int32_t limit)
{
    (void)dguard(status, index >= 0 && index < limit);
}

// ----------------------------------------------------------------------------------- calls by words
template <typename A> static bool word_fits(int64_t v)
{
    if constexpr (std::is_pointer_v<A>) return true;
    else return std::is_same_v<A, size_t> ? v >= 0 : (int64_t)(A)v == v;
}
template <typename A> static A word_as(int64_t v)
{
    if constexpr (std::is_pointer_v<A>) return reinterpret_cast<A>((uintptr_t)v);
    else return (A)v;
}
template <typename... A, size_t... I>
static k3moe_status spread_words(k3moe_status (*f)(A...), const int64_t *args, std::index_sequence<I...>)
{
    return (word_fits<A>(args[I]) && ...) ? f(word_as<A>(args[I])...) : K3MOE_ESHAPE;
}
template <typename... A> static k3moe_status call_words(k3moe_status (*f)(A...), const int64_t *words)
{
    return words[1] == (int64_t)sizeof...(A) ? spread_words(f, words + 2, std::index_sequence_for<A...>()) : K3MOE_EINVAL;
}

}  // namespace k3moe

using namespace k3moe;

extern "C" {

const char *k3moe_strerror(k3moe_status s)
{
    switch (s) {
    case K3MOE_OK: return "ok";
    case K3MOE_EINVAL: return "invalid config field or argument";
    case K3MOE_ESHAPE: return "size outside what the call supports";
    case K3MOE_EALIGN: return "pointer lacks the required alignment";
    case K3MOE_EWORKSPACE: return "workspace missing, misaligned or too small";
    case K3MOE_ECUDA: return "CUDA runtime call failed";
    case K3MOE_EDEVICE: return "device status word reports an error";
    case K3MOE_ETIMEOUT: return "a bounded device-side wait gave up";
    }
    return "unknown status";
}

k3moe_status k3moe_validate_config(const k3moe_config *cfg) { return check_config(cfg); }

size_t k3moe_packed_bytes(const k3moe_config *cfg)
{
    if (check_config(cfg) != K3MOE_OK) return 0;
    return packed_table_bytes(cfg->n_experts, cfg->d, cfg->f);
}

k3moe_status k3moe_workspace_bytes(const k3moe_config *cfg, int32_t T_max, size_t *bytes)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT) return K3MOE_ESHAPE;
    *bytes = max_total(*cfg, T_max, [&](int32_t T) { return ws_layout(*cfg, T).total; });
    return K3MOE_OK;
}

static k3moe_status pack_checks(const k3moe_config *cfg, int32_t lo, int32_t n, const void *p1,
                                const void *s1, const void *p3, const void *s3, const void *p2,
                                const void *s2, const void *table, size_t table_bytes)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (lo < 0 || n < 0 || (int64_t)lo + n > cfg->n_experts) return K3MOE_ESHAPE;
    if (n == 0) return K3MOE_OK;
    if (!p1 || !s1 || !p3 || !s3 || !p2 || !s2 || !table) return K3MOE_EINVAL;
    if (!aligned(p1, 16) || !aligned(p3, 16) || !aligned(p2, 16) || !aligned(table, 256))
        return K3MOE_EALIGN;
    if (table_bytes < packed_table_bytes(cfg->n_experts, cfg->d, cfg->f)) return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_pack_mxfp4(const k3moe_config *cfg, int32_t expert_lo, int32_t n_in,
                              const uint8_t *w1_packed, const uint8_t *w1_scale,
                              const uint8_t *w3_packed, const uint8_t *w3_scale,
                              const uint8_t *w2_packed, const uint8_t *w2_scale, void *table,
                              size_t table_bytes, void *ws, k3moe_stream stream)
{
    k3moe_status st = pack_checks(cfg, expert_lo, n_in, w1_packed, w1_scale, w3_packed, w3_scale,
                                  w2_packed, w2_scale, table, table_bytes);
    if (st != K3MOE_OK || n_in == 0) return st;
    if (ws && !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    cudaError_t e = launch_pack(*cfg, expert_lo, n_in, w1_packed, w1_scale, w3_packed, w3_scale,
                                w2_packed, w2_scale, static_cast<uint8_t *>(table),
                                ws ? static_cast<int32_t *>(ws) : nullptr, (cudaStream_t)stream);
    return e == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_unpack_mxfp4(const k3moe_config *cfg, int32_t expert_lo, int32_t n_out,
                                const void *table, size_t table_bytes, uint8_t *w1_packed,
                                uint8_t *w1_scale, uint8_t *w3_packed, uint8_t *w3_scale,
                                uint8_t *w2_packed, uint8_t *w2_scale, k3moe_stream stream)
{
    k3moe_status st = pack_checks(cfg, expert_lo, n_out, w1_packed, w1_scale, w3_packed, w3_scale,
                                  w2_packed, w2_scale, table, table_bytes);
    if (st != K3MOE_OK || n_out == 0) return st;
    cudaError_t e = launch_unpack(*cfg, expert_lo, n_out, static_cast<const uint8_t *>(table),
                                  w1_packed, w1_scale, w3_packed, w3_scale, w2_packed, w2_scale,
                                  (cudaStream_t)stream);
    return e == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_route(const k3moe_config *cfg, int32_t T, const uint16_t *x,
                         const uint16_t *w_router, const float *bias, int32_t *idx, float *weight,
                         int32_t *offsets, int32_t *perm, void *ws, size_t ws_bytes,
                         k3moe_stream stream)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (!offsets) return K3MOE_EINVAL;
    if (T > 0 && (!x || !w_router || !idx || !weight || !perm)) return K3MOE_EINVAL;
    if (T > 0 && (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(idx, 4) ||
                  !aligned(weight, 4) || !aligned(perm, 4) || (bias && !aligned(bias, 4))))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    const WsLayout L = ws_layout(*cfg, T);
    if (ws_bytes < L.total) return K3MOE_EWORKSPACE;
    cudaError_t e = launch_route(*cfg, T, x, w_router, bias, idx, weight, offsets, perm,
                                 static_cast<uint8_t *>(ws), L, (cudaStream_t)stream);
    return waited(e, (cudaStream_t)stream);
}

k3moe_status k3moe_router_scores(const k3moe_config *cfg, int32_t T, const uint16_t *x,
                                 const uint16_t *w_router, const float *bias, float *scores,
                                 float *choice, void *ws, size_t ws_bytes, k3moe_stream stream)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!x || !w_router || !scores || !choice) return K3MOE_EINVAL;
    if (!aligned(x, 16) || !aligned(w_router, 16) || !aligned(scores, 4) || !aligned(choice, 4) ||
        (bias && !aligned(bias, 4)))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    const WsLayout L = ws_layout(*cfg, T);
    if (ws_bytes < L.total) return K3MOE_EWORKSPACE;
    cudaError_t e = launch_router_scores(*cfg, T, x, w_router, bias, scores, choice,
                                         reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + L.status),
                                         (cudaStream_t)stream);
    return e == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_forward(const k3moe_config *cfg, int32_t T, const uint16_t *x,
                           const int32_t *idx, const float *weight, const int32_t *offsets,
                           const int32_t *perm, const void *expert_table, size_t table_bytes,
                           const uint16_t *sh_w1, const uint16_t *sh_w3, const uint16_t *sh_w2,
                           float *out, void *ws, size_t ws_bytes, k3moe_stream stream)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!x || !idx || !weight || !offsets || !perm || !expert_table || !out) return K3MOE_EINVAL;
    if (cfg->n_shared > 0 && (!sh_w1 || !sh_w3 || !sh_w2)) return K3MOE_EINVAL;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(expert_table, 256) || !aligned(idx, 4) ||
        !aligned(weight, 4) || !aligned(offsets, 4) || !aligned(perm, 4))
        return K3MOE_EALIGN;
    if (cfg->n_shared > 0 && (!aligned(sh_w1, 16) || !aligned(sh_w3, 16) || !aligned(sh_w2, 16)))
        return K3MOE_EALIGN;
    if (table_bytes < packed_table_bytes(cfg->n_experts, cfg->d, cfg->f)) return K3MOE_ESHAPE;
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    const WsLayout L = ws_layout(*cfg, T);
    if (ws_bytes < L.total) return K3MOE_EWORKSPACE;
    cudaError_t e = launch_forward(*cfg, T, x, idx, weight, offsets, perm,
                                        static_cast<const uint8_t *>(expert_table), sh_w1, sh_w3,
                                        sh_w2, out, static_cast<uint8_t *>(ws), L, (cudaStream_t)stream);
    return waited(e, (cudaStream_t)stream);
}

static k3moe_status check_full(const k3moe_config *cfg, const k3moe_full_dims *fd)
{
    k3moe_status st = check_config(cfg);
    if (st != K3MOE_OK) return st;
    if (!fd || fd->hidden <= 0 || (fd->latent_norm != 0 && fd->latent_norm != 1) ||
        !finite_pos(fd->rms_eps))
        return K3MOE_EINVAL;
    if (fd->hidden % kTileK || fd->hidden > kMaxWidth) return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_full_workspace_bytes(const k3moe_config *cfg, const k3moe_full_dims *fd,
                                        int32_t T_max, size_t *bytes)
{
    k3moe_status st = check_full(cfg, fd);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT) return K3MOE_ESHAPE;
    *bytes = max_total(*cfg, T_max, [&](int32_t T) { return full_layout(*cfg, fd->hidden, T).total; });
    return K3MOE_OK;
}

k3moe_status k3moe_full_forward(const k3moe_config *cfg, const k3moe_full_dims *fd, int32_t T,
                                const uint16_t *h, const uint16_t *w_router, const float *bias,
                                const uint16_t *w_down, const void *expert_table,
                                size_t table_bytes, const float *norm_gain,
                                const uint16_t *w_up, const uint16_t *sh_w1,
                                const uint16_t *sh_w3, const uint16_t *sh_w2, int32_t *idx,
                                float *weight, int32_t *offsets, int32_t *perm, float *out,
                                void *ws, size_t ws_bytes, k3moe_stream stream)
{
    k3moe_status st = check_full(cfg, fd);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (!offsets) return K3MOE_EINVAL;
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    const FullLayout F = full_layout(*cfg, fd->hidden, T);
    if (ws_bytes < F.total) return K3MOE_EWORKSPACE;
    if (T == 0) {
        // no tokens: the routing is empty, exactly as k3moe_route leaves it
        cudaError_t e = launch_route(F.cr, 0, h, w_router, bias, idx, weight, offsets, perm,
                                     static_cast<uint8_t *>(ws), F.route, (cudaStream_t)stream);
        return e == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
    }
    if (!h || !w_router || !w_down || !expert_table || !w_up || !idx || !weight || !perm || !out ||
        (fd->latent_norm && !norm_gain))
        return K3MOE_EINVAL;
    if (cfg->n_shared > 0 && (!sh_w1 || !sh_w3 || !sh_w2)) return K3MOE_EINVAL;
    if (!aligned(h, 16) || !aligned(w_router, 16) || !aligned(w_down, 16) || !aligned(w_up, 16) ||
        !aligned(out, 16) || !aligned(expert_table, 256) || !aligned(idx, 4) || !aligned(weight, 4) ||
        !aligned(offsets, 4) || !aligned(perm, 4) || (bias && !aligned(bias, 4)) ||
        (norm_gain && !aligned(norm_gain, 4)))
        return K3MOE_EALIGN;
    if (cfg->n_shared > 0 && (!aligned(sh_w1, 16) || !aligned(sh_w3, 16) || !aligned(sh_w2, 16)))
        return K3MOE_EALIGN;
    if (table_bytes < packed_table_bytes(cfg->n_experts, cfg->d, cfg->f)) return K3MOE_ESHAPE;
    cudaError_t e = launch_full(*cfg, fd->hidden, fd->latent_norm, fd->rms_eps, T, h, w_router, bias,
                                w_down, static_cast<const uint8_t *>(expert_table), norm_gain, w_up,
                                sh_w1, sh_w3, sh_w2, idx, weight, offsets, perm, out,
                                static_cast<uint8_t *>(ws), F, (cudaStream_t)stream);
    return waited(e, (cudaStream_t)stream);
}

static k3moe_status check_linear(const k3moe_linear_config *lc)
{
    if (!lc) return K3MOE_EINVAL;
    if (lc->n <= 0 || lc->k <= 0 || (lc->y_f32 != 0 && lc->y_f32 != 1)) return K3MOE_EINVAL;
    if (lc->act < K3MOE_ACT_NONE || lc->act > K3MOE_ACT_LOGSIGMOID) return K3MOE_EINVAL;
    if (lc->n > (1 << 20) || lc->k > 65536 || lc->k % 8) return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_linear_workspace_bytes(const k3moe_linear_config *lc, int32_t T_max, size_t *bytes)
{
    k3moe_status st = check_linear(lc);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT) return K3MOE_ESHAPE;
    *bytes = kCtrOffset + kCtrBytes;
    return K3MOE_OK;
}

k3moe_status k3moe_linear(const k3moe_linear_config *lc, int32_t T, const uint16_t *x, int64_t x_stride,
                          const uint16_t *w, const float *bias, const void *residual,
                          int64_t residual_stride, void *y, int64_t y_stride, void *ws,
                          size_t ws_bytes, k3moe_stream stream)
{
    k3moe_status st = check_linear(lc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!x || !w || !y) return K3MOE_EINVAL;
    if (x_stride < lc->k || x_stride % 8 || x_stride > kMaxStride || y_stride < lc->n ||
        y_stride > kMaxStride ||
        (residual && (residual_stride < lc->n || residual_stride > kMaxStride)))
        return K3MOE_ESHAPE;
    if (residual == y && residual_stride != y_stride) return K3MOE_EINVAL;
    const size_t ysz = lc->y_f32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, ysz) || (residual && !aligned(residual, ysz)) ||
        (bias && !aligned(bias, 4)))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < kCtrOffset + kCtrBytes) return K3MOE_EWORKSPACE;
    const LinearArgs a{T, lc->n, lc->k, lc->act, lc->y_f32, x, x_stride, w, bias, residual,
                       residual ? residual_stride : 0, y, y_stride, static_cast<int32_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_linear(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_delta_validate_config(const k3moe_delta_config *dc)
{
    if (!dc) return K3MOE_EINVAL;
    if (dc->n_heads <= 0 || dc->n_qk_heads <= 0 || dc->head_dim <= 0 || dc->gate_dim <= 0 ||
        (dc->qk_norm != 0 && dc->qk_norm != 1) || !std::isfinite(dc->scale) ||
        (dc->qk_norm && !finite_pos(dc->norm_eps)) || dc->n_heads % dc->n_qk_heads)
        return K3MOE_EINVAL;
    if (dc->gate_dim != 1 && dc->gate_dim != dc->head_dim) return K3MOE_EINVAL;
    if (dc->head_dim != kDeltaD || dc->n_heads > kMaxDeltaHeads) return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_delta_workspace_bytes(const k3moe_delta_config *dc, int32_t n_seq_max, int32_t T_max,
                                         size_t *bytes)
{
    k3moe_status st = k3moe_delta_validate_config(dc);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT || n_seq_max < 0 || n_seq_max > kMaxSeqs) return K3MOE_ESHAPE;
    *bytes = delta_workspace(*dc, n_seq_max, T_max);
    return K3MOE_OK;
}

k3moe_status k3moe_delta_rule(const k3moe_delta_config *dc, int32_t n_seq, int32_t T,
                              const int32_t *seq_start, const uint16_t *q, int64_t q_stride,
                              const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                              const float *g, const float *beta, const float *state_in,
                              float *state_out, int32_t n_slots, const int32_t *slots, uint16_t *out,
                              void *ws, size_t ws_bytes, k3moe_stream stream)
{
    k3moe_status st = k3moe_delta_validate_config(dc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT || n_seq < 0 || n_seq > kMaxSeqs) return K3MOE_ESHAPE;
    if (n_seq == 0) return T == 0 ? K3MOE_OK : K3MOE_ESHAPE;
    if (!seq_start && n_seq != 1 && T != n_seq) return K3MOE_EINVAL;
    if (!state_out) return K3MOE_EINVAL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !out)) return K3MOE_EINVAL;
    const int64_t wq = (int64_t)dc->n_qk_heads * kDeltaD, wv = (int64_t)dc->n_heads * kDeltaD;
    if (q_stride < wq || k_stride < wq || v_stride < wv || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
        q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride)
        return K3MOE_ESHAPE;
    if (n_slots < 1 || (!slots && n_slots < n_seq)) return K3MOE_ESHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 16) || !aligned(beta, 4) ||
        !aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(out, 16) || !aligned(seq_start, 4) ||
        !aligned(slots, 4))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < delta_workspace(*dc, n_seq, T)) return K3MOE_EWORKSPACE;
    const DeltaArgs a{n_seq, T, dc->n_heads, dc->n_qk_heads, dc->gate_dim, dc->qk_norm, dc->norm_eps,
                      dc->scale, seq_start, q, k, v, q_stride, k_stride, v_stride, g, beta, state_in,
                      state_out, n_slots, slots, out, static_cast<uint8_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_delta(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

// Row strides of 16-byte accesses: within [width, kMaxStride], a multiple of 8.
static bool row_stride(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride <= kMaxStride; }
// A token's and a head's stride of `heads` heads of `width` columns: no two overlap.
static bool head_strides(int64_t stride, int64_t head, int64_t heads, int64_t width, int64_t each)
{
    return head >= width && head <= kMaxStride && head % each == 0 && stride >= (heads - 1) * head + width &&
           stride <= kMaxStride && stride % each == 0;
}

k3moe_status k3moe_norm(const k3moe_norm_config *nc, int32_t T, const void *x, int64_t x_stride,
                        const uint16_t *gate, int64_t gate_stride, const float *post_gain,
                        const void *residual, int64_t residual_stride, const float *scale,
                        void *total, int64_t total_stride, const float *pre_gain, uint16_t *out,
                        int64_t out_stride, k3moe_stream stream)
{
    if (!nc || nc->n <= 0 || nc->group <= 0) return K3MOE_EINVAL;
    const auto flag = [](int32_t f) { return f == 0 || f == 1; };
    if (!flag(nc->post_norm) || !flag(nc->pre_norm) || !flag(nc->x_f32) || !flag(nc->sum_f32) ||
        nc->gate < K3MOE_GATE_NONE || nc->gate > K3MOE_GATE_SILU || !std::isfinite(nc->alpha) ||
        ((nc->post_norm || nc->pre_norm) && !finite_pos(nc->eps)))
        return K3MOE_EINVAL;
    if (nc->n > kMaxNorm || nc->n % 8) return K3MOE_ESHAPE;
    if (nc->group != nc->n && ((nc->group != 64 && nc->group != 128 && nc->group != 256) || nc->n % nc->group)) return K3MOE_ESHAPE;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!x || (nc->post_norm && !post_gain) || (nc->pre_norm && !pre_gain) || !out != !nc->pre_norm ||
        (!total && !out) || !gate != (nc->gate == K3MOE_GATE_NONE))
        return K3MOE_EINVAL;
    if (!row_stride(x_stride, nc->n) || (gate && !row_stride(gate_stride, nc->n)) ||
        (residual && !row_stride(residual_stride, nc->n)) || (total && !row_stride(total_stride, nc->n)) ||
        (out && !row_stride(out_stride, nc->n)))
        return K3MOE_ESHAPE;
    // in place where each element is read and written by one thread; not otherwise
    const auto same = [&](const void *w, int64_t ws, int wf, const void *r, int64_t rs, int rf) {
        return w && w == r && (ws != rs || wf != rf);
    };
    if (same(total, total_stride, nc->sum_f32, x, x_stride, nc->x_f32) || same(total, total_stride, nc->sum_f32, gate, gate_stride, 0) ||
        same(total, total_stride, nc->sum_f32, residual, residual_stride, nc->sum_f32) || same(out, out_stride, 0, x, x_stride, nc->x_f32) ||
        same(out, out_stride, 0, gate, gate_stride, 0) || same(out, out_stride, 0, residual, residual_stride, nc->sum_f32) ||
        (total && total == out))
        return K3MOE_EINVAL;
    for (const void *p : {x, (const void *)gate, (const void *)post_gain, residual, (const void *)scale, (const void *)total,
                          (const void *)pre_gain, (const void *)out})
        if (!aligned(p, 16)) return K3MOE_EALIGN;
    const NormArgs a{T, nc->n, nc->group, nc->post_norm, nc->pre_norm, nc->gate, nc->x_f32, nc->sum_f32, nc->eps, nc->alpha, x, x_stride,
                     gate, gate_stride, post_gain, residual, residual_stride, scale, total, total_stride, pre_gain, out, out_stride};
    result_pending_begin((cudaStream_t)stream);
    return launch_norm(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

static k3moe_status check_head_linear(const k3moe_head_linear_config *hc)
{
    if (!hc || hc->n_heads <= 0 || hc->n <= 0 || hc->k <= 0) return K3MOE_EINVAL;
    if (hc->n_heads > kMaxLatHeads || hc->n > kMaxHeadN || hc->k > kMaxHeadK || hc->k % 8) return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_head_linear_workspace_bytes(const k3moe_head_linear_config *hc, int32_t T_max, size_t *bytes)
{
    const k3moe_status st = check_head_linear(hc);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT) return K3MOE_ESHAPE;
    *bytes = kCtrOffset + kCtrBytes;
    return K3MOE_OK;
}

k3moe_status k3moe_head_linear(const k3moe_head_linear_config *hc, int32_t T, const uint16_t *x,
                               int64_t x_stride, int64_t x_head_stride, const uint16_t *w, uint16_t *y,
                               int64_t y_stride, int64_t y_head_stride, void *ws, size_t ws_bytes,
                               k3moe_stream stream)
{
    const k3moe_status st = check_head_linear(hc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!x || !w || !y) return K3MOE_EINVAL;
    if (!head_strides(x_stride, x_head_stride, hc->n_heads, hc->k, 8) || !head_strides(y_stride, y_head_stride, hc->n_heads, hc->n, 1))
        return K3MOE_ESHAPE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 2)) return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < kCtrOffset + kCtrBytes) return K3MOE_EWORKSPACE;
    const HeadLinearArgs a{T, hc->n_heads, hc->n, hc->k, x, x_stride, x_head_stride, w, y, y_stride, y_head_stride,
                           static_cast<int32_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_head_linear(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_latent_validate_config(const k3moe_latent_config *lc)
{
    if (!lc || lc->n_heads <= 0 || lc->rank <= 0 || lc->rope_dim <= 0 || lc->key_dim <= 0 || lc->value_dim <= 0 || lc->page_size <= 0 ||
        lc->rope < K3MOE_ROPE_NONE || lc->rope > K3MOE_ROPE_HALVES || (lc->norm != 0 && lc->norm != 1) ||
        (lc->norm && !finite_pos(lc->norm_eps)) || !finite_pos(lc->scale) || (lc->causal != 0 && lc->causal != 1))
        return K3MOE_EINVAL;
    if (lc->n_heads > kMaxLatHeads || lc->rank != kLatC || lc->rope_dim != kLatR || lc->key_dim != kLatK || lc->value_dim != kLatV ||
        lc->page_size < 16 || lc->page_size > 256 || (lc->page_size & (lc->page_size - 1)))
        return K3MOE_ESHAPE;
    return K3MOE_OK;
}

k3moe_status k3moe_latent_workspace_bytes(const k3moe_latent_config *lc, int32_t n_seq_max, int32_t T_max,
                                          size_t *bytes)
{
    const k3moe_status st = k3moe_latent_validate_config(lc);
    if (st != K3MOE_OK) return st;
    if (!bytes) return K3MOE_EINVAL;
    if (T_max < 0 || T_max > kMaxT || n_seq_max < 0 || n_seq_max > kMaxSeqs) return K3MOE_ESHAPE;
    *bytes = latent_workspace(*lc, n_seq_max, T_max);
    return K3MOE_OK;
}

k3moe_status k3moe_latent_write(const k3moe_latent_config *lc, int32_t T, const uint16_t *c, int64_t c_stride,
                                const float *gain, const int32_t *positions, const double *inv_freq,
                                uint16_t *rows, int64_t rows_stride, uint16_t *cache, int32_t n_pages,
                                const int64_t *slots, const uint16_t *q, int64_t q_stride, int64_t q_head_stride,
                                uint16_t *q_rope, int64_t q_rope_stride, int64_t q_rope_head_stride, void *ws,
                                size_t ws_bytes, k3moe_stream stream)
{
    const k3moe_status st = k3moe_latent_validate_config(lc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT) return K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!c || (lc->norm && !gain) || (lc->rope != K3MOE_ROPE_NONE && (!positions || !inv_freq)) || !cache != !slots || !q != !q_rope ||
        (!rows && !cache && !q))
        return K3MOE_EINVAL;
    if (!row_stride(c_stride, kLatRow) || (rows && !row_stride(rows_stride, kLatRow)) || (cache && n_pages < 1) ||
        (q && (!head_strides(q_stride, q_head_stride, lc->n_heads, kLatR, 8) ||
               !head_strides(q_rope_stride, q_rope_head_stride, lc->n_heads, kLatR, 8))))
        return K3MOE_ESHAPE;
    if ((rows == c && rows_stride != c_stride) || (q && q == q_rope && (q_stride != q_rope_stride || q_head_stride != q_rope_head_stride)))
        return K3MOE_EINVAL;
    if (!aligned(c, 16) || !aligned(gain, 16) || !aligned(positions, 4) || !aligned(inv_freq, 8) || !aligned(rows, 16) ||
        !aligned(cache, 16) || !aligned(slots, 8) || !aligned(q, 16) || !aligned(q_rope, 16))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < kCtrOffset + kCtrBytes) return K3MOE_EWORKSPACE;
    const LatentWriteArgs a{T, lc->n_heads, lc->rope, lc->norm, lc->norm_eps, c, c_stride, gain, positions, inv_freq, rows, rows_stride,
                            cache, (int64_t)n_pages * lc->page_size, slots, q, q_stride, q_head_stride, q_rope, q_rope_stride,
                            q_rope_head_stride, static_cast<int32_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_latent_write(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_latent_attend(const k3moe_latent_config *lc, int32_t n_seq, int32_t T, const int32_t *seq_start,
                                 const uint16_t *q, int64_t q_stride, int64_t q_head_stride, const uint16_t *cache,
                                 int32_t n_pages, const int32_t *pages, int32_t max_pages, const int32_t *kv_len,
                                 uint16_t *out, float *lse, void *ws, size_t ws_bytes, k3moe_stream stream)
{
    const k3moe_status st = k3moe_latent_validate_config(lc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT || n_seq < 0 || n_seq > kMaxSeqs) return K3MOE_ESHAPE;
    if (n_seq == 0) return T == 0 ? K3MOE_OK : K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!seq_start && n_seq != 1 && T != n_seq) return K3MOE_EINVAL;
    if (!q || !cache || !pages || !kv_len || !out) return K3MOE_EINVAL;
    // a row of the cache is a 32-bit coordinate of its loads
    if (!head_strides(q_stride, q_head_stride, lc->n_heads, kLatRow, 8) || n_pages < 1 || max_pages < 1 ||
        (int64_t)n_pages * lc->page_size > INT32_MAX - 1024 || (int64_t)max_pages * lc->page_size > INT32_MAX - 1024)
        return K3MOE_ESHAPE;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(seq_start, 4) || !aligned(pages, 4) ||
        !aligned(kv_len, 4) || !aligned(lse, 4))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < latent_workspace(*lc, n_seq, T)) return K3MOE_EWORKSPACE;
    int32_t page_shift = 4;
    while ((1 << page_shift) < lc->page_size) page_shift++;
    const AttendArgs a{n_seq, T, lc->n_heads, lc->page_size, page_shift, lc->causal, 0, lc->scale, seq_start, q, q_stride, q_head_stride, cache, n_pages,
                       pages, max_pages, kv_len, out, lse, static_cast<uint8_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_attend(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_latent_prompt(const k3moe_latent_config *lc, int32_t n_seq, int32_t T, int32_t S,
                                 const int32_t *seq_start, const int32_t *kv_start, const uint16_t *q,
                                 int64_t q_stride, int64_t q_head_stride, const uint16_t *kv, int64_t kv_stride,
                                 int64_t kv_head_stride, const uint16_t *rope_key, int64_t rope_stride, uint16_t *out,
                                 float *lse, void *ws, size_t ws_bytes, k3moe_stream stream)
{
    const k3moe_status st = k3moe_latent_validate_config(lc);
    if (st != K3MOE_OK) return st;
    if (T < 0 || T > kMaxT || S < 0 || S > kMaxT || n_seq < 0 || n_seq > kMaxSeqs) return K3MOE_ESHAPE;
    if (n_seq == 0) return T == 0 ? K3MOE_OK : K3MOE_ESHAPE;
    if (T == 0) return K3MOE_OK;
    if (!seq_start && n_seq != 1 && T != n_seq) return K3MOE_EINVAL;
    // without offsets of their own the keys are the queries' tokens; one sequence has all of both
    if (!kv_start && S != T && !(n_seq == 1 && !seq_start)) return K3MOE_EINVAL;
    if (!q || !out || (S > 0 && (!kv || !rope_key))) return K3MOE_EINVAL;
    if (!head_strides(q_stride, q_head_stride, lc->n_heads, kLatK + kLatR, 8) ||
        !head_strides(kv_stride, kv_head_stride, lc->n_heads, kLatK + kLatV, 8) || !row_stride(rope_stride, kLatR))
        return K3MOE_ESHAPE;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(rope_key, 16) || !aligned(out, 16) || !aligned(seq_start, 4) ||
        !aligned(kv_start, 4) || !aligned(lse, 4))
        return K3MOE_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < latent_workspace(*lc, n_seq, T)) return K3MOE_EWORKSPACE;
    const PromptArgs a{n_seq, T, S, lc->n_heads, lc->causal, lc->scale, seq_start, kv_start, q, q_stride, q_head_stride, kv, kv_stride,
                       kv_head_stride, rope_key, rope_stride, out, lse, static_cast<uint8_t *>(ws)};
    result_pending_begin((cudaStream_t)stream);
    return launch_prompt(a, (cudaStream_t)stream) == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

k3moe_status k3moe_call(const int64_t *words)
{
    if (!words) return K3MOE_EINVAL;
    switch (words[0]) {
    case K3MOE_ENTRY_NORM: return call_words(k3moe_norm, words);
    case K3MOE_ENTRY_HEAD_LINEAR: return call_words(k3moe_head_linear, words);
    case K3MOE_ENTRY_LATENT_WRITE: return call_words(k3moe_latent_write, words);
    case K3MOE_ENTRY_LATENT_ATTEND: return call_words(k3moe_latent_attend, words);
    case K3MOE_ENTRY_LATENT_PROMPT: return call_words(k3moe_latent_prompt, words);
    default: return K3MOE_EINVAL;
    }
}

k3moe_status k3moe_device_status(void *ws, k3moe_stream stream, int32_t *code)
{
    if (!ws || !aligned(ws, 256) || !code) return K3MOE_EINVAL;
    int32_t v = 0;
    cudaStream_t s = (cudaStream_t)stream;
    if (cudaMemcpyAsync(&v, ws, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return K3MOE_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return K3MOE_ECUDA;
    if (cudaMemsetAsync(ws, 0, sizeof(int32_t), s) != cudaSuccess) return K3MOE_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return K3MOE_ECUDA;
    *code = v;
    if (v & K3MOE_DEV_TIMEOUT) return K3MOE_ETIMEOUT;
    return (v & K3MOE_DEV_ERROR_MASK) ? K3MOE_EDEVICE : K3MOE_OK;
}

k3moe_status k3moe_check_wait_timeout(void *ws, int64_t limit_cycles, k3moe_stream stream)
{
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    if (limit_cycles < 1 || limit_cycles > 4000000000ll) return K3MOE_ESHAPE;
    int32_t *status = static_cast<int32_t *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    if (launch_wait_check_gemv(status, limit_cycles, s) != cudaSuccess) return K3MOE_ECUDA;
    if (launch_wait_check_tc(status, limit_cycles, s) != cudaSuccess) return K3MOE_ECUDA;
    return K3MOE_OK;
}

k3moe_status k3moe_check_bounds(void *ws, int32_t index, int32_t limit, k3moe_stream stream)
{
    if (!ws || !aligned(ws, 256)) return K3MOE_EWORKSPACE;
    if (limit < 1) return K3MOE_ESHAPE;
    cudaStream_t s = (cudaStream_t)stream;
    check_bounds_kernel<<<1, 1, 0, s>>>(static_cast<int32_t *>(ws), index, limit);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? K3MOE_OK : K3MOE_ECUDA;
}

int32_t k3moe_build_flags(void)
{
#ifdef K3MOE_DEBUG
    return K3MOE_BUILD_DEBUG;
#else
    return 0;
#endif
}

int64_t k3moe_launch_count(void) { return g_launches.load(); }

k3moe_status k3moe_set_prefill_gemm(int32_t variant)
{
    if (variant < 0 || variant > 2) return K3MOE_EINVAL;
    g_prefill_gemm.store(variant, std::memory_order_relaxed);
    return K3MOE_OK;
}

int32_t k3moe_get_prefill_gemm(void) { return prefill_gemm_setting(); }

void k3moe_timing_enable(int32_t on) { g_timing_on.store(on ? 1 : 0); }

int32_t k3moe_timing_read(const char **names, int64_t *launches, double *ms, int32_t cap)
{
    std::lock_guard<std::mutex> lk(g_tmu);
    int32_t n = 0;
    for (auto &kv : g_timing) {
        TimingEntry &t = kv.second;
        for (auto &pr : t.pending) {
            float v = 0.0f;
            cudaEventSynchronize(pr.second);
            if (cudaEventElapsedTime(&v, pr.first, pr.second) == cudaSuccess) t.ms += v;
            g_event_pool.push_back(pr.first);
            g_event_pool.push_back(pr.second);
        }
        t.pending.clear();
        if (n < cap) {
            if (names) names[n] = kv.first.c_str();
            if (launches) launches[n] = t.launches;
            if (ms) ms[n] = t.ms;
        }
        n++;
    }
    return n;
}

void k3moe_timing_reset(void)
{
    std::lock_guard<std::mutex> lk(g_tmu);
    for (auto &kv : g_timing) {
        for (auto &pr : kv.second.pending) {
            cudaEventSynchronize(pr.second);
            g_event_pool.push_back(pr.first);
            g_event_pool.push_back(pr.second);
        }
        kv.second.pending.clear();
        kv.second.launches = 0;
        kv.second.ms = 0.0;
    }
}

}  // extern "C"
