// extern "C" entry points of include/arops.h: argument validation, dispatch to
// the kernel launchers, status codes and the thread-local error string.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

#include "common.cuh"
#include "paged.cuh"

namespace arops {

namespace {

thread_local char g_last_error[512] = "";
std::atomic<int> g_pdl{0};
std::atomic<int> g_streaming{0};
std::atomic<int> g_topk_cluster{1};
std::atomic<uint64_t> g_launches{0};

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];  // 0 = not queried yet

arops_status fail(arops_status st, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return st;
}

arops_status ok()
{
    g_last_error[0] = '\0';
    return AROPS_OK;
}

arops_status from_cuda(cudaError_t err, const char* op)
{
    if (err == cudaSuccess)
        return ok();
    return fail(AROPS_ERR_CUDA, "%s: CUDA error %d (%s): %s", op, (int)err, cudaGetErrorName(err),
                cudaGetErrorString(err));
}

bool valid_dtype(arops_dtype d)
{
    return d == AROPS_F32 || d == AROPS_BF16;
}

}  // namespace

// The device error word: kernels that abandon their work (a bounded wait ran
// out) OR a bit into it; arops_device_errors reads and clears it.
__device__ unsigned int g_device_errors = 0;

// Looked up on every call rather than cached per device ordinal: a __device__
// variable has one instance per CUDA context, and the caller's current context
// need not be the one a cached address came from (a context of its own, or a
// primary context reset and created anew).
cudaError_t device_error_word(unsigned** word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_device_errors);
}

cudaError_t current_device_info(DeviceInfo* info)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    int sms = (dev >= 0 && dev < kMaxDevices) ? g_sm_count[dev].load(std::memory_order_relaxed) : 0;
    if (sms == 0) {
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess)
            return err;
        if (dev >= 0 && dev < kMaxDevices)
            g_sm_count[dev].store(sms, std::memory_order_relaxed);
    }
    info->sm_count = sms;
    return cudaSuccess;
}

bool pdl_enabled()
{
    return g_pdl.load(std::memory_order_relaxed) != 0;
}

bool streaming_enabled()
{
    return g_streaming.load(std::memory_order_relaxed) != 0;
}

int topk_cluster_mode()
{
    return g_topk_cluster.load(std::memory_order_relaxed);
}

void count_launch()
{
    g_launches.fetch_add(1, std::memory_order_relaxed);
}

}  // namespace arops

using namespace arops;

namespace {

// Shared validation and dispatch of the four norm entry points.
arops_status norm_entry(const char* name, const void* x, const void* residual_in,
                        void* residual_out, const void* gamma, const void* beta, void* y,
                        int64_t rows, int64_t hidden, float eps, arops_dtype dtype, void* stream,
                        bool add, bool ln)
{
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "%s: unknown dtype %d", name, (int)dtype);
    if (rows < 0 || hidden <= 0 || hidden > INT32_MAX)
        return fail(AROPS_ERR_INVALID, "%s: bad shape rows=%lld hidden=%lld", name,
                    (long long)rows, (long long)hidden);
    if (!(eps >= 0.0f) || isinf(eps))
        return fail(AROPS_ERR_INVALID, "%s: eps must be finite and >= 0", name);
    if (rows == 0)
        return ok();
    if (!x || !gamma || !y || (add && (!residual_in || !residual_out)) || (ln && !beta))
        return fail(AROPS_ERR_INVALID, "%s: null pointer", name);
    if (add && y == residual_out)
        return fail(AROPS_ERR_INVALID, "%s: y and residual_out are one buffer", name);
    return from_cuda(launch_norm(x, add ? residual_in : nullptr, add ? residual_out : nullptr,
                                 gamma, ln ? beta : nullptr, y, rows, hidden, eps, dtype,
                                 static_cast<cudaStream_t>(stream)),
                     name);
}

}  // namespace

extern "C" {

AROPS_API arops_status arops_rmsnorm(const void* x, const void* gamma, void* y, int64_t rows,
                                     int64_t hidden, float eps, arops_dtype dtype, void* stream)
{
    return norm_entry("arops_rmsnorm", x, nullptr, nullptr, gamma, nullptr, y, rows, hidden, eps,
                      dtype, stream, false, false);
}

AROPS_API arops_status arops_add_rmsnorm(const void* x, const void* residual_in,
                                         void* residual_out, const void* gamma, void* y,
                                         int64_t rows, int64_t hidden, float eps,
                                         arops_dtype dtype, void* stream)
{
    return norm_entry("arops_add_rmsnorm", x, residual_in, residual_out, gamma, nullptr, y, rows,
                      hidden, eps, dtype, stream, true, false);
}

AROPS_API arops_status arops_layernorm(const void* x, const void* gamma, const void* beta, void* y,
                                       int64_t rows, int64_t hidden, float eps, arops_dtype dtype,
                                       void* stream)
{
    return norm_entry("arops_layernorm", x, nullptr, nullptr, gamma, beta, y, rows, hidden, eps,
                      dtype, stream, false, true);
}

AROPS_API arops_status arops_add_layernorm(const void* x, const void* residual_in,
                                           void* residual_out, const void* gamma,
                                           const void* beta, void* y, int64_t rows,
                                           int64_t hidden, float eps, arops_dtype dtype,
                                           void* stream)
{
    return norm_entry("arops_add_layernorm", x, residual_in, residual_out, gamma, beta, y, rows,
                      hidden, eps, dtype, stream, true, true);
}

AROPS_API arops_status arops_mrope_qk(const void* q, const void* k, void* q_out, void* k_out,
                                      const int32_t* pos, int64_t tokens, int32_t n_q_heads,
                                      int32_t n_k_heads, int32_t head_dim,
                                      const int32_t* sections, float theta, arops_dtype dtype,
                                      void* stream)
{
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: unknown dtype %d", (int)dtype);
    if (tokens < 0 || n_q_heads < 0 || n_k_heads < 0)
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: negative size");
    if (head_dim <= 0 || head_dim % 2 != 0)
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: head_dim must be even and > 0 (got %d)",
                    (int)head_dim);
    if (head_dim > 512)
        return fail(AROPS_ERR_UNSUPPORTED, "arops_mrope_qk: head_dim %d > 512", (int)head_dim);
    if (!sections)
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: sections is null");
    if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 ||
        (int64_t)sections[0] + sections[1] + sections[2] != head_dim / 2)
        return fail(AROPS_ERR_INVALID,
                    "arops_mrope_qk: sections [%d,%d,%d] must be >= 0 and sum to head_dim/2 = %d",
                    (int)sections[0], (int)sections[1], (int)sections[2], (int)head_dim / 2);
    if (!(theta > 0.0f) || isinf(theta))
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: theta must be finite and > 0");
    if (tokens == 0 || n_q_heads + n_k_heads == 0)
        return ok();
    if (!pos || (n_q_heads > 0 && (!q || !q_out)) || (n_k_heads > 0 && (!k || !k_out)))
        return fail(AROPS_ERR_INVALID, "arops_mrope_qk: null pointer");
    MropeArgs a;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.pos = pos;
    a.tokens = tokens;
    a.n_q_heads = n_q_heads;
    a.n_k_heads = n_k_heads;
    a.head_dim = head_dim;
    a.sections[0] = sections[0];
    a.sections[1] = sections[1];
    a.sections[2] = sections[2];
    a.theta = theta;
    return from_cuda(launch_mrope(a, dtype, static_cast<cudaStream_t>(stream)), "arops_mrope_qk");
}

AROPS_API arops_status arops_mrope_kv_append(const void* q, const void* k, const void* v,
                                             void* q_out, void* k_cache, void* v_cache,
                                             const int32_t* pos, const int32_t* cache_loc,
                                             int64_t tokens, int32_t n_q_heads, int32_t n_kv_heads,
                                             int32_t head_dim, int64_t cache_rows, int64_t max_seq,
                                             const int32_t* sections, float theta,
                                             arops_dtype dtype, void* stream)
{
    const char* name = "arops_mrope_kv_append";
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "%s: unknown dtype %d", name, (int)dtype);
    if (tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || cache_rows < 0 || max_seq < 0)
        return fail(AROPS_ERR_INVALID, "%s: negative size", name);
    if (head_dim <= 0 || head_dim % 2 != 0)
        return fail(AROPS_ERR_INVALID, "%s: head_dim must be even and > 0 (got %d)", name,
                    (int)head_dim);
    if (head_dim > 512)
        return fail(AROPS_ERR_UNSUPPORTED, "%s: head_dim %d > 512", name, (int)head_dim);
    if (!sections)
        return fail(AROPS_ERR_INVALID, "%s: sections is null", name);
    if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 ||
        (int64_t)sections[0] + sections[1] + sections[2] != head_dim / 2)
        return fail(AROPS_ERR_INVALID, "%s: sections [%d,%d,%d] must be >= 0 and sum to %d", name,
                    (int)sections[0], (int)sections[1], (int)sections[2], (int)head_dim / 2);
    if (!(theta > 0.0f) || isinf(theta))
        return fail(AROPS_ERR_INVALID, "%s: theta must be finite and > 0", name);
    if (tokens == 0 || n_q_heads + n_kv_heads == 0)
        return ok();
    if (!pos || (n_q_heads > 0 && (!q || !q_out)) ||
        (n_kv_heads > 0 && (!k || !v || !k_cache || !v_cache || !cache_loc)))
        return fail(AROPS_ERR_INVALID, "%s: null pointer", name);
    if (k_cache == v_cache && n_kv_heads > 0)
        return fail(AROPS_ERR_INVALID, "%s: k_cache and v_cache are one buffer", name);
    MropeArgs a;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = nullptr;
    a.pos = pos;
    a.tokens = tokens;
    a.n_q_heads = n_q_heads;
    a.n_k_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.sections[0] = sections[0];
    a.sections[1] = sections[1];
    a.sections[2] = sections[2];
    a.theta = theta;
    AppendArgs x;
    x.v = v;
    x.k_cache = k_cache;
    x.v_cache = v_cache;
    x.cache_loc = cache_loc;
    x.cache_rows = cache_rows;
    x.max_seq = max_seq;
    return from_cuda(launch_mrope_append(a, x, dtype, static_cast<cudaStream_t>(stream)), name);
}

}  // extern "C"

namespace {

// Positions of a sequence: the kernels step past the last one by less than this
// leaves of 32 bits.
constexpr int64_t kMaxPositions = INT32_MAX - 1024;

// A pool of pages: its sizes, and (when it holds anything) its pointers.
arops_status check_cache(const char* name, const arops_paged_cache* c, int32_t max_head_dim)
{
    if (!c)
        return fail(AROPS_ERR_INVALID, "%s: cache is null", name);
    if (!valid_dtype(c->dtype))
        return fail(AROPS_ERR_INVALID, "%s: unknown dtype %d", name, (int)c->dtype);
    if (c->num_pages < 1 || c->page_size < 1 || c->n_kv_heads < 0 || c->head_dim < 1)
        return fail(AROPS_ERR_INVALID,
                    "%s: bad cache shape [%lld pages, %d heads, %d slots, %d values]", name,
                    (long long)c->num_pages, (int)c->n_kv_heads, (int)c->page_size,
                    (int)c->head_dim);
    if (c->num_pages > INT32_MAX)
        return fail(AROPS_ERR_UNSUPPORTED, "%s: %lld pages > 2^31 - 1", name,
                    (long long)c->num_pages);
    if (c->head_dim > max_head_dim)
        return fail(AROPS_ERR_UNSUPPORTED, "%s: head_dim %d > %d", name, (int)c->head_dim,
                    (int)max_head_dim);
    if (c->n_kv_heads > 0 && (!c->k_pages || !c->v_pages))
        return fail(AROPS_ERR_INVALID, "%s: null page pool", name);
    if (c->n_kv_heads > 0 && c->k_pages == c->v_pages)
        return fail(AROPS_ERR_INVALID, "%s: k_pages and v_pages are one buffer", name);
    return AROPS_OK;
}

arops_status check_batch(const char* name, const arops_paged_batch* b, const arops_paged_cache* c,
                         int64_t tokens, bool needs_q_start)
{
    if (!b)
        return fail(AROPS_ERR_INVALID, "%s: batch is null", name);
    if (tokens < 0 || b->n_seqs < 0 || b->max_pages < 0)
        return fail(AROPS_ERR_INVALID, "%s: negative size", name);
    if (tokens > INT32_MAX || (int64_t)b->max_pages * c->page_size > kMaxPositions)
        return fail(AROPS_ERR_UNSUPPORTED,
                    "%s: supported tokens < 2^31, max_pages * page_size <= 2^31 - 1025", name);
    if (tokens == 0 || b->n_seqs == 0)
        return AROPS_OK;
    if ((needs_q_start && !b->q_start) || !b->kv_lens || (b->max_pages > 0 && !b->block_table))
        return fail(AROPS_ERR_INVALID, "%s: null batch array", name);
    return AROPS_OK;
}

// Distance between two tokens of a [tokens, heads, head_dim] operand whose
// heads are dense.
arops_status check_stride(const char* name, const char* what, int64_t stride, int64_t heads,
                          int64_t head_dim)
{
    if (stride < heads * head_dim)
        return fail(AROPS_ERR_INVALID, "%s: %s_stride %lld < heads * head_dim = %lld", name, what,
                    (long long)stride, (long long)(heads * head_dim));
    return AROPS_OK;
}

arops_status check_workspace(const char* name, const void* workspace, size_t bytes, size_t need)
{
    if (!workspace)
        return fail(AROPS_ERR_INVALID, "%s: workspace is null", name);
    if (bytes < need)
        return fail(AROPS_ERR_INVALID, "%s: workspace of %zu bytes < %zu needed", name, bytes,
                    need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return fail(AROPS_ERR_INVALID, "%s: workspace not 16-byte aligned", name);
    return AROPS_OK;
}

arops_status workspace_entry(const char* name, int64_t tokens, int32_t n_q_heads,
                             int32_t head_dim, bool shared_prefix, size_t* bytes)
{
    if (!bytes)
        return fail(AROPS_ERR_INVALID, "%s: bytes is null", name);
    if (tokens < 0 || n_q_heads < 1 || head_dim < 1)
        return fail(AROPS_ERR_INVALID, "%s: bad shape tokens=%lld n_q_heads=%d head_dim=%d", name,
                    (long long)tokens, (int)n_q_heads, (int)head_dim);
    if (tokens > INT32_MAX || n_q_heads > 65535 || head_dim > 256)
        return fail(AROPS_ERR_UNSUPPORTED,
                    "%s: supported tokens < 2^31, n_q_heads <= 65535, head_dim <= 256", name);
    *bytes = attention_workspace_bytes(tokens, n_q_heads, head_dim, shared_prefix);
    return ok();
}

// The checks and the launch that the two attention operators share.
arops_status attention_entry(const char* name, const void* q, int64_t q_stride, void* out,
                             const arops_paged_cache* cache, const arops_paged_batch* batch,
                             const arops_prefix_groups* groups,
                             const arops_attention_options* opt, int64_t tokens,
                             int32_t n_q_heads, void* workspace, size_t workspace_bytes,
                             void* stream)
{
    arops_status st = check_cache(name, cache, 256);
    if (st != AROPS_OK)
        return st;
    if (cache->dtype == AROPS_F32 && cache->head_dim > 128)
        return fail(AROPS_ERR_UNSUPPORTED, "%s: head_dim %d > 128 in fp32", name,
                    (int)cache->head_dim);
    st = check_batch(name, batch, cache, tokens, groups == nullptr);
    if (st != AROPS_OK)
        return st;
    if (batch->n_seqs > 65535 || n_q_heads > 65535)
        return fail(AROPS_ERR_UNSUPPORTED, "%s: supported n_seqs <= 65535, n_q_heads <= 65535",
                    name);
    if (n_q_heads < 1 || cache->n_kv_heads < 1 || n_q_heads % cache->n_kv_heads != 0)
        return fail(AROPS_ERR_INVALID, "%s: n_q_heads %d is not a multiple of n_kv_heads %d", name,
                    (int)n_q_heads, (int)cache->n_kv_heads);
    if (tokens * (n_q_heads / cache->n_kv_heads) > INT32_MAX)
        return fail(AROPS_ERR_UNSUPPORTED,
                    "%s: tokens * n_q_heads / n_kv_heads must be < 2^31", name);
    if (!opt)
        return fail(AROPS_ERR_INVALID, "%s: options is null", name);
    if (!isfinite(opt->scale) || !isfinite(opt->softcap) || opt->window < 0 ||
        (opt->softcap != 0.0f && !(opt->softcap >= 1e-30f)))
        return fail(AROPS_ERR_INVALID,
                    "%s: scale and softcap must be finite, softcap 0 or >= 1e-30, window >= 0",
                    name);
    st = check_stride(name, "q", q_stride, n_q_heads, cache->head_dim);
    if (st != AROPS_OK)
        return st;
    if (groups) {
        if (groups->n_groups < 0 || groups->max_prefix_pages < 0)
            return fail(AROPS_ERR_INVALID, "%s: negative size", name);
        if (opt->bidir_lens)
            return fail(AROPS_ERR_INVALID, "%s: bidir_lens must be null", name);
        if (((int64_t)groups->max_prefix_pages + batch->max_pages) * cache->page_size >
            kMaxPositions)
            return fail(AROPS_ERR_UNSUPPORTED,
                        "%s: supported (max_prefix_pages + max_pages) * page_size <= 2^31 - 1025",
                        name);
        if (groups->n_groups > batch->n_seqs)
            return fail(AROPS_ERR_INVALID, "%s: more groups (%d) than sequences (%d)", name,
                        (int)groups->n_groups, (int)batch->n_seqs);
    }
    if (tokens == 0 || batch->n_seqs == 0 || (groups && groups->n_groups == 0))
        return ok();
    if (groups && (!groups->group_start || !groups->prefix_lens ||
                   (groups->max_prefix_pages > 0 && !groups->prefix_table)))
        return fail(AROPS_ERR_INVALID, "%s: null group array", name);
    if (!q || !out)
        return fail(AROPS_ERR_INVALID, "%s: null pointer", name);
    if (q == out)
        return fail(AROPS_ERR_INVALID, "%s: q and out are one buffer", name);
    st = check_workspace(name, workspace, workspace_bytes,
                         attention_workspace_bytes(tokens, n_q_heads, cache->head_dim,
                                                   groups != nullptr));
    if (st != AROPS_OK)
        return st;
    AttentionParams p = {};
    p.q = q;
    p.out = out;
    p.k_pages = cache->k_pages;
    p.v_pages = cache->v_pages;
    p.q_start = groups ? nullptr : batch->q_start;
    p.kv_lens = batch->kv_lens;
    p.block_table = batch->block_table;
    if (groups) {
        p.group_start = groups->group_start;
        p.prefix_lens = groups->prefix_lens;
        p.prefix_table = groups->prefix_table;
        p.n_groups = groups->n_groups;
        p.max_prefix_pages = groups->max_prefix_pages;
    }
    p.slopes = opt->slopes;
    p.bidir_lens = opt->bidir_lens;
    p.q_stride = q_stride;
    p.tokens = tokens;
    p.map = make_page_map(*cache);
    p.n_seqs = batch->n_seqs;
    p.max_pages = batch->max_pages;
    p.hq = n_q_heads;
    p.hk = cache->n_kv_heads;
    p.head_dim = cache->head_dim;
    p.window = opt->window;
    p.scale = opt->scale;
    p.softcap = opt->softcap;
    cudaError_t err = device_error_word(&p.err);
    if (err != cudaSuccess)
        return from_cuda(err, name);
    return from_cuda(launch_attention(p, cache->dtype, workspace,
                                      static_cast<cudaStream_t>(stream)),
                     name);
}

}  // namespace

extern "C" {

AROPS_API arops_status arops_mrope_paged_append(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, void* q_out, int64_t q_out_stride, const arops_paged_cache* cache,
    const arops_paged_batch* batch, const void* gamma_q, const void* gamma_k, float eps,
    const int32_t* pos, int64_t tokens, int32_t n_q_heads, const int32_t* sections, float theta,
    void* stream)
{
    const char* name = "arops_mrope_paged_append";
    arops_status st = check_cache(name, cache, 512);
    if (st != AROPS_OK)
        return st;
    st = check_batch(name, batch, cache, tokens, true);
    if (st != AROPS_OK)
        return st;
    const int32_t d = cache->head_dim, hk = cache->n_kv_heads;
    if (n_q_heads < 0)
        return fail(AROPS_ERR_INVALID, "%s: negative size", name);
    if (d % 2 != 0)
        return fail(AROPS_ERR_INVALID, "%s: head_dim must be even (got %d)", name, (int)d);
    if (!sections)
        return fail(AROPS_ERR_INVALID, "%s: sections is null", name);
    if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 ||
        (int64_t)sections[0] + sections[1] + sections[2] != d / 2)
        return fail(AROPS_ERR_INVALID, "%s: sections [%d,%d,%d] must be >= 0 and sum to %d", name,
                    (int)sections[0], (int)sections[1], (int)sections[2], (int)d / 2);
    if (!(theta > 0.0f) || isinf(theta))
        return fail(AROPS_ERR_INVALID, "%s: theta must be finite and > 0", name);
    if ((gamma_q || gamma_k) && (!(eps >= 0.0f) || isinf(eps)))
        return fail(AROPS_ERR_INVALID, "%s: eps must be finite and >= 0", name);
    if ((st = check_stride(name, "q", q_stride, n_q_heads, d)) != AROPS_OK ||
        (st = check_stride(name, "q_out", q_out_stride, n_q_heads, d)) != AROPS_OK ||
        (st = check_stride(name, "k", k_stride, hk, d)) != AROPS_OK ||
        (st = check_stride(name, "v", v_stride, hk, d)) != AROPS_OK)
        return st;
    if (tokens == 0 || batch->n_seqs == 0 || (n_q_heads == 0 && hk == 0))
        return ok();
    if (!pos || (n_q_heads > 0 && (!q || !q_out)) || (hk > 0 && (!k || !v)))
        return fail(AROPS_ERR_INVALID, "%s: null pointer", name);
    if (n_q_heads > 0 && q == q_out && q_stride != q_out_stride)
        return fail(AROPS_ERR_INVALID, "%s: q_out is q with another stride", name);
    PagedAppendArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.q_start = batch->q_start;
    a.kv_lens = batch->kv_lens;
    a.block_table = batch->block_table;
    a.pos = pos;
    a.gamma_q = gamma_q;
    a.gamma_k = gamma_k;
    a.tokens = tokens;
    a.map = make_page_map(*cache);
    a.n_seqs = batch->n_seqs;
    a.max_pages = batch->max_pages;
    a.hq = n_q_heads;
    a.hk = hk;
    a.head_dim = d;
    for (int i = 0; i < 3; ++i)
        a.sections[i] = sections[i];
    a.theta = theta;
    a.eps = eps;
    return from_cuda(launch_paged_append(a, cache->dtype, static_cast<cudaStream_t>(stream)),
                     name);
}

AROPS_API arops_status arops_attention_workspace(int64_t tokens, int32_t n_q_heads,
                                                 int32_t head_dim, size_t* bytes)
{
    return workspace_entry("arops_attention_workspace", tokens, n_q_heads, head_dim, true, bytes);
}

AROPS_API arops_status arops_paged_attention_workspace(int64_t tokens, int32_t n_q_heads,
                                                       int32_t head_dim, size_t* bytes)
{
    return workspace_entry("arops_paged_attention_workspace", tokens, n_q_heads, head_dim, false,
                           bytes);
}

AROPS_API arops_status arops_attention_prepare(void* workspace, size_t workspace_bytes,
                                               void* stream)
{
    const char* name = "arops_attention_prepare";
    const arops_status st =
        check_workspace(name, workspace, workspace_bytes, attention_counter_bytes());
    if (st != AROPS_OK)
        return st;
    return from_cuda(cudaMemsetAsync(workspace, 0, attention_counter_bytes(),
                                     static_cast<cudaStream_t>(stream)),
                     name);
}

AROPS_API arops_status arops_paged_attention(const void* q, int64_t q_stride, void* out,
                                             const arops_paged_cache* cache,
                                             const arops_paged_batch* batch,
                                             const arops_attention_options* options,
                                             int64_t tokens, int32_t n_q_heads, void* workspace,
                                             size_t workspace_bytes, void* stream)
{
    return attention_entry("arops_paged_attention", q, q_stride, out, cache, batch, nullptr,
                           options, tokens, n_q_heads, workspace, workspace_bytes, stream);
}

AROPS_API arops_status arops_shared_prefix_attention(
    const void* q, int64_t q_stride, void* out, const arops_paged_cache* cache,
    const arops_paged_batch* batch, const arops_prefix_groups* groups,
    const arops_attention_options* options, int32_t n_q_heads, void* workspace,
    size_t workspace_bytes, void* stream)
{
    const char* name = "arops_shared_prefix_attention";
    if (!groups || !batch)
        return fail(AROPS_ERR_INVALID, "%s: %s is null", name, groups ? "batch" : "groups");
    return attention_entry(name, q, q_stride, out, cache, batch, groups, options, batch->n_seqs,
                           n_q_heads, workspace, workspace_bytes, stream);
}

AROPS_API arops_status arops_swiglu(const void* gate, const void* up, void* out, int64_t rows,
                                    int64_t inter, arops_dtype dtype, void* stream)
{
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "arops_swiglu: unknown dtype %d", (int)dtype);
    if (rows < 0 || inter <= 0 || (rows > 0 && inter > INT64_MAX / rows))
        return fail(AROPS_ERR_INVALID, "arops_swiglu: bad shape rows=%lld inter=%lld",
                    (long long)rows, (long long)inter);
    if (rows == 0)
        return ok();
    if (!gate || !up || !out)
        return fail(AROPS_ERR_INVALID, "arops_swiglu: null pointer");
    return from_cuda(launch_swiglu(gate, up, out, rows * inter, dtype,
                                   static_cast<cudaStream_t>(stream)),
                     "arops_swiglu");
}

}  // extern "C"

namespace {

arops_status topk_check(const char* name, int64_t rows, int64_t vocab, int32_t top_k,
                        float temperature)
{
    if (rows < 0 || vocab <= 0)
        return fail(AROPS_ERR_INVALID, "%s: bad shape rows=%lld vocab=%lld", name,
                    (long long)rows, (long long)vocab);
    if (top_k < 1 || top_k > vocab)
        return fail(AROPS_ERR_INVALID, "%s: top_k %d must be in [1, vocab]", name, (int)top_k);
    if (top_k > topk_max_k() || vocab > (int64_t)topk_max_slices() * 4096 || rows > 65535)
        return fail(AROPS_ERR_UNSUPPORTED,
                    "%s: supported top_k <= %d, vocab <= %d, rows <= 65535", name, topk_max_k(),
                    topk_max_slices() * 4096);
    if (!(temperature > 0.0f) || isinf(temperature))
        return fail(AROPS_ERR_INVALID, "%s: temperature must be finite and > 0", name);
    return AROPS_OK;
}

}  // namespace

extern "C" {

AROPS_API arops_status arops_topk_sample_workspace(int64_t rows, int64_t vocab, int32_t top_k,
                                                   size_t* bytes)
{
    if (!bytes)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample_workspace: bytes is null");
    const arops_status st = topk_check("arops_topk_sample_workspace", rows, vocab, top_k, 1.0f);
    if (st != AROPS_OK)
        return st;
    *bytes = topk_counter_bytes() +
             (size_t)rows * (size_t)topk_slices(vocab) * (size_t)top_k * sizeof(uint64_t);
    return ok();
}

AROPS_API arops_status arops_topk_sample_prepare(void* workspace, size_t workspace_bytes,
                                                 void* stream)
{
    if (!workspace)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample_prepare: workspace is null");
    if (workspace_bytes < topk_counter_bytes())
        return fail(AROPS_ERR_INVALID,
                    "arops_topk_sample_prepare: workspace of %zu bytes < the %zu bytes of counters",
                    workspace_bytes, topk_counter_bytes());
    return from_cuda(cudaMemsetAsync(workspace, 0, topk_counter_bytes(),
                                     static_cast<cudaStream_t>(stream)),
                     "arops_topk_sample_prepare");
}

AROPS_API arops_status arops_topk_sample(const void* logits, const float* gumbel,
                                         int32_t* token_out, float* prob_out, int64_t rows,
                                         int64_t vocab, int32_t top_k, float temperature,
                                         arops_dtype dtype, void* workspace,
                                         size_t workspace_bytes, void* stream)
{
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "arops_topk_sample: unknown dtype %d", (int)dtype);
    const arops_status st = topk_check("arops_topk_sample", rows, vocab, top_k, temperature);
    if (st != AROPS_OK)
        return st;
    if (rows == 0)
        return ok();
    if (!logits || !gumbel || !token_out || !prob_out || !workspace)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample: null pointer");
    const size_t need =
        topk_counter_bytes() + (size_t)rows * (size_t)topk_slices(vocab) * (size_t)top_k * 8u;
    if (workspace_bytes < need)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample: workspace of %zu bytes < %zu needed",
                    workspace_bytes, need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample: workspace not 16-byte aligned");
    return from_cuda(launch_topk_sample(logits, gumbel, token_out, prob_out, rows, vocab, top_k,
                                        temperature, dtype, workspace,
                                        static_cast<cudaStream_t>(stream)),
                     "arops_topk_sample");
}

AROPS_API arops_status arops_topk_sample_noalloc(const void* logits, const float* gumbel,
                                                 int32_t* token_out, float* prob_out,
                                                 int64_t rows, int64_t vocab, int32_t top_k,
                                                 float temperature, arops_dtype dtype,
                                                 void* stream)
{
    if (!valid_dtype(dtype))
        return fail(AROPS_ERR_INVALID, "arops_topk_sample_noalloc: unknown dtype %d", (int)dtype);
    const arops_status st =
        topk_check("arops_topk_sample_noalloc", rows, vocab, top_k, temperature);
    if (st != AROPS_OK)
        return st;
    const size_t need = (size_t)rows * (size_t)topk_slices(vocab) * (size_t)top_k * 8u;
    if (need > topk_noalloc_scratch_bytes())
        return fail(AROPS_ERR_UNSUPPORTED,
                    "arops_topk_sample_noalloc: this shape needs %zu bytes of scratch "
                    "(rows x ceil(vocab/4096) x top_k x 8) but the built-in array holds %zu; "
                    "use arops_topk_sample with a caller workspace",
                    need, topk_noalloc_scratch_bytes());
    // resolved before the rows == 0 return, so that a call with no rows is the
    // set-up call: it makes the current context load this code and its array
    void* scratch = nullptr;
    cudaError_t err = topk_noalloc_scratch(&scratch);
    if (err != cudaSuccess)
        return from_cuda(err, "arops_topk_sample_noalloc (scratch address)");
    if (rows == 0)
        return ok();
    if (!logits || !gumbel || !token_out || !prob_out)
        return fail(AROPS_ERR_INVALID, "arops_topk_sample_noalloc: null pointer");
    return from_cuda(launch_topk_sample(logits, gumbel, token_out, prob_out, rows, vocab, top_k,
                                        temperature, dtype, scratch,
                                        static_cast<cudaStream_t>(stream)),
                     "arops_topk_sample_noalloc");
}

AROPS_API arops_status arops_device_errors(uint32_t* errors, int clear)
{
    if (!errors)
        return fail(AROPS_ERR_INVALID, "arops_device_errors: errors is null");
    unsigned v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_device_errors, sizeof(v));
    if (err == cudaSuccess && clear) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_device_errors, &zero, sizeof(zero));
    }
    if (err != cudaSuccess)
        return from_cuda(err, "arops_device_errors");
    *errors = v;
    return ok();
}

AROPS_API arops_status arops_selftest_wait_timeout(uint64_t timeout_ns, int32_t* waited_out,
                                                   void* stream)
{
    if (!waited_out)
        return fail(AROPS_ERR_INVALID, "arops_selftest_wait_timeout: waited_out is null");
    if (timeout_ns == 0 || timeout_ns > 2000000000ull)
        return fail(AROPS_ERR_INVALID, "arops_selftest_wait_timeout: timeout must be in (0, 2 s]");
    return from_cuda(launch_wait_timeout_selftest(timeout_ns, waited_out,
                                                  static_cast<cudaStream_t>(stream)),
                     "arops_selftest_wait_timeout");
}

AROPS_API int arops_set_pdl(int enable)
{
    return g_pdl.exchange(enable ? 1 : 0);
}

AROPS_API int arops_set_streaming(int enable)
{
    return g_streaming.exchange(enable ? 1 : 0);
}

AROPS_API int arops_set_topk_cluster(int mode)
{
    return g_topk_cluster.exchange(mode < 0 ? 0 : (mode > 3 ? 3 : mode));
}

AROPS_API uint64_t arops_launch_count(void)
{
    return g_launches.load(std::memory_order_relaxed);
}

AROPS_API const char* arops_status_string(arops_status status)
{
    switch (status) {
    case AROPS_OK: return "ok";
    case AROPS_ERR_INVALID: return "invalid argument";
    case AROPS_ERR_UNSUPPORTED: return "unsupported size";
    case AROPS_ERR_CUDA: return "CUDA error";
    }
    return "unknown status";
}

AROPS_API const char* arops_last_error(void)
{
    return g_last_error;
}

AROPS_API int arops_version(void)
{
    return AROPS_VERSION;
}

}  // extern "C"
