// api_pages.cu -- the C ABI of the calls that keep pages and entries of the cache
// (declared in include/ternary_linear.h): argument validation, then the launches.
#include "api_util.h"

namespace {

using tl::aligned;
using tl::from_cuda;

constexpr int64_t kMaxPlaces = ((int64_t)1 << 31) - 256;
constexpr int32_t kMaxLayers = 512;
// moves of a sequence: a block looks up to five groups of 1024 ahead of one in 31 bits
constexpr int64_t kMaxMoves = ((int64_t)1 << 31) - (1 << 13);

tl_status check_pages(const tl_kv_pages *p, tl::KvPages *out) {
    if (p == nullptr) return TL_ERR_NULL;
    if (p->rows < 0 || p->rows > tl::kMaxPageRows) return TL_ERR_SHAPE;
    if (p->page_size < 16 || p->page_size % 16 != 0 || p->page_size > (1 << 20)) return TL_ERR_SHAPE;
    if (p->pages < 1 || p->pages >= (int64_t)tl::kMaxPages) return TL_ERR_SHAPE;
    if (p->max_pages < 0 || p->max_pages > kMaxPlaces / p->page_size) return TL_ERR_SHAPE;
    if (p->table_stride < p->max_pages || p->table_stride >= ((int64_t)1 << 40)) return TL_ERR_SHAPE;
    if (p->rows > 0 && (!p->refs || !p->lens || !p->held || (!p->table && p->max_pages > 0))) return TL_ERR_NULL;
    if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->held, 4)) return TL_ERR_ALIGN;
    *out = tl::KvPages{p->refs, p->table, p->lens, p->held, p->table_stride, p->pages, p->max_pages, p->rows, p->page_size};
    return TL_OK;
}

// `layers` caches of one geometry, none twice.
tl_status check_layers(const tl_kv_cache *c, int32_t layers) {
    if (layers < 0 || layers > kMaxLayers) return TL_ERR_SHAPE;
    if (layers > 0 && c == nullptr) return TL_ERR_NULL;
    for (int i = 0; i < layers; ++i) {
        tl::KvCache k;
        if (const tl_status s = tl::check_cache(c + i, &k)) return s;
        if (c[i].pages != c->pages || c[i].page_size != c->page_size || c[i].kv_heads != c->kv_heads ||
            c[i].head_dim != c->head_dim || c[i].format != c->format)
            return TL_ERR_SHAPE;
        // rows are counted in 32 bits (2^32 of 32 bytes and their scales, keys and values: beyond any memory)
        if (c[i].pages * c[i].kv_heads >= (((int64_t)1 << 32) - 1) / c[i].page_size) return TL_ERR_SHAPE;
        if (c[i].k_codes == c[i].v_codes || c[i].k_scale == c[i].v_scale) return TL_ERR_VALUE;
        for (int j = 0; j < i; ++j)
            if (c[i].k_codes == c[j].k_codes || c[i].v_codes == c[j].v_codes || c[i].k_scale == c[j].k_scale ||
                c[i].v_scale == c[j].v_scale)
                return TL_ERR_VALUE;
    }
    return TL_OK;
}

// Up to kMoveLayers layers from the first-th on.
tl::KvMove move_of(const tl_kv_cache *c, int first, int layers, int *status) {
    tl::KvMove m{};
    m.status = status;
    m.L = layers - first < tl::kMoveLayers ? layers - first : tl::kMoveLayers;
    if (m.L == 0) return m;
    m.pages = c->pages;
    m.P = c->page_size;
    m.shift = -1;
    for (int i = 4; i <= 20; ++i)
        if (m.P == 1 << i) m.shift = i;
    m.Hk = c->kv_heads;
    m.rb = c->format == TL_KV_INT4 ? c->head_dim / 2 : c->head_dim;
    for (int i = 0; i < m.L; ++i) {
        m.kc[i] = static_cast<uint8_t *>(c[first + i].k_codes);
        m.vc[i] = static_cast<uint8_t *>(c[first + i].v_codes);
        m.ks[i] = c[first + i].k_scale;
        m.vs[i] = c[first + i].v_scale;
    }
    return m;
}

// held: pages of each sequence (null: all of its table's)
tl_status compact(const tl_kv_cache *caches, int32_t layers, const int32_t *page_table, int64_t page_table_stride, int64_t max_pages,
                  const int32_t *held, const int32_t *start, const int32_t *keep, int64_t keep_stride, const int32_t *count,
                  int64_t batch, int64_t n, void *stream) {
    if (layers < 1) return TL_ERR_SHAPE;
    if (const tl_status s = check_layers(caches, layers)) return s;
    if (batch < 0 || batch > (1 << 16) || n < 0 || n > kMaxMoves) return TL_ERR_SHAPE;
    if (max_pages < 0 || max_pages > kMaxPlaces / caches->page_size) return TL_ERR_SHAPE;
    if (!tl::stride_ok(page_table_stride) || !tl::stride_ok(keep_stride)) return TL_ERR_SHAPE;
    if (batch == 0 || n == 0) return TL_OK;
    if (!start || !keep || !count || (!page_table && max_pages > 0)) return TL_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(start, 4) || !aligned(keep, 4) || !aligned(count, 4)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    tl::KvCompactArgs a{};
    a.table = page_table;
    a.table_stride = page_table_stride;
    a.max_places = max_pages * caches->page_size;
    a.start = start;
    a.keep = keep;
    a.keep_stride = keep_stride;
    a.count = count;
    a.held = held;
    a.batch = batch;
    a.n = n;
    cudaError_t e = cudaSuccess;
    for (int i = 0; e == cudaSuccess && i < layers; i += tl::kMoveLayers)
        e = tl::launch_kv_compact(move_of(caches, i, layers, d.status), a, d.sm_count, reinterpret_cast<cudaStream_t>(stream));
    return from_cuda(e);
}

}  // namespace

extern "C" {

tl_status ternary_pages_free(const tl_kv_pages *pages, const int32_t *keep, void *stream) {
    tl::KvPages g;
    if (const tl_status s = check_pages(pages, &g)) return s;
    if (g.rows == 0) return TL_OK;
    if (!keep) return TL_ERR_NULL;
    if (!aligned(keep, 4)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    return from_cuda(tl::launch_pages_free(g, keep, d.status, reinterpret_cast<cudaStream_t>(stream)));
}

tl_status ternary_pages_reserve(const tl_kv_pages *pages, const int32_t *extra, int64_t *slots,
                                int32_t width, uint8_t *ok, void *stream) {
    tl::PagesTakeArgs a{};
    if (const tl_status s = check_pages(pages, &a.g)) return s;
    if (width < 0) return TL_ERR_SHAPE;
    if (a.g.rows == 0) return TL_OK;
    if (!extra) return TL_ERR_NULL;
    if (!aligned(extra, 4) || !aligned(slots, 8)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    a.want = extra;
    a.slots = reinterpret_cast<long long *>(slots);
    a.width = width;
    if (width == 0) a.slots = nullptr;
    a.ok = ok;
    a.status = d.status;
    return from_cuda(tl::launch_pages_take(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t ternary_pages_fork_workspace(int64_t rows) {
    if (rows < 0 || rows > tl::kMaxPageRows) return -1;
    return 16 + rows * (int64_t)sizeof(tl::ForkItem);
}

tl_status ternary_pages_fork(const tl_kv_pages *pages, const int32_t *parent,
                             const tl_kv_cache *caches, int32_t layers, uint8_t *ok,
                             void *workspace, int64_t workspace_bytes, void *stream) {
    tl::PagesTakeArgs a{};
    if (const tl_status s = check_pages(pages, &a.g)) return s;
    if (const tl_status s = check_layers(caches, layers)) return s;
    if (layers > 0 && (caches->pages != a.g.pages || caches->page_size != a.g.P)) return TL_ERR_SHAPE;
    if (a.g.rows == 0) return TL_OK;
    if (!parent || !workspace) return TL_ERR_NULL;
    if (!aligned(parent, 4) || !aligned(workspace, 16)) return TL_ERR_ALIGN;
    if (workspace_bytes < ternary_pages_fork_workspace(a.g.rows)) return TL_ERR_SHAPE;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    a.want = parent;
    a.ok = ok;
    a.listed = static_cast<int *>(workspace);
    a.items = reinterpret_cast<tl::ForkItem *>(static_cast<char *>(workspace) + 16);
    a.status = d.status;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = tl::launch_pages_take(a, true, st);
    for (int i = 0; e == cudaSuccess && (i == 0 || i < layers); i += tl::kMoveLayers)
        e = tl::launch_fork_apply(move_of(caches, i, layers, d.status), a.g, a.listed, a.items, i == 0, d.sm_count, st);
    return from_cuda(e);
}

tl_status ternary_kv_copy(const tl_kv_cache *caches, int32_t layers, const int32_t *src,
                          const int32_t *dst, const int32_t *tokens, int64_t n, void *stream) {
    if (layers < 1) return TL_ERR_SHAPE;
    if (const tl_status s = check_layers(caches, layers)) return s;
    if (n < 0 || n >= ((int64_t)1 << 31)) return TL_ERR_SHAPE;
    if (n == 0) return TL_OK;
    if (!src || !dst) return TL_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(tokens, 4)) return TL_ERR_ALIGN;
    tl::CallDevice d;
    if (const int s = tl::begin_call(&d)) return (tl_status)s;
    cudaError_t e = cudaSuccess;
    for (int i = 0; e == cudaSuccess && i < layers; i += tl::kMoveLayers)
        e = tl::launch_kv_copy(move_of(caches, i, layers, d.status), src, dst, tokens, n, d.sm_count,
                               reinterpret_cast<cudaStream_t>(stream));
    return from_cuda(e);
}

tl_status ternary_kv_compact(const tl_kv_cache *caches, int32_t layers, const int32_t *page_table,
                             int64_t page_table_stride, int64_t max_pages, const int32_t *start,
                             const int32_t *keep, int64_t keep_stride, const int32_t *count,
                             int64_t batch, int64_t n, void *stream) {
    return compact(caches, layers, page_table, page_table_stride, max_pages, nullptr, start, keep, keep_stride, count, batch, n, stream);
}

tl_status ternary_pages_compact(const tl_kv_pages *pages, const tl_kv_cache *caches, int32_t layers,
                                const int32_t *start, const int32_t *keep, int64_t keep_stride,
                                const int32_t *count, int64_t n, void *stream) {
    tl::KvPages g;
    if (const tl_status s = check_pages(pages, &g)) return s;
    if (layers > 0 && caches && (caches->pages != g.pages || caches->page_size != g.P)) return TL_ERR_SHAPE;
    return compact(caches, layers, g.table, g.stride, g.max_pages, g.held, start, keep, keep_stride, count, g.rows, n, stream);
}

}  // extern "C"
