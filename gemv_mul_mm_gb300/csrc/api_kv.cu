// api_kv.cu -- the C ABI of the rotary, cache and attention operators
// (include/qmm.h): argument validation and dispatch.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "kv_common.cuh"

using namespace qmm;

namespace {

bool dtype_ok(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
int64_t esize(int t) { return t == QMM_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether rows x cols x last elements with these strides stay inside `elems`
// elements. Strides and sizes are at most 2^40, so nothing overflows.
constexpr int64_t kBig = int64_t(1) << 40;
bool fits(size_t elems, int64_t rows, int64_t rs, int64_t cols, int64_t cs, int64_t last) {
    const __int128 need = static_cast<__int128>(rows - 1) * rs + static_cast<__int128>(cols - 1) * cs + last;
    return need <= static_cast<__int128>(elems);
}

// Whether some |o + t * ts| < D with |t| < T (t = 0 not counted with `apart`).
bool comes_near(int64_t o, int64_t T, int64_t ts, int64_t D, bool apart) {
    const int64_t at = ts ? std::min(std::max(-o / ts, 1 - T), T - 1) : T > 1;
    for (int64_t t = std::max(at - 1, 1 - T); t <= std::min(at + 1, T - 1); ++t)
        if (!(apart && t == 0) && std::llabs(o + t * ts) < D) return true;
    return false;
}

// Whether two rows of Y (t, h), D elements at t * ts + h * hs, share an element.
bool rows_meet(int64_t T, int64_t ts, int64_t H, int64_t hs, int64_t D) {
    if ((H == 1 || hs >= D) && (T == 1 || ts >= (H - 1) * hs + D)) return false;   // the usual order
    if ((T == 1 || ts >= D) && (H == 1 || hs >= (T - 1) * ts + D)) return false;
    for (int64_t h = 0; h < H; ++h)
        if (comes_near(h * hs, T, ts, D, h == 0)) return true;
    return false;
}

// Whether rows of Y may be written while those of X are read, T x H rows of D
// elements each: Y is X, or they share no element. Where their ranges meet and
// their token strides differ that is not looked into.
bool apart_or_same(const void* X, int64_t x_ts, int64_t x_hs, const void* Y, int64_t y_ts, int64_t y_hs, int64_t T, int64_t H,
                   int64_t D, int64_t size) {
    const int64_t x0 = reinterpret_cast<intptr_t>(X) / size, y0 = reinterpret_cast<intptr_t>(Y) / size;
    const int64_t xn = (T - 1) * x_ts + (H - 1) * x_hs + D, yn = (T - 1) * y_ts + (H - 1) * y_hs + D;
    if (x0 + xn <= y0 || y0 + yn <= x0) return true;
    const bool same_ts = T == 1 || x_ts == y_ts, same_hs = H == 1 || x_hs == y_hs;
    if (X == Y && same_ts && same_hs) return true;
    if (!same_ts || (!same_hs && H > 1024)) return false;
    const int64_t lo = same_hs ? 1 - H : 0;          // same_hs: h is a difference of heads
    for (int64_t h = lo; h < H; ++h)
        for (int64_t g = 0; g < (same_hs ? 1 : H); ++g)
            if (comes_near(y0 - x0 + h * y_hs - g * x_hs, T, x_ts, D, false)) return false;
    return true;
}

// The rotary arguments shared by qrope and qkv_store.
int check_rope(const int32_t* pos, const uint64_t* turns, int rot, int layout, float mscale, int64_t D) {
    if (layout != QMM_ROPE_HALF && layout != QMM_ROPE_INTERLEAVED) return QMM_ERR_BAD_ARGUMENT;
    if (rot <= 0 || rot % 2 || rot > D || !std::isfinite(mscale)) return QMM_ERR_BAD_ARGUMENT;
    if (!pos || !turns) return QMM_ERR_NULL_POINTER;
    if (!aligned(pos, 4) || !aligned(turns, 8)) return QMM_ERR_MISALIGNED;
    return QMM_OK;
}

int check_cache(KvCache* c, int fmt, const void* k, const void* v, size_t cache_bytes, int64_t n_pages,
                int64_t page_stride, int page_size, int heads, int D) {
    if (fmt != QMM_KV_F16 && fmt != QMM_KV_BF16 && fmt != QMM_KV_Q8_0) return QMM_ERR_BAD_KIND;
    if (n_pages < 0 || heads < 0 || D < 0 || page_stride < 0) return QMM_ERR_BAD_ARGUMENT;
    if (n_pages == 0 || heads == 0 || D == 0) return QMM_ERR_EMPTY_SHAPE;
    if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1))) return QMM_ERR_BAD_ARGUMENT;
    if (D % 32 || D > 1024) return QMM_ERR_COLS_NOT_BLOCK_ALIGNED;
    if (n_pages > 0x7fffffff || page_stride > kBig || heads > 65536) return QMM_ERR_BAD_ARGUMENT;
    if (!k || !v) return QMM_ERR_NULL_POINTER;
    if (!aligned(k, 16) || !aligned(v, 16) || page_stride % 16) return QMM_ERR_MISALIGNED;
    c->k = static_cast<uint8_t*>(const_cast<void*>(k));
    c->v = static_cast<uint8_t*>(const_cast<void*>(v));
    c->fmt = fmt;
    c->page_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    c->heads = heads;
    c->D = D;
    c->n_pages = n_pages;
    c->page_stride = page_stride;
    const int64_t page = c->unit() * heads;
    if (page_stride < page) return QMM_ERR_CACHE_TOO_SMALL;
    if (static_cast<__int128>(n_pages - 1) * page_stride + page > static_cast<__int128>(cache_bytes))
        return QMM_ERR_CACHE_TOO_SMALL;
    return QMM_OK;
}

// attn_plan on the current device. A thread's last plan is kept with its sizes:
// a workspace query and its call, and the layers of one step, share it.
int plan_for(int fmt, int dtype, int64_t B, int Hq, int Hkv, int D, int max_len, int window, AttnPlan* p) {
    struct Key {
        int64_t B;
        int dev, fmt, dtype, Hq, Hkv, D, max_len, window;
        bool operator==(const Key& o) const {
            return B == o.B && dev == o.dev && fmt == o.fmt && dtype == o.dtype && Hq == o.Hq && Hkv == o.Hkv && D == o.D &&
                   max_len == o.max_len && window == o.window;
        }
    };
    static thread_local Key last{};      // B 0: none
    static thread_local AttnPlan plan{};
    Key k{B, 0, fmt, dtype, Hq, Hkv, D, max_len, window};
    if (cudaGetDevice(&k.dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (!(k == last)) {
        last.B = 0;
        if (attn_plan(fmt, dtype, B, Hq, Hkv, D, max_len, window, sm_count(k.dev), &plan) != cudaSuccess) return QMM_ERR_CUDA;
        last = k;
    }
    *p = plan;
    return QMM_OK;
}

// The same for sizes that are not checked yet; false where qattn_decode would
// refuse them.
bool plan_of(int fmt, int dtype, int64_t B, int Hq, int Hkv, int D, int max_len, int window, AttnPlan* p) {
    if ((fmt != QMM_KV_F16 && fmt != QMM_KV_BF16 && fmt != QMM_KV_Q8_0) || !dtype_ok(dtype)) return false;
    if (B <= 0 || B > (1 << 24) || Hq <= 0 || Hq > 65536 || Hkv <= 0 || Hq % Hkv || !attn_dim_ok(D) || max_len <= 0 ||
        max_len > (1 << 30) || window < 0)
        return false;
    return plan_for(fmt, dtype, B, Hq, Hkv, D, max_len, window, p) == QMM_OK;
}

int done(cudaError_t e, int path) {
    if (e != cudaSuccess) return QMM_ERR_CUDA;
    set_last_path(path);
    return QMM_OK;
}

}  // namespace

extern "C" {

size_t qkv_page_bytes(int fmt, int page_size, int n_kv_heads, int head_dim) {
    if (fmt != QMM_KV_F16 && fmt != QMM_KV_BF16 && fmt != QMM_KV_Q8_0) return 0;
    if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)) || n_kv_heads <= 0 || n_kv_heads > 65536 ||
        head_dim <= 0 || head_dim % 32 || head_dim > 1024)
        return 0;
    return kv_row_bytes(fmt, head_dim) * static_cast<size_t>(page_size) * static_cast<size_t>(n_kv_heads);
}

int qrope_turns(double base, int rot_dim, int scaling, double factor, double orig_len, double fast, double slow,
                uint64_t* turns, float* mscale) {
    if (!turns || !mscale) return QMM_ERR_NULL_POINTER;
    if (rot_dim <= 0 || rot_dim % 2 || rot_dim > (1 << 20)) return QMM_ERR_BAD_ARGUMENT;
    if (!(base > 1.0) || !std::isfinite(base)) return QMM_ERR_BAD_ARGUMENT;
    if (scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_BANDS) return QMM_ERR_BAD_ARGUMENT;
    if (scaling != QMM_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return QMM_ERR_BAD_ARGUMENT;
    if (scaling == QMM_ROPE_BASE && rot_dim == 2) return QMM_ERR_BAD_ARGUMENT;
    if (scaling >= QMM_ROPE_RAMP &&
        (!(orig_len > 0.0) || !std::isfinite(orig_len) || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return QMM_ERR_BAD_ARGUMENT;
    const double two_pi = 6.283185307179586476925286766559;
    const int n = rot_dim / 2;
    if (scaling == QMM_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    double lo = 0.0, hi = 0.0;   // RAMP: pairs up to lo are kept, from hi on divided
    if (scaling == QMM_ROPE_RAMP) {
        // the pair whose frequency makes r turns in orig_len positions
        auto pair_of = [&](double r) { return rot_dim * std::log(orig_len / (r * two_pi)) / (2.0 * std::log(base)); };
        lo = std::fmax(std::floor(pair_of(fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(slow)), rot_dim - 1.0);
    }
    for (int i = 0; i < n; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == QMM_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == QMM_ROPE_RAMP) {
            const double x = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f / factor * x + f * (1.0 - x);
        } else if (scaling == QMM_ROPE_BANDS) {
            const double turns_in_len = orig_len * f / two_pi;
            const double x = std::fmin(std::fmax((turns_in_len - slow) / (fast - slow), 0.0), 1.0);
            f = f / factor * (1.0 - x) + f * x;
        }
        // below 1/(2 pi) of a turn: no overflow
        turns[i] = static_cast<uint64_t>(std::rint(std::ldexp(f / two_pi, 64)));
    }
    *mscale = scaling == QMM_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    return QMM_OK;
}

int qrope(const void* X, int dtype, size_t x_elems, int64_t x_ts, int64_t x_hs, const int32_t* positions,
          const uint64_t* turns, int rot_dim, int layout, float mscale, void* Y, size_t y_elems, int64_t y_ts,
          int64_t y_hs, int64_t T, int64_t H, int64_t D, void* stream) {
    if (!dtype_ok(dtype)) return QMM_ERR_BAD_DTYPE;
    if (T < 0 || H < 0 || D < 0 || x_ts < 0 || x_hs < 0 || y_ts < 0 || y_hs < 0) return QMM_ERR_BAD_ARGUMENT;
    if (T == 0 || H == 0 || D == 0) return QMM_ERR_EMPTY_SHAPE;
    if (T > kBig || H > 65536 || D > 2048 || x_ts > kBig || x_hs > kBig || y_ts > kBig || y_hs > kBig)
        return QMM_ERR_BAD_ARGUMENT;
    if (!X || !Y) return QMM_ERR_NULL_POINTER;
    if (!aligned(X, esize(dtype)) || !aligned(Y, esize(dtype))) return QMM_ERR_MISALIGNED;
    if (int r = check_rope(positions, turns, rot_dim, layout, mscale, D)) return r;
    if (!fits(x_elems, T, x_ts, H, x_hs, D)) return QMM_ERR_ACTIVATIONS_TOO_SMALL;
    if (!fits(y_elems, T, y_ts, H, y_hs, D)) return QMM_ERR_OUTPUT_TOO_SMALL;
    if (rows_meet(T, y_ts, H, y_hs, D) || !apart_or_same(X, x_ts, x_hs, Y, y_ts, y_hs, T, H, D, esize(dtype)))
        return QMM_ERR_BAD_ARGUMENT;
    RopeArgs a;
    a.X = X;
    a.Y = Y;
    a.dtype = dtype;
    a.x_ts = x_ts;
    a.x_hs = x_hs;
    a.y_ts = y_ts;
    a.y_hs = y_hs;
    a.pos = positions;
    a.turns = turns;
    a.rot = rot_dim;
    a.layout = layout;
    a.mscale = mscale;
    a.T = T;
    a.H = H;
    a.D = D;
    return done(launch_rope(a, static_cast<cudaStream_t>(stream)), 8);
}

int qkv_store(int fmt, const void* K, size_t k_elems, int64_t k_ts, int64_t k_hs, const void* V, size_t v_elems,
              int64_t v_ts, int64_t v_hs, int dtype, const int64_t* slots, const int32_t* positions,
              const uint64_t* turns, int rot_dim, int layout, float mscale, void* k_cache, void* v_cache,
              size_t cache_bytes, int64_t n_pages, int64_t page_stride, int page_size, int64_t T, int n_kv_heads,
              int head_dim, void* stream) {
    KvStoreArgs a;
    if (!dtype_ok(dtype)) return QMM_ERR_BAD_DTYPE;
    if (int r = check_cache(&a.c, fmt, k_cache, v_cache, cache_bytes, n_pages, page_stride, page_size, n_kv_heads,
                            head_dim))
        return r;
    if (T < 0 || k_ts < 0 || k_hs < 0 || v_ts < 0 || v_hs < 0) return QMM_ERR_BAD_ARGUMENT;
    if (T == 0) return QMM_ERR_EMPTY_SHAPE;
    if (T > kBig || k_ts > kBig || k_hs > kBig || v_ts > kBig || v_hs > kBig) return QMM_ERR_BAD_ARGUMENT;
    if (!K || !V || !slots) return QMM_ERR_NULL_POINTER;
    if (!aligned(K, esize(dtype)) || !aligned(V, esize(dtype)) || !aligned(slots, 8)) return QMM_ERR_MISALIGNED;
    if (positions || turns) {
        if (int r = check_rope(positions, turns, rot_dim, layout, mscale, head_dim)) return r;
    }
    if (!fits(k_elems, T, k_ts, n_kv_heads, k_hs, head_dim) || !fits(v_elems, T, v_ts, n_kv_heads, v_hs, head_dim))
        return QMM_ERR_ACTIVATIONS_TOO_SMALL;
    a.K = K;
    a.V = V;
    a.dtype = dtype;
    a.k_ts = k_ts;
    a.k_hs = k_hs;
    a.v_ts = v_ts;
    a.v_hs = v_hs;
    a.slots = slots;
    a.pos = positions;
    a.turns = turns;
    a.rot = positions ? rot_dim : 0;
    a.layout = layout;
    a.mscale = mscale;
    a.T = T;
    if (int r = device_latch(&a.err)) return r;
    return done(launch_kv_store(a, static_cast<cudaStream_t>(stream)), 9);
}

int qkv_load(int fmt, const int64_t* slots, const void* k_cache, const void* v_cache, size_t cache_bytes,
             int64_t n_pages, int64_t page_stride, int page_size, void* K, void* V, int dtype, size_t kv_elems,
             int64_t T, int n_kv_heads, int head_dim, void* stream) {
    KvLoadArgs a;
    if (!dtype_ok(dtype)) return QMM_ERR_BAD_DTYPE;
    if (int r = check_cache(&a.c, fmt, k_cache, v_cache, cache_bytes, n_pages, page_stride, page_size, n_kv_heads,
                            head_dim))
        return r;
    if (T < 0) return QMM_ERR_BAD_ARGUMENT;
    if (T == 0) return QMM_ERR_EMPTY_SHAPE;
    if (T > kBig) return QMM_ERR_BAD_ARGUMENT;
    if (!K || !V || !slots) return QMM_ERR_NULL_POINTER;
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8)) return QMM_ERR_MISALIGNED;
    if (!fits(kv_elems, T, static_cast<int64_t>(n_kv_heads) * head_dim, n_kv_heads, head_dim, head_dim))
        return QMM_ERR_OUTPUT_TOO_SMALL;
    a.slots = slots;
    a.K = K;
    a.V = V;
    a.dtype = dtype;
    a.T = T;
    if (int r = device_latch(&a.err)) return r;
    return done(launch_kv_load(a, static_cast<cudaStream_t>(stream)), 10);
}

size_t qattn_decode_workspace_bytes(int fmt, int dtype, int64_t B, int n_q_heads, int n_kv_heads, int head_dim,
                                    int max_len, int window) {
    AttnPlan p;
    return plan_of(fmt, dtype, B, n_q_heads, n_kv_heads, head_dim, max_len, window, &p) ? p.ws_bytes : 0;
}

int qattn_decode_splits(int fmt, int dtype, int64_t B, int n_q_heads, int n_kv_heads, int head_dim, int max_len, int window) {
    AttnPlan p;
    return plan_of(fmt, dtype, B, n_q_heads, n_kv_heads, head_dim, max_len, window, &p) ? p.splits : 0;
}

int qattn_decode(int fmt, const void* q, int dtype, size_t q_elems, int64_t q_bs, int64_t q_hs, const void* k_cache,
                 const void* v_cache, size_t cache_bytes, int64_t n_pages, int64_t page_stride, int page_size,
                 const int32_t* block_table, size_t table_elems, int64_t table_stride, int table_width,
                 const int32_t* seq_lens, int max_len, int64_t B, int n_q_heads, int n_kv_heads, int head_dim,
                 float scale, int window, float softcap, void* out, size_t out_elems, float* lse, void* workspace,
                 size_t workspace_bytes, void* stream) {
    AttnArgs a;
    if (!dtype_ok(dtype)) return QMM_ERR_BAD_DTYPE;
    if (int r = check_cache(&a.c, fmt, k_cache, v_cache, cache_bytes, n_pages, page_stride, page_size, n_kv_heads,
                            head_dim))
        return r;
    if (B < 0 || n_q_heads < 0 || max_len < 0 || window < 0 || q_bs < 0 || q_hs < 0 || table_stride < 0 ||
        table_width < 0)
        return QMM_ERR_BAD_ARGUMENT;
    if (B == 0 || n_q_heads == 0 || max_len == 0 || table_width == 0) return QMM_ERR_EMPTY_SHAPE;
    if (B > (1 << 24) || n_q_heads > 65536 || max_len > (1 << 30) || q_bs > kBig || q_hs > kBig || table_stride > kBig)
        return QMM_ERR_BAD_ARGUMENT;
    if (n_q_heads % n_kv_heads || !std::isfinite(scale) || !(softcap >= 0.f) || !std::isfinite(softcap))
        return QMM_ERR_BAD_ARGUMENT;
    if (max_len > static_cast<int64_t>(table_width) * page_size) return QMM_ERR_BAD_ARGUMENT;
    if (!attn_dim_ok(head_dim)) return QMM_ERR_UNIMPLEMENTED;
    if (!q || !block_table || !seq_lens || !out) return QMM_ERR_NULL_POINTER;
    if (!aligned(q, esize(dtype)) || !aligned(out, esize(dtype)) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return QMM_ERR_MISALIGNED;
    if (!fits(q_elems, B, q_bs, n_q_heads, q_hs, head_dim) || !fits(table_elems, B, table_stride, 1, 0, table_width))
        return QMM_ERR_ACTIVATIONS_TOO_SMALL;
    if (!fits(out_elems, B, static_cast<int64_t>(n_q_heads) * head_dim, n_q_heads, head_dim, head_dim))
        return QMM_ERR_OUTPUT_TOO_SMALL;
    if (!apart_or_same(q, q_bs, q_hs, out, static_cast<int64_t>(n_q_heads) * head_dim, head_dim, B, n_q_heads, head_dim,
                       esize(dtype)))
        return QMM_ERR_BAD_ARGUMENT;
    AttnPlan p;
    if (int r = plan_for(fmt, dtype, B, n_q_heads, n_kv_heads, head_dim, max_len, window, &p)) return r;
    if (p.splits > 1) {
        if (!workspace) return QMM_ERR_NULL_POINTER;
        if (workspace_bytes < p.ws_bytes) return QMM_ERR_WORKSPACE_TOO_SMALL;
    }
    a.q = q;
    a.dtype = dtype;
    a.q_bs = q_bs;
    a.q_hs = q_hs;
    a.table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.lens = seq_lens;
    a.max_len = max_len;
    a.B = B;
    a.Hq = n_q_heads;
    a.scale = scale;
    a.softcap = softcap;
    a.window = window;
    a.out = out;
    a.lse = lse;
    a.ws = workspace;
    if (int r = device_latch(&a.err)) return r;
    return done(launch_attn(a, p, static_cast<cudaStream_t>(stream)), 11);
}

}  // extern "C"
