// C ABI of the rotation, the append to a paged cache and the attention over it:
// argument checks, kernel choice and launches.
#include <cuda_runtime.h>

#include <climits>
#include <initializer_list>
#include <cmath>
#include <cstdint>

#include "../../include/sparse_attn.h"
#include "sm100.cuh"
#include "cached_sm100.cuh"
#include "rotary_sm100.cuh"
#include "runtime.h"

namespace sa {
namespace {

// One extent of a view and its stride: not negative, whole 16-byte units, and
// not 0 where a written tensor has more than one element along it.
int stride_status(int64_t stride, int64_t extent, bool written)
{
    if (extent <= 1) return SA_OK;
    if (stride < 0 || (written && stride == 0)) return SA_ERR_INVALID_ARG;
    return stride % 8 ? SA_ERR_MISALIGNED : SA_OK;
}

int view_status(const sa_view* v, int64_t B, int64_t H, int64_t T, bool written)
{
    if (!v || !v->data) return SA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(v->data) & 15u) return SA_ERR_MISALIGNED;
    if (int rc = stride_status(v->batch_stride, B, written)) return rc;
    if (int rc = stride_status(v->head_stride, H, written)) return rc;
    return stride_status(v->token_stride, T, written);
}

// A stride along an extent of one is never multiplied by anything but 0.
RotView rot_view(const sa_view& v, int64_t B, int64_t H, int64_t T)
{
    return RotView{static_cast<__nv_bfloat16*>(v.data), B > 1 ? v.batch_stride : 0, H > 1 ? v.head_stride : 0,
                   T > 1 ? v.token_stride : 0};
}

int rotary_status(const sa_rotary* r, int32_t D)
{
    if (!r || r->n_pairs < 0 || 2 * int64_t(r->n_pairs) > D || r->n_axes < 1 || r->n_axes > kMaxAxes ||
        (r->interleaved != 0 && r->interleaved != 1) || (r->n_pairs > 0 && !r->freq))
        return SA_ERR_INVALID_ARG;
    for (int i = 0; i < r->n_pairs; i++) {
        if (!std::isfinite(r->freq[i])) return SA_ERR_INVALID_ARG;
        if (r->axis && (r->axis[i] < 0 || r->axis[i] >= r->n_axes)) return SA_ERR_INVALID_ARG;
    }
    return SA_OK;
}

RotSpec rot_spec(const sa_rotary* r)
{
    RotSpec s{};
    if (!r) return s;
    s.n_pairs = r->n_pairs;
    for (int i = 0; i < r->n_pairs; i++) {
        s.turns[i] = r->freq[i] * 0.15915494309189533576888376337251;  // 1 / 2 pi
        s.axis[i] = static_cast<uint8_t>(r->axis ? r->axis[i] : 0);
    }
    return s;
}

template <int D, bool PAGED>
int rot_launch(const RotSpec& spec, const RotParams& p, bool inter, cudaStream_t st)
{
    const int V = inter || spec.n_pairs % 8 == 0 ? 8 : spec.n_pairs % 2 == 0 ? 2 : 1;
    const int64_t blocks = (p.rows * (D / (2 * V)) + kRotThreads - 1) / kRotThreads;
    if (blocks > INT_MAX) return SA_ERR_UNSUPPORTED;
    const int heads = p.Hq + p.Hk + p.Hv;
    RotParams pp = p;
    // heads of one thread: as many as leave each SM eight blocks, so that the sines are taken few
    // times, and no fewer than one batch of loads
    const int64_t want = 8 * int64_t(device_sm_count());
    const int64_t parts = blocks >= want ? 1 : (want + blocks - 1) / blocks;
    int64_t per = (heads + parts - 1) / parts;
    per = (per + kRotUnroll - 1) / kRotUnroll * kRotUnroll;
    pp.heads_per = static_cast<int32_t>(per);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + per - 1) / per));
    if (grid.y > 65535) return SA_ERR_UNSUPPORTED;
    if (inter)
        rotary_kernel<D, 8, true, PAGED><<<grid, kRotThreads, 0, st>>>(spec, pp);
    else if (V == 8)
        rotary_kernel<D, 8, false, PAGED><<<grid, kRotThreads, 0, st>>>(spec, pp);
    else if (V == 2)
        rotary_kernel<D, 2, false, PAGED><<<grid, kRotThreads, 0, st>>>(spec, pp);
    else
        rotary_kernel<D, 1, false, PAGED><<<grid, kRotThreads, 0, st>>>(spec, pp);
    return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

int page_shift_of(int32_t page_size)
{
    for (int s = 4; s <= 8; s++)
        if (page_size == 1 << s) return s;
    return -1;
}

int cache_status(const sa_kv_cache* c)
{
    if (!c || c->n_pages < 0 || c->Hkv < 0 || c->D <= 0) return SA_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128) return SA_ERR_UNSUPPORTED;
    if (page_shift_of(c->page_size) < 0) return SA_ERR_UNSUPPORTED;
    if (c->n_pages == 0 || c->Hkv == 0) return SA_OK;
    const sa_view k{c->k, c->page_stride, c->head_stride, c->token_stride};
    const sa_view v{c->v, c->page_stride, c->head_stride, c->token_stride};
    if (int rc = view_status(&k, c->n_pages, c->Hkv, c->page_size, true)) return rc;
    return view_status(&v, c->n_pages, c->Hkv, c->page_size, true);
}

int batch_status(const sa_cache_batch* b, const sa_kv_cache* c)
{
    if (!b || b->B < 0 || b->T < 0 || b->max_q < 0 || b->max_pages < 0 || b->table_stride < 0) return SA_ERR_INVALID_ARG;
    if (b->B == 0 || b->T == 0) return SA_OK;
    if (!b->q_start || !b->kv_len || (b->max_pages > 0 && !b->table)) return SA_ERR_INVALID_ARG;
    if (b->B > 1 && b->table_stride < b->max_pages) return SA_ERR_INVALID_ARG;
    if (int64_t(b->max_pages) * c->page_size > INT_MAX / 2) return SA_ERR_UNSUPPORTED;  // positions are 32 bits
    return SA_OK;
}

// The arrays a kernel follows are readable by the current device.
int device_arrays(std::initializer_list<const void*> arrays)
{
    for (const void* a : arrays)
        if (a)
            if (int rc = check_device_array(a)) return rc;
    return SA_OK;
}

}  // namespace
}  // namespace sa

extern "C" int sparse_attn_rotary(const sa_view* q, const sa_view* k, const int32_t* positions,
                                  int64_t pos_axis_stride, int64_t pos_batch_stride, const sa_rotary* rotary,
                                  const sa_shape* shape, int32_t backward, const sa_view* q_out, const sa_view* k_out,
                                  void* stream)
{
    using namespace sa;
    if (!shape || (k == nullptr) != (k_out == nullptr) || (backward != 0 && backward != 1)) return SA_ERR_INVALID_ARG;
    const sa_shape s = *shape;
    const int32_t Hk = k ? s.Hkv : 0;
    if (s.B < 0 || s.Hq < 0 || Hk < 0 || s.N < 0 || s.D <= 0) return SA_ERR_INVALID_ARG;
    if (s.D != 64 && s.D != 128) return SA_ERR_UNSUPPORTED;
    if (int rc = rotary_status(rotary, s.D)) return rc;
    if (s.B == 0 || s.N == 0 || s.Hq + Hk == 0) return SA_OK;
    if (pos_axis_stride < 0 || pos_batch_stride < 0 || !positions) return SA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(positions) & 3u) return SA_ERR_MISALIGNED;
    RotParams p{};
    if (s.Hq > 0) {
        if (int rc = view_status(q, s.B, s.Hq, s.N, false)) return rc;
        if (int rc = view_status(q_out, s.B, s.Hq, s.N, true)) return rc;
        p.q = rot_view(*q, s.B, s.Hq, s.N);
        p.qo = rot_view(*q_out, s.B, s.Hq, s.N);
    }
    if (Hk > 0) {
        if (int rc = view_status(k, s.B, Hk, s.N, false)) return rc;
        if (int rc = view_status(k_out, s.B, Hk, s.N, true)) return rc;
        p.k = rot_view(*k, s.B, Hk, s.N);
        p.ko = rot_view(*k_out, s.B, Hk, s.N);
    }
    if (int rc = device_arrays({positions})) return rc;
    p.Hq = s.Hq;
    p.Hk = Hk;
    p.rows = int64_t(s.B) * s.N;
    p.N = s.N;
    p.pos = positions;
    p.pos_axis = pos_axis_stride;
    p.pos_batch = pos_batch_stride;
    p.sign = backward ? -1.f : 1.f;
    const RotSpec spec = rot_spec(rotary);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return s.D == 128 ? rot_launch<128, false>(spec, p, rotary->interleaved, st)
                      : rot_launch<64, false>(spec, p, rotary->interleaved, st);
}

extern "C" int sparse_attn_cache_append(const sa_view* k, const sa_view* v, const sa_kv_cache* cache,
                                        const sa_cache_batch* batch, const sa_rotary* rotary,
                                        const int32_t* positions, int64_t pos_axis_stride, int32_t pos_offset,
                                        const sa_view* q, const sa_view* q_out, int32_t Hq, void* stream)
{
    using namespace sa;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch, cache)) return rc;
    if (rotary)
        if (int rc = rotary_status(rotary, cache->D)) return rc;
    if ((q == nullptr) != (q_out == nullptr) || (q && (!rotary || Hq < 0)) || pos_axis_stride < 0 || pos_offset < 0 ||
        (positions && !rotary))
        return SA_ERR_INVALID_ARG;
    if (pos_offset > INT_MAX / 2) return SA_ERR_UNSUPPORTED;  // a token's position is 32 bits
    const int32_t B = batch->B, T = batch->T, Hkv = cache->n_pages > 0 ? cache->Hkv : 0;
    const int32_t H = q ? Hq : 0;
    if (B == 0 || T == 0 || H + Hkv == 0) return SA_OK;
    RotParams p{};
    if (Hkv > 0) {
        if (int rc = view_status(k, 1, Hkv, T, false)) return rc;
        if (int rc = view_status(v, 1, Hkv, T, false)) return rc;
        p.k = rot_view(*k, 1, Hkv, T);
        p.v = rot_view(*v, 1, Hkv, T);
    }
    if (H > 0) {
        if (int rc = view_status(q, 1, H, T, false)) return rc;
        if (int rc = view_status(q_out, 1, H, T, true)) return rc;
        p.q = rot_view(*q, 1, H, T);
        p.qo = rot_view(*q_out, 1, H, T);
    }
    if (reinterpret_cast<uintptr_t>(positions) & 3u) return SA_ERR_MISALIGNED;
    if (int rc = device_arrays({batch->q_start, batch->kv_len, batch->table, positions})) return rc;
    p.ko = rot_view(sa_view{cache->k, cache->page_stride, cache->head_stride, cache->token_stride}, cache->n_pages,
                    Hkv, cache->page_size);
    p.vo = static_cast<__nv_bfloat16*>(cache->v);
    p.Hq = H;
    p.Hk = p.Hv = Hkv;
    p.rows = T;
    p.N = T;
    p.pos = positions;
    p.pos_axis = pos_axis_stride;
    p.sign = 1.f;
    p.B = B;
    p.n_pages = cache->n_pages;
    p.page_shift = page_shift_of(cache->page_size);
    p.max_pages = batch->max_pages;
    p.pos_offset = pos_offset;
    p.table_stride = batch->table_stride;
    p.q_start = batch->q_start;
    p.kv_len = batch->kv_len;
    p.table = batch->table;
    const RotSpec spec = rot_spec(rotary);
    const bool inter = rotary && rotary->interleaved;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cache->D == 128 ? rot_launch<128, true>(spec, p, inter, st) : rot_launch<64, true>(spec, p, inter, st);
}

namespace sa {
namespace {

size_t cached_bytes(int32_t T, int32_t Hq, int32_t D) { return 256; }

int workspace_status(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (!bytes || T < 0 || Hq < 0 || Hkv < 0 || D <= 0) return SA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SA_ERR_UNSUPPORTED;
    if (Hq > 0 && (Hkv == 0 || Hq % Hkv)) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

int fwd_paged(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch, const int32_t* prefix_table,
              int32_t prefix_len, const sa_pattern* pattern, int32_t Hq, float scale, const sa_view* o, float* lse,
              void* workspace, size_t workspace_bytes, size_t need, void* stream)
{
    if (!pattern || Hq < 0 || prefix_len < 0) return SA_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch, cache)) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return SA_ERR_INVALID_ARG;
    if (int rc = check_pattern(*pattern)) return rc;
    if (pattern->causal != 1 || pattern->stride > 0 || pattern->area > 0) return SA_ERR_UNSUPPORTED;
    if (prefix_len > INT_MAX / 2) return SA_ERR_UNSUPPORTED;
    const int32_t T = batch->T;
    if (batch->B == 0 || T == 0 || Hq == 0) return SA_OK;
    if (cache->Hkv == 0 || Hq % cache->Hkv) return SA_ERR_UNSUPPORTED;
    if (prefix_len > 0 && !prefix_table) return SA_ERR_INVALID_ARG;
    if (int rc = view_status(q, 1, Hq, T, false)) return rc;
    if (int rc = view_status(o, 1, Hq, T, true)) return rc;
    if (!lse || !workspace) return SA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return SA_ERR_MISALIGNED;
    if (workspace_bytes < need) return SA_ERR_BUFFER_TOO_SMALL;
    if (int rc = device_arrays({batch->q_start, batch->kv_len, batch->table, prefix_len > 0 ? prefix_table : nullptr}))
        return rc;
    CachedParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q->data);
    p.q_token = T > 1 ? q->token_stride : 0;
    p.q_head = Hq > 1 ? q->head_stride : 0;
    p.o = static_cast<__nv_bfloat16*>(o->data);
    p.o_token = T > 1 ? o->token_stride : 0;
    p.o_head = Hq > 1 ? o->head_stride : 0;
    p.lse = lse;
    p.k = static_cast<const __nv_bfloat16*>(cache->k);
    p.v = static_cast<const __nv_bfloat16*>(cache->v);
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.token_stride = cache->token_stride;
    p.n_pages = cache->n_pages;
    p.page_shift = page_shift_of(cache->page_size);
    p.max_pages = batch->max_pages;
    p.table_stride = batch->table_stride;
    p.q_start = batch->q_start;
    p.kv_len = batch->kv_len;
    p.table = batch->table;
    p.prefix_table = prefix_table;
    p.prefix_len = prefix_len;
    p.B = batch->B;
    p.T = T;
    p.Hq = Hq;
    p.group = Hq / cache->Hkv;
    p.window = pattern->window;
    p.n_global = pattern->n_global;
    p.cols = pattern->sinks > pattern->n_global ? pattern->sinks : pattern->n_global;
    p.scale_log2 = scale * 1.44269504088896340736f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(T, Hq);
    if (cache->D == 128)
        cached_plain_kernel<128><<<grid, 128, 0, st>>>(p);
    else
        cached_plain_kernel<64><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace
}  // namespace sa

extern "C" int sparse_attn_fwd_cached_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (int rc = sa::workspace_status(T, Hq, Hkv, D, bytes)) return rc;
    *bytes = sa::cached_bytes(T, Hq, D);
    return SA_OK;
}

extern "C" int sparse_attn_fwd_shared_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (int rc = sa::workspace_status(T, Hq, Hkv, D, bytes)) return rc;
    *bytes = sa::cached_bytes(T, Hq, D);
    return SA_OK;
}

extern "C" int sparse_attn_fwd_cached(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch,
                                      const sa_pattern* pattern, int32_t Hq, float scale, const sa_view* o, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (!batch || !cache) return SA_ERR_INVALID_ARG;
    return sa::fwd_paged(q, cache, batch, nullptr, 0, pattern, Hq, scale, o, lse, workspace, workspace_bytes,
                         sa::cached_bytes(batch->T, Hq, cache->D), stream);
}

extern "C" int sparse_attn_fwd_shared(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch,
                                      const int32_t* prefix_table, int32_t prefix_len, const sa_pattern* pattern,
                                      int32_t Hq, float scale, const sa_view* o, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream)
{
    if (!batch || !cache) return SA_ERR_INVALID_ARG;
    return sa::fwd_paged(q, cache, batch, prefix_table, prefix_len, pattern, Hq, scale, o, lse, workspace,
                         workspace_bytes, sa::cached_bytes(batch->T, Hq, cache->D), stream);
}
