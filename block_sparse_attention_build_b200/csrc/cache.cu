// C ABI of the rotation, the append to a paged cache and the attention over it:
// argument checks, kernel choice and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <cmath>
#include <cstdint>

#include "../../include/sparse_attn.h"
#include "chunk_sm100.cuh"
#include "decode_sm100.cuh"
#include "rotary_sm100.cuh"
#include "runtime.h"
#include "tma_host.h"

namespace sa {
namespace {

constexpr int kMaxDevices = 64;

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
        // freq / 2 pi modulo 1 as a 64-bit fraction, whose low bit stays 0 (whole turns drop out: positions are
        // whole numbers).  Done for every call, so without a division or a call of floor.
        long double turns = static_cast<long double>(r->freq[i]) * 0.159154943091895335768883763372514362L;
        if (fabsl(turns) >= 0x1p62L) turns = fmodl(turns, 1.0L);
        const long double frac = turns - static_cast<long double>(static_cast<int64_t>(turns));  // in (-1, 1)
        s.turns[i] = static_cast<uint64_t>(static_cast<int64_t>(frac * 0x1p63L)) << 1;
        s.axis[i] = static_cast<uint8_t>(r->axis ? r->axis[i] : 0);
    }
    return s;
}

// A launch that may be set up while the stream's previous kernel still runs; the kernel waits for that one
// before its first access to memory.  In clusters of `cluster`.
template <typename... Args>
int launch_after(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, const Args&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        n++;
    }
    cfg.attrs = at;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int D, bool PAGED>
int rot_launch(const RotSpec& spec, const RotParams& p, bool inter, cudaStream_t st)
{
    const RotLayout layout = inter ? kInterleaved : spec.n_pairs % 8 == 0 ? kHalves : kShuffled;
    const int64_t blocks = (p.rows * (D / (layout == kShuffled ? 4 : 16)) + kRotThreads - 1) / kRotThreads;
    if (blocks > INT_MAX) return SA_ERR_UNSUPPORTED;
    const int heads = p.Hq + p.Hk + p.Hv;
    RotParams pp = p;
    // Heads of one thread.  Few tokens: as many parts as the SMs hold blocks, so that all have work, and
    // three at least.  Many: parts that make three rounds of blocks, whose ends then even out, but no fewer
    // than 16 heads, over which the sines are shared.  16 + 16 heads of 128 at 8192 tokens (512 blocks of the
    // 888 held at once): 1 or 3 parts 27.6 us a call, 8 parts 29.9; an append of 64 + 8 + 8 heads of 64 at
    // 12900 tokens (408 blocks): 2 parts 55.7, 3 51.2, 8 50.1; 64 + 8 heads of 64 at 2 x 16384 (1024 blocks):
    // 1 part 109 us, 3 parts 99, 18 parts 111.
    const int64_t held = int64_t(rot_blocks(layout)) * device_sm_count();
    const bool few = 3 * blocks <= 2 * held;
    const int64_t parts = few ? (held / blocks > 3 ? held / blocks : 3) : (3 * held + blocks - 1) / blocks;
    int64_t per = (heads + parts - 1) / parts;
    if (!few && per < 16) per = 16;
    per = (per + 3) / 4 * 4;
    pp.heads_per = static_cast<int32_t>(per);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + per - 1) / per));
    if (grid.y > 65535) return SA_ERR_UNSUPPORTED;
    auto kern = layout == kInterleaved ? rotary_kernel<D, kInterleaved, PAGED>
                : layout == kHalves    ? rotary_kernel<D, kHalves, PAGED>
                                       : rotary_kernel<D, kShuffled, PAGED>;
    return launch_after(kern, grid, kRotThreads, 0, st, 1, spec, pp);
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
    if (int64_t(b->max_pages) * c->page_size > kMaxTokens) return SA_ERR_UNSUPPORTED;  // positions are 32 bits
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
    if (pos_offset > kMaxTokens) return SA_ERR_UNSUPPORTED;  // a token's position is 32 bits
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

constexpr int kDecodeCtas = 2;  // CTAs of decode_kernel on one SM

// Workspace: the parts of cut items, where each row's result lies, and, with a
// prefix, each pass's finished rows.
struct CachedLayout {
    size_t part_o, part_ml, info[2], tails[2], acc[2], acc_ml[2], total;
    int64_t rows_decode, rows_chunk;  // part rows of one pass by either kernel
    int64_t part_rows;                // of all passes
};

CachedLayout cached_layout(int32_t T, int32_t Hq, int32_t D, bool prefix)
{
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const int n_sm = device_sm_count() > 0 ? device_sm_count() : 148;
    CachedLayout w{};
    w.rows_decode = 2 * int64_t(kDecodeCtas) * n_sm * 32;
    w.rows_chunk = 2 * int64_t(n_sm) * 256;
    // the sequences' own pass may take both kernels, that over the prefix takes one; where decode_kernel's warps
    // each have a piece it runs alone, and their 2 x 4 x 2 n_sm x 16 rows lie in both kernels'
    w.part_rows = w.rows_decode + w.rows_chunk + (prefix ? w.rows_chunk : 0);
    const size_t th = size_t(T) * Hq;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t x = at;
        at += up(bytes);
        return x;
    };
    w.part_o = take(size_t(w.part_rows) * D * 4);
    w.part_ml = take(size_t(w.part_rows) * 8);
    for (int i = 0; i < (prefix ? 2 : 1); i++) w.info[i] = take(th * sizeof(RowInfo));
    w.tails[0] = take(size_t(w.rows_decode) / 2 * sizeof(TailRow));
    w.tails[1] = take(size_t(w.rows_chunk) / 2 * sizeof(TailRow));
    if (prefix)
        for (int i = 0; i < 2; i++) {
            w.acc[i] = take(th * D * 4);
            w.acc_ml[i] = take(th * 8);
        }
    w.total = at;
    return w;
}

int workspace_status(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (!bytes || T < 0 || Hq < 0 || Hkv < 0 || D <= 0) return SA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SA_ERR_UNSUPPORTED;
    if (Hq > 0 && (Hkv == 0 || Hq % Hkv)) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

// Map of a cache's K or V pages for boxes of box_rows places of one head and page:
// (64 columns, place, column panel, head, page), so that one box lands in shared
// memory as the panels of a 128-byte-swizzled tile.  Heads and places may come in
// any order in memory; pages past the end read as zeros.
bool make_map_pages(CUtensorMap* map, const void* base, const sa_kv_cache& c, uint32_t box_rows, uint32_t panels)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    // a stride along an extent of one is never used; give the map a valid one
    const uint64_t hs = c.Hkv > 1 ? c.head_stride : c.D, ps = c.n_pages > 1 ? c.page_stride : c.D;
    cuuint64_t dims[5] = {64, cuuint64_t(c.page_size), cuuint64_t(c.D / 64), cuuint64_t(c.Hkv), cuuint64_t(c.n_pages)};
    cuuint64_t strides[4] = {cuuint64_t(c.token_stride) * 2, 128, hs * 2, ps * 2};
    cuuint32_t box[5] = {64, box_rows, panels, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How decode_kernel runs a pass (see its modes; in kClusters nothing is left to join).
struct DecodePlan {
    int mt;       // rows of an item: 16 or 32
    DecodeMode mode;
    int cluster;  // CTAs of a cluster
    int64_t ctas;
};

// keys: most keys of an item, seqs: sequences, rows: most rows of one, as far as the host knows; held: CTAs
// that have room at once.
// Whole items by clusters where each CTA then has at most six units: the cut is even for any lengths, but
// its join costs a launch and some 3 us.  The line by warps (`by_warps`: it may be) where there is an item or
// more to every CTA and none has many keys: 256 sequences of up to 256 keys and 8 heads of 128, 40.8 us by CTAs
// and 28.3 by warps, 500 of up to 500, 91.8 and 71.9, 300 of up to 1000, 80.9 and 75.7, 256 of up to 2048, 110
// and 116; below one item to a CTA there is nothing in it.  Items of up to 128 keys are whole to a CTA each
// until there are two to every CTA (64 sequences of up to 60: 9.3 us, by warps 11.3; 80 of up to 100: 14.9, 13.1).
template <int D>
DecodePlan plan_decode(int64_t keys, int64_t seqs, int64_t rows, int32_t Hkv, int64_t held, bool by_warps)
{
    DecodePlan d;
    d.mt = rows <= 16 ? 1 : 2;
    const int64_t items = seqs * Hkv * ((rows + 16 * d.mt - 1) / (16 * d.mt));
    const int64_t units = keys / DecodeCfg<D, 1>::UK + 3;  // the sinks' and the band's first and last may be part full
    d.cluster = 1;
    if (by_warps && d.mt == 1 && items >= held && keys <= 1024 && (keys > 128 || items >= 2 * held)) {
        d.mode = kWarps;
        d.ctas = held;
        return d;
    }
    int64_t c = 1;
    while (c < 8 && items * c * 2 <= held && c < units) c *= 2;
    const bool whole = (units + c - 1) / c <= 6 && items * c <= 4 * held;
    d.mode = whole ? kClusters : kLine;
    if (whole) d.cluster = static_cast<int>(c);
    d.ctas = whole ? std::min(items, std::max<int64_t>(held / c, 1)) * c : kDecodeCtas * int64_t(device_sm_count());
    return d;
}

template <int D, int MT, DecodeMode MODE>
int launch_decode_as(const sa_kv_cache& cache, const PassParams& p, const DecodePlan& plan, cudaStream_t st)
{
    using C = DecodeCfg<D, MT>;
    auto kern = decode_kernel<D, MT, MODE>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
            return SA_ERR_CUDA;
        attr_set[dev] = true;
    }
    CUtensorMap mk, mv;
    const uint32_t rows = cache.page_size < C::TK ? cache.page_size : C::TK;
    if (!make_map_pages(&mk, cache.k, cache, rows, D / 64) || !make_map_pages(&mv, cache.v, cache, rows, D / 64))
        return SA_ERR_CUDA;
    return launch_after(kern, dim3(static_cast<unsigned>(plan.ctas)), C::kThreads, C::kSmemBytes, st,
                        plan.cluster, mk, mv, p);
}

template <int D>
int launch_decode(const sa_kv_cache& cache, const PassParams& p, const DecodePlan& plan, cudaStream_t st)
{
    if (plan.mt == 1)
        return plan.mode == kWarps      ? launch_decode_as<D, 1, kWarps>(cache, p, plan, st)
               : plan.mode == kBoth     ? launch_decode_as<D, 1, kBoth>(cache, p, plan, st)
               : plan.mode == kClusters ? launch_decode_as<D, 1, kClusters>(cache, p, plan, st)
                                        : launch_decode_as<D, 1, kLine>(cache, p, plan, st);
    return plan.mode == kBoth       ? launch_decode_as<D, 2, kBoth>(cache, p, plan, st)
           : plan.mode == kClusters ? launch_decode_as<D, 2, kClusters>(cache, p, plan, st)
                                    : launch_decode_as<D, 2, kLine>(cache, p, plan, st);
}

template <int D>
int launch_join(const JoinParams& j, bool prefix, cudaStream_t st)
{
    const int64_t rows = int64_t(j.T) * j.Hq, sms = device_sm_count();
    const bool few = rows <= 8 * sms;  // eight warps a row, else one
    const int64_t blocks = few ? rows : (rows + 7) / 8;
    const dim3 grid(static_cast<unsigned>(std::min(blocks, 8 * sms)));
    auto kern = few ? (prefix ? join_kernel<D, 8, true> : join_kernel<D, 8, false>)
                    : (prefix ? join_kernel<D, 1, true> : join_kernel<D, 1, false>);
    return launch_after(kern, grid, 256, 0, st, 1, j);
}

template <int D>
int launch_chunk(const sa_kv_cache& cache, const PassParams& p, cudaStream_t st)
{
    using C = ChunkCfg<D>;
    auto kern = chunk_kernel<D>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SA_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
            return SA_ERR_CUDA;
        // the warpgroups' register split must fit what the kernel is launched with
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SA_ERR_CUDA;
        if (fa.numRegs * C::kThreads < kRegSplitTotal) return SA_ERR_UNSUPPORTED;
        attr_set[dev] = true;
    }
    CUtensorMap mk, mv;
    const uint32_t rows = cache.page_size < C::UK ? cache.page_size : C::UK;
    if (!make_map_pages(&mk, cache.k, cache, rows, 1) || !make_map_pages(&mv, cache.v, cache, rows, 1))
        return SA_ERR_CUDA;
    return launch_after(kern, dim3(device_sm_count()), C::kThreads, C::kSmemBytes, st, 1, mk, mv, p);
}

// Part arrays and row entries of one pass, from part row `row0` on.
void use_parts(PassParams& p, const CachedLayout& w, uint8_t* ws, int which, int64_t row0, int D, bool prefix)
{
    p.part_row0 = static_cast<int32_t>(row0);
    p.part_o = reinterpret_cast<float*>(ws + w.part_o) + row0 * D;
    p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml) + row0;
    p.info = reinterpret_cast<RowInfo*>(ws + w.info[which]);
    p.acc = prefix ? reinterpret_cast<float*>(ws + w.acc[which]) : nullptr;
    p.acc_ml = prefix ? reinterpret_cast<float2*>(ws + w.acc_ml[which]) : nullptr;
}

// Most rows of an item of decode_kernel; a sequence with more goes to chunk_kernel,
// whose 128-row tiles it fills at least a quarter.
constexpr int kDecodeRows = 32;

// Most new tokens of a sequence, as far as the host knows.
int64_t most_new(const PassParams& p, int32_t max_q)
{
    return max_q > 0 ? max_q : (int64_t(p.T) + p.B - 1) / p.B;
}

// The kernels count a pass's units in 31 bits: items times the most units of one, for the kernels that
// run_paged takes.
bool units_fit(const PassParams& p, int64_t room, int64_t prefix_len, int32_t max_q)
{
    auto fit = [&](int64_t rows, int64_t seqs, int R, int64_t keys, int UK) {
        return rows / R + seqs <= INT_MAX / (keys / UK + 6) / p.Hkv;
    };
    const int64_t all = int64_t(p.T) * p.group;
    const bool decode = most_new(p, max_q) * p.group <= kDecodeRows;
    const bool own = decode ? fit(all, p.B, 16, room, 64) : fit(0, p.B, 16, room, 64) && fit(all, p.B, 256, room, 128);
    return own && (all <= kDecodeRows ? fit(all, 1, 16, prefix_len, 64) : fit(all, 1, 256, prefix_len, 128));
}

template <int D>
int run_paged(const sa_kv_cache& cache, PassParams p, const JoinParams& j, const CachedLayout& w, uint8_t* ws,
              const int32_t* prefix_table, int32_t max_q, cudaStream_t st)
{
    const bool prefix = p.prefix_len > 0;
    p.rows_above = 0;
    p.rows_upto = INT_MAX;
    // most keys of an item, out of `room`: what the window, the sinks and an item's tokens span
    auto most_keys = [&](int64_t room, int64_t tokens) {
        if (p.n_global > 0 || p.window < 0) return p.n_global > 0 ? room : std::min<int64_t>(room, p.cols);
        return std::min<int64_t>(room, int64_t(p.window) + tokens + p.cols);
    };
    const int64_t room = int64_t(p.max_pages) << p.page_shift;
    const int64_t most_q = most_new(p, max_q);
    const int64_t rows = most_q * p.group, all_rows = int64_t(p.T) * p.group;
    const int64_t held = kDecodeCtas * int64_t(device_sm_count());
    const DecodePlan over = plan_decode<D>(p.prefix_len, 1, all_rows, p.Hkv, held, false);
    const bool whole_over = prefix && all_rows <= kDecodeRows && over.mode == kClusters;
    // the warps' line has more and smaller units: it is counted in 31 bits too
    const bool by_warps = (all_rows / 16 + p.B) * p.Hkv <= INT_MAX / (room / DecodeCfg<D, 1>::TK + 8);
    const DecodePlan plan = plan_decode<D>(most_keys(room, most_q), p.B, rows, p.Hkv, held, by_warps);
    // Nothing is left for join_kernel where each item is finished by its CTAs; over a prefix the sequences'
    // pass then adds what the prefix's left: whole rows, or the parts of cut ones where these are few (122 rows a
    // head behind 151 tokens, 2 parts: 28.0 us on the device with join_kernel, 25.7 without; 12 sequences behind
    // 1223, 15 parts: 23.7 and 23.5; behind 12230, 20 parts: 33.4 and 35.0).
    auto parts_over = [&]() {
        const bool few = all_rows <= kDecodeRows;
        const int64_t R = few ? 16 * over.mt : ChunkCfg<D>::R, ctas = few ? over.ctas : device_sm_count();
        const int64_t UK = few ? DecodeCfg<D, 1>::UK : ChunkCfg<D>::UK;
        const int64_t units = most_keys(p.prefix_len, most_q) / UK + 3;
        return std::min(units, ctas / ((all_rows + R - 1) / R * p.Hkv) + 2);
    };
    const bool finished = rows <= kDecodeRows && plan.mode == kClusters &&
                          (!prefix || whole_over || parts_over() <= 16);
    // Both passes in one launch where each is whole items by clusters and the sequences' fit beside the prefix's:
    // in the prefix's clusters, or a CTA to each of few units.  On the device, one after another and like this (24
    // calls of 1 to 32 rows, none slower): 2 sequences behind 200 tokens, 1 head of 64, 11.1 and 7.5 us; 4 behind
    // 1000, 64/16 heads of 128, 15.9 and 12.0; 8 behind 2043, 16 heads of 128, 18.2 and 13.2.
    if (whole_over && rows <= kDecodeRows && over.ctas < held) {
        DecodePlan own = plan_decode<D>(most_keys(room, most_q), p.B, rows, p.Hkv, held - over.ctas, false);
        const int64_t items = int64_t(p.B) * p.Hkv, units = most_keys(room, most_q) / DecodeCfg<D, 1>::UK + 3;
        const int64_t c = own.cluster > 1 && items * over.cluster <= held - over.ctas ? over.cluster : 1;
        if (own.mode == kClusters && (units + c - 1) / c <= 6) {
            const int64_t ctas = std::min(items * c, held - over.ctas);
            own.mt = over.mt;  // of all rows: no less than the sequences' own
            own.mode = kBoth;
            own.cluster = over.cluster;
            own.ctas = over.ctas + (ctas + over.cluster - 1) / over.cluster * over.cluster;
            use_parts(p, w, ws, 1, w.rows_decode + w.rows_chunk, D, true);
            p.side_ctas = static_cast<int32_t>(over.ctas);
            p.cluster = static_cast<int32_t>(c);
            p.side_table = prefix_table;
            p.side_info = p.info;
            p.side_acc = p.acc;
            p.side_ml = p.acc_ml;
            use_parts(p, w, ws, 0, 0, D, true);
            if (int rc = launch_decode<D>(cache, p, own, st)) return rc;
            return launch_join<D>(j, true, st);
        }
    }
    if (prefix) {
        // the rows of all sequences against the prefix
        PassParams pp = p;
        pp.over_prefix = 1;
        pp.table = prefix_table;
        pp.table_stride = 0;
        use_parts(pp, w, ws, 1, w.rows_decode + w.rows_chunk, D, true);
        if (finished && whole_over) pp.info = nullptr;
        if (int rc = all_rows <= kDecodeRows ? launch_decode<D>(cache, pp, over, st) : launch_chunk<D>(cache, pp, st))
            return rc;
    }
    // each sequence against its own tokens: by decode_kernel alone where no sequence is known to have
    // more than its rows (it can take any), by chunk_kernel alone where there is one sequence of many rows,
    // else by both, each taking the sequences that suit it
    if (finished) {
        if (prefix) {
            p.pre_acc = reinterpret_cast<const float*>(ws + w.acc[1]);
            p.pre_ml = reinterpret_cast<const float2*>(ws + w.acc_ml[1]);
            if (!whole_over) {
                p.pre_info = j.info[1];
                p.pre_part_o = j.part_o;
                p.pre_part_ml = j.part_ml;
                p.part_rows = j.part_rows;
            }
        }
        return launch_decode<D>(cache, p, plan, st);
    }
    use_parts(p, w, ws, 0, 0, D, prefix);
    if (rows <= kDecodeRows) {
        if (int rc = launch_decode<D>(cache, p, plan, st)) return rc;
        return launch_join<D>(j, prefix, st);
    }
    // Rows may be many here, and few of them cut: then, without a prefix, the CTAs' tail slots are joined instead
    // of looking at every row (4.6 thousand tokens of 32 heads: 25 us for that).
    // Up to 16 thousand rows every row is looked at: the slots of all CTAs are 42 thousand entries whatever the batch
    // (517 tokens of 4 heads: 29 us by slots, 23 by rows; 2988 of 32 heads: 44 and 53).
    const bool by_tails = !prefix && int64_t(p.T) * p.Hq > 16384;
    TailJoinParams tj{};
    if (by_tails) {
        tj.part_o = j.part_o;
        tj.part_ml = j.part_ml;
        tj.o = j.o;
        tj.o_token = j.o_token;
        tj.o_head = j.o_head;
        tj.lse = j.lse;
        tj.Hq = j.Hq;
        tj.rows = j.T * j.Hq;
        tj.part_rows = j.part_rows;
    }
    auto use_tails = [&](PassParams& pp, int which, int64_t ctas, int R) {
        if (!by_tails) return;
        pp.info = nullptr;
        pp.tails = reinterpret_cast<TailRow*>(ws + w.tails[which]);
        tj.tails[which] = pp.tails;
        tj.entries[which] = static_cast<int32_t>(ctas * R);
        tj.part_row0[which] = pp.part_row0;
        while ((1 << tj.shift[which]) < R) tj.shift[which]++;
    };
    if (p.B > 1) {
        PassParams pp = p;
        pp.rows_upto = p.group <= 16 ? 16 : kDecodeRows;
        const DecodePlan line{pp.rows_upto <= 16 ? 1 : 2, kLine, 1, kDecodeCtas * int64_t(device_sm_count())};
        use_tails(pp, 0, line.ctas, 16 * line.mt);
        if (int rc = launch_decode<D>(cache, pp, line, st)) return rc;
        p.rows_above = pp.rows_upto;
    }
    use_parts(p, w, ws, 0, w.rows_decode, D, prefix);
    use_tails(p, 1, device_sm_count(), ChunkCfg<D>::R);
    if (int rc = launch_chunk<D>(cache, p, st)) return rc;
    if (!by_tails) return launch_join<D>(j, prefix, st);
    const int64_t blocks = (int64_t(tj.entries[0]) + tj.entries[1] + 31) / 32;  // eight threads an entry
    return launch_after(join_tails_kernel<D>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, 1, tj);
}

int32_t clip_to(int32_t v, int64_t n) { return v > n ? static_cast<int32_t>(n) : v; }

int fwd_paged(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch, const int32_t* prefix_table,
              int32_t prefix_len, bool shared, const sa_pattern* pattern, int32_t Hq, float scale, const sa_view* o,
              float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!pattern || Hq < 0 || prefix_len < 0) return SA_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch, cache)) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return SA_ERR_INVALID_ARG;
    if (int rc = check_pattern(*pattern)) return rc;
    if (pattern->causal != 1 || pattern->stride > 0 || pattern->area > 0) return SA_ERR_UNSUPPORTED;
    if (prefix_len > kMaxTokens) return SA_ERR_UNSUPPORTED;
    const int32_t T = batch->T;
    if (batch->B == 0 || T == 0 || Hq == 0) return SA_OK;
    if (cache->Hkv == 0 || cache->n_pages == 0 || Hq % cache->Hkv) return SA_ERR_UNSUPPORTED;
    if (int64_t(T) * Hq > INT_MAX / 2) return SA_ERR_UNSUPPORTED;  // rows are counted in 32 bits
    if (prefix_len > 0 && !prefix_table) return SA_ERR_INVALID_ARG;
    PassParams p{};
    p.B = batch->B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = cache->Hkv;
    p.group = Hq / cache->Hkv;
    if (!units_fit(p, int64_t(batch->max_pages) * cache->page_size, prefix_len, batch->max_q)) return SA_ERR_UNSUPPORTED;
    if (int rc = view_status(q, 1, Hq, T, false)) return rc;
    if (int rc = view_status(o, 1, Hq, T, true)) return rc;
    if (!lse || !workspace) return SA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return SA_ERR_MISALIGNED;
    // fwd_shared asks for its own size for every prefix_len, 0 too
    const CachedLayout w = cached_layout(T, Hq, cache->D, shared);
    if (workspace_bytes < w.total) return SA_ERR_BUFFER_TOO_SMALL;
    if (int rc = device_arrays({batch->q_start, batch->kv_len, batch->table, prefix_len > 0 ? prefix_table : nullptr}))
        return rc;
    int32_t* status = nullptr;
    if (int rc = device_status_word(&status)) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.q = static_cast<const __nv_bfloat16*>(q->data);
    p.q_token = T > 1 ? q->token_stride : 0;
    p.q_head = Hq > 1 ? q->head_stride : 0;
    p.o = static_cast<__nv_bfloat16*>(o->data);
    p.o_token = T > 1 ? o->token_stride : 0;
    p.o_head = Hq > 1 ? o->head_stride : 0;
    p.lse = lse;
    p.q_start = batch->q_start;
    p.kv_len = batch->kv_len;
    p.table = batch->table;
    p.table_stride = batch->B > 1 ? batch->table_stride : 0;
    while ((int64_t(1) << p.group_shift) < p.group) p.group_shift++;
    p.group_shift += 31;
    p.group_mul = static_cast<uint32_t>((uint64_t(1) << p.group_shift) / p.group + 1);
    p.n_pages = cache->n_pages;
    p.page_shift = page_shift_of(cache->page_size);
    p.max_pages = batch->max_pages;
    p.prefix_len = prefix_len;
    // window and global rows clipped to the farthest position, columns to the last key: the same keys, no overflow
    const int64_t farthest = 2 * int64_t(kMaxTokens);
    p.window = clip_to(pattern->window, farthest);
    p.n_global = clip_to(pattern->n_global, farthest);
    p.cols = clip_to(pattern->sinks > pattern->n_global ? pattern->sinks : pattern->n_global,
                     prefix_len + int64_t(batch->max_pages) * cache->page_size);
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.status = status;
    p.timeout = wait_limit_cycles();
    p.debug_flags = debug_flags();
    JoinParams j{};
    j.part_o = reinterpret_cast<const float*>(ws + w.part_o);
    j.part_ml = reinterpret_cast<const float2*>(ws + w.part_ml);
    j.info[0] = reinterpret_cast<const RowInfo*>(ws + w.info[0]);
    j.o = p.o;
    j.o_token = p.o_token;
    j.o_head = p.o_head;
    j.lse = lse;
    j.q_start = batch->q_start;
    j.B = batch->B;
    j.T = T;
    j.Hq = Hq;
    j.part_rows = static_cast<int32_t>(w.part_rows);
    if (prefix_len > 0) {
        j.info[1] = reinterpret_cast<const RowInfo*>(ws + w.info[1]);
        for (int i = 0; i < 2; i++) {
            j.acc[i] = reinterpret_cast<const float*>(ws + w.acc[i]);
            j.acc_ml[i] = reinterpret_cast<const float2*>(ws + w.acc_ml[i]);
        }
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cache->D == 128 ? run_paged<128>(*cache, p, j, w, ws, prefix_table, batch->max_q, st)
                           : run_paged<64>(*cache, p, j, w, ws, prefix_table, batch->max_q, st);
}

}  // namespace
}  // namespace sa

extern "C" int sparse_attn_fwd_cached_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (int rc = sa::workspace_status(T, Hq, Hkv, D, bytes)) return rc;
    *bytes = sa::cached_layout(T, Hq, D, false).total;
    return SA_OK;
}

extern "C" int sparse_attn_fwd_shared_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t* bytes)
{
    if (int rc = sa::workspace_status(T, Hq, Hkv, D, bytes)) return rc;
    *bytes = sa::cached_layout(T, Hq, D, true).total;
    return SA_OK;
}

extern "C" int sparse_attn_fwd_cached(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch,
                                      const sa_pattern* pattern, int32_t Hq, float scale, const sa_view* o, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (!batch || !cache) return SA_ERR_INVALID_ARG;
    return sa::fwd_paged(q, cache, batch, nullptr, 0, false, pattern, Hq, scale, o, lse, workspace, workspace_bytes,
                         stream);
}

extern "C" int sparse_attn_fwd_shared(const sa_view* q, const sa_kv_cache* cache, const sa_cache_batch* batch,
                                      const int32_t* prefix_table, int32_t prefix_len, const sa_pattern* pattern,
                                      int32_t Hq, float scale, const sa_view* o, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream)
{
    if (!batch || !cache) return SA_ERR_INVALID_ARG;
    return sa::fwd_paged(q, cache, batch, prefix_table, prefix_len, true, pattern, Hq, scale, o, lse, workspace,
                         workspace_bytes, stream);
}
