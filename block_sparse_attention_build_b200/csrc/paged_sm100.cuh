// What the kernels of attention over a paged cache share: the description of a
// pass, how its work is cut into items and units and spread over the CTAs, and
// the kernel that joins the parts of an item that several CTAs computed.
//
// A pass computes, for the new tokens of every sequence of a batch (or, over a
// shared prefix, for all of them as one), O = softmax(scale Q K^T) V over the
// keys a row sees.  The query heads of one key/value head and the new tokens of
// a sequence form one column of rows (row = token * group + head of the group):
// they read the same keys, so each key and value is loaded once for all of them.
//
//   item  R consecutive rows of one sequence and key/value head
//   unit  UK consecutive keys of an item; only units that hold a key some row of
//         the item sees exist: those of the sinks [0, cols) and those of the band
//         [first row's position - window, last row's position]
//
// All units of a pass, item after item, form one line of U units that the G CTAs
// cut into G pieces of equal length.  So the work is even for any lengths, few
// rows over a long cache use all SMs, and nothing about it is decided on the
// host: lengths are read when the kernel runs and a captured graph follows them.
// An item's start and end take time too (its queries, joining its warps, writing
// its rows): on the line each item is preceded by `w` places that hold no unit
// (64 sequences of 34 to 1024 tokens, 8 heads: 1 us a unit, 1.9 us an item; without
// the places the CTAs' times went from 21 to 39 us).
// An item that lies inside one piece is finished there.  One that is cut leaves
// its parts, unnormalised in 32 bits with the rows' running maximum and sum: the
// CTA in which the item begins writes its part to its "tail" slot, every later one
// to its "head" slot (a CTA has at most one of each), and join_kernel adds them in
// the order of the CTAs, so results do not depend on which finished first.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sm100.cuh"

namespace sa {

// Where a row's result lies (one per row and query head): in n > 0 parts at rows
// `first`, `second`, `second` + stride, ... of the part arrays, or, n = 0,
// finished by its CTA.
struct alignas(16) RowInfo {
    int32_t first, second, n, stride;
};

// A row that no sequence covers (q_start not ascending from 0) has no entry: nothing of one that is out of range
// is followed.
__device__ __forceinline__ bool in_range(const RowInfo& r, int part_rows)
{
    return r.n >= 0 && r.n <= part_rows && r.stride >= 0 && r.stride <= part_rows && r.first >= 0 && r.second >= 0 &&
           (r.n == 0 || (r.first < part_rows && r.second + static_cast<int64_t>(r.n - 2) * r.stride < part_rows));
}

// The same from the other side, where rows are many and few of them are cut: the
// rows of each CTA's tail slot (n = 0: none), R entries a CTA.
struct alignas(8) TailRow {
    int32_t row, n;  // token * Hq + head; parts
};

// Every kernel is launched while the one before it on the stream may still run, and reads or writes memory only
// behind griddepcontrol.wait: nothing else promises it the writes of the kernels before, not even of those that the
// previous one has waited for.  All of what it reads may have been written after its launch, so its loads are plain
// ones: the non-coherent path is for data that does not change while a kernel lives.
struct PassParams {
    const __nv_bfloat16* q;
    int64_t q_token, q_head;
    __nv_bfloat16* o;
    int64_t o_token, o_head;
    float* lse;                // [T, Hq]
    const int32_t* q_start;    // [B + 1]
    const int32_t* kv_len;     // [B]
    const int32_t* table;      // [B, max_pages]; over the prefix: its pages
    int64_t table_stride;
    int32_t B, T, Hq, Hkv, group;
    uint32_t group_mul, group_shift;  // x / group = x * group_mul >> group_shift for 0 <= x < 2^31
    int32_t n_pages, page_shift, max_pages;
    int32_t prefix_len;        // tokens before a sequence's own
    int32_t over_prefix;       // 1: all rows against the prefix; 0: each sequence against its own tokens
    int32_t rows_above;        // the pass takes sequences with more rows than this (a sequence's rows are its
    int32_t rows_upto;         // new tokens * group) and no more than this
    int32_t window, cols, n_global;  // cols = max(sinks, n_global)
    float scale_log2;
    float* part_o;             // [2 * CTAs * R, D] parts of cut items (this pass's)
    float2* part_ml;           // [2 * CTAs * R] running maximum (log2 units), sum
    int32_t part_row0;         // index of the first of them in the arrays that join_kernel reads
    RowInfo* info;             // [T, Hq]; null where no row is read from parts or where there are
    TailRow* tails;            // [CTAs * R]
    float* acc;                // null: finished rows go to o and lse; else [T, Hq, D] unnormalised,
    float2* acc_ml;            // [T, Hq]
    int32_t side_ctas;         // kBoth: the launch's first CTAs, which run the pass over the prefix, with these
    int32_t cluster;           // in place of over_prefix, table, info, acc; CTAs that share an item of the others
    const int32_t* side_table;
    RowInfo* side_info;
    float* side_acc;
    float2* side_ml;
    const float* pre_acc;      // not null: what the pass over the prefix left, added to every row
    const float2* pre_ml;
    const RowInfo* pre_info;   // not null: rows of that pass may lie in parts instead, of the arrays
    const float* pre_part_o;   // that join_kernel reads
    const float2* pre_part_ml;
    int32_t part_rows;
    int32_t* status;
    long long timeout;
    int32_t debug_flags;
};

enum : int32_t { ST_PAGED_WAIT = 64 };

// LSE of a row with maximum m (log2 units) and sum l: -inf where the row sees nothing (a sum of exactly 0), NaN
// where a score is NaN or +inf (the sum is NaN then).
__device__ __forceinline__ float lse_of(float m, float log2_l, float l)
{
    return l == 0.f ? -INFINITY : (m + log2_l) * 0.69314718055994530942f;
}

// One sequence as a pass sees it.
struct SeqView {
    int32_t first;  // its first row in the token tensors
    int32_t m;      // new tokens
    int32_t len;    // keys
    int32_t p0;     // position of its first new token, relative to its first key
};

// Tokens of a sequence as its kv_len gives them: where its new tokens stand.  The limit keeps a position behind a
// prefix within 31 bits.
constexpr int kMaxTokens = INT32_MAX / 4;
__device__ __forceinline__ int tokens_of(int kv_len) { return min(max(kv_len, 0), kMaxTokens); }

// Those of them that are in the cache: no more than the table has room for.
__device__ __forceinline__ int cached_len(const PassParams& p, int tokens)
{
    return min(tokens, p.max_pages << p.page_shift);
}

__device__ __forceinline__ SeqView load_seq(const PassParams& p, int b)
{
    SeqView s;
    if (p.over_prefix) {
        s.first = 0;
        s.m = min(max(p.q_start[p.B], 0), p.T);
        s.len = p.prefix_len;
        s.p0 = 0;  // differs from row to row: see PassBounds
    } else {
        const int a = min(max(p.q_start[b], 0), p.T);
        s.first = a;
        s.m = max(min(p.q_start[b + 1], p.T) - a, 0);
        const int tokens = tokens_of(p.kv_len[b]);
        s.len = cached_len(p, tokens);
        s.p0 = tokens - s.m;
    }
    return s;
}

__device__ __forceinline__ int div_group(const PassParams& p, int x)
{
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(x)) * p.group_mul >> p.group_shift);
}

// Does the pass take a sequence of this many rows?
__device__ __forceinline__ bool takes(const PassParams& p, int rows)
{
    return rows > p.rows_above && rows <= p.rows_upto;
}

// Units of the items whose rows stand at positions pa .. pb (counted like the keys
// they are compared with): `ns` units of sinks from 0 on, then those from `bs` on;
// nt in all (one, empty, where a row sees nothing: it still has to be written).
struct Units {
    int32_t ns, bs, nt, hi;  // keys end before hi
    __device__ __forceinline__ int key(int i, int UK) const { return (i < ns ? i : bs + (i - ns)) * UK; }
};

__device__ __forceinline__ Units units_of(const PassParams& p, int pa, int pb, int len, int UK)
{
    // positions count the prefix; a sequence's own keys begin behind it
    const int off = p.over_prefix ? 0 : p.prefix_len;
    Units u;
    u.hi = min(max(pb - off + 1, 0), len);
    const int c = min(max(p.cols - off, 0), u.hi);
    int lo = u.hi;
    if (pa < p.n_global)
        lo = 0;
    else if (p.window >= 0)  // 64 bits: a row before its sequence's first key stands at a negative position
        lo = static_cast<int>(min(max(static_cast<int64_t>(pa) - p.window - off, int64_t(0)),
                                  static_cast<int64_t>(u.hi)));
    u.ns = (c + UK - 1) / UK;
    u.bs = max(lo / UK, u.ns);
    const int be = lo < u.hi ? (u.hi + UK - 1) / UK : u.bs;
    u.nt = max(u.ns + max(be - u.bs, 0), 1);
    return u;
}

// Positions of the first and last row of an item; over the prefix the rows come
// from many sequences and the bounds hold for all rows of the pass.
struct PassBounds {
    int lo, hi;
};

template <int R, int UK>
__device__ __forceinline__ Units item_units(const PassParams& p, const PassBounds& pb, const SeqView& s, int rb)
{
    if (p.over_prefix) return units_of(p, pb.lo, pb.hi, s.len, UK);
    const int r0 = rb * R;
    const int r1 = min(r0 + R, s.m * p.group) - 1;
    const int base = p.prefix_len + s.p0;
    return units_of(p, base + div_group(p, r0), base + div_group(p, r1), s.len, UK);
}

// Position of a token (prefix included), for a pass over the prefix: the sequence
// is the last one that starts at or before it.
__device__ __forceinline__ int token_position(const PassParams& p, int t)
{
    int lo = 0, hi = p.B;  // q_start[lo] <= t < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.q_start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int first = p.q_start[lo], next = p.q_start[lo + 1];
    return p.prefix_len + tokens_of(p.kv_len[lo]) - (next - first) + (t - first);
}

// Where a CTA is on the line of units.
struct Cursor {
    int b, rb, h;  // item
    int i;         // unit of the item
    SeqView s;
    Units u;
};

// Move to the first unit of the next item; at the end of the line b reaches n_seq.
template <int R, int UK>
__device__ __forceinline__ void next_item(const PassParams& p, const PassBounds& pb, Cursor& c, int n_seq)
{
    c.i = 0;
    if (++c.h < p.Hkv) return;
    c.h = 0;
    if (++c.rb * R >= c.s.m * p.group) {
        c.rb = 0;
        do {
            if (++c.b >= n_seq) return;
            c.s = load_seq(p, c.b);
        } while (c.s.m == 0 || !takes(p, c.s.m * p.group));
    }
    c.u = item_units<R, UK>(p, pb, c.s, c.rb);
}

// The piece of the line that this CTA takes: [u0, u1) of U units (or items: ITEMS),
// cut into G equal pieces.  The host has checked that U stays below 2^31.
struct Piece {
    int U, u0, u1;
    int each, more;  // units of a piece; the first `more` pieces (of an item's) have one more
    int G;
    int of_item;     // > 0: that many whole pieces make an item, of item_nt units
    int item_nt;
    int w;           // places before an item's units
    int avail;       // units of the item at u0 that lie before u1 (more than it has: the piece goes on)
    PassBounds pb;
    Cursor c;        // at u0 (valid when u0 < u1)
};

template <int R, int UK, bool ITEMS>
__device__ __forceinline__ int seq_units(const PassParams& p, const PassBounds& pb, const SeqView& s, int w)
{
    const int rows = s.m * p.group;
    if (rows == 0 || !takes(p, rows)) return 0;
    const int nrb = (rows + R - 1) / R;
    int n = nrb;
    if (!ITEMS && p.over_prefix) n = nrb * (item_units<R, UK>(p, pb, s, 0).nt + w);
    if (!ITEMS && !p.over_prefix) {
        n = 0;
#pragma unroll 1
        for (int rb = 0; rb < nrb; rb++) n += item_units<R, UK>(p, pb, s, rb).nt + w;
    }
    return n * p.Hkv;
}

// Over the prefix: the lowest and the highest position of all sequences' rows (whole warp).
__device__ __forceinline__ PassBounds pass_bounds(const PassParams& p)
{
    int lo = INT32_MAX, hi = INT32_MIN;
#pragma unroll 1
    for (int b = threadIdx.x % 32; b < p.B; b += 32) {
        const int m = p.q_start[b + 1] - p.q_start[b];
        const int last = p.prefix_len + tokens_of(p.kv_len[b]) - 1;
        if (m <= 0) continue;
        lo = min(lo, last - m + 1);
        hi = max(hi, last);
    }
    return PassBounds{__reduce_min_sync(0xffffffffu, lo), __reduce_max_sync(0xffffffffu, hi)};
}

// The sequence that find_piece looks at first in this lane.
__device__ __forceinline__ SeqView peek_seq(const PassParams& p)
{
    const int n_seq = p.over_prefix ? 1 : p.B;
    return load_seq(p, min(static_cast<int>(threadIdx.x % 32) * ((n_seq + 31) / 32), n_seq - 1));
}

// Find the piece that `cta` of n_cta takes (`ahead`: from peek_seq).  By a whole warp, on its own (no barrier: each
// warp of a CTA finds the same).  It is the first thing every CTA does, and its code runs
// once: it is kept short, since instructions come from L2 the first time.
template <int R, int UK, bool ITEMS>
__device__ __forceinline__ Piece find_piece(const PassParams& p, const SeqView& ahead, int cta, int n_cta, int w)
{
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x % 32;
    Piece r;
    r.pb = PassBounds{0, 0};
    const int n_seq = p.over_prefix ? 1 : p.B;
    if (p.over_prefix) r.pb = pass_bounds(p);
    // Over the prefix all items have the same units: where they are few, each is cut into as many pieces of
    // its own as there are CTAs for, so that no CTA pays for the end of one item and the start of another
    // (8 items of 256 units: two segments took a CTA 48 us, one 40).
    r.of_item = 0;
    r.w = w;
    int items = 0;
    if (!ITEMS && p.over_prefix) {
        items = (ahead.m * p.group + R - 1) / R * p.Hkv;
        if (2 * items <= n_cta && items > 0) r.w = 0;
    }
    // units of this lane's sequences, and of those before them
    const int per = (n_seq + 31) / 32;
    const int b0 = lane * per, b1 = min(b0 + per, n_seq);
    int own = 0, own_items = 0;
    SeqView s = ahead;
#pragma unroll 1
    for (int b = b0; b < b1;) {
        own += seq_units<R, UK, ITEMS>(p, r.pb, s, 0);
        if (!ITEMS) own_items += seq_units<R, UK, true>(p, r.pb, s, 0);
        if (++b < b1) s = load_seq(p, b);
    }
    if (!ITEMS) {
        // places before the items only where the pieces are a few units long: below that a CTA would get a
        // piece without any
        if (__reduce_add_sync(kAll, own) < 4 * n_cta) r.w = 0;
        own += r.w * own_items;
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
    }
    r.U = __shfl_sync(kAll, incl, 31);
    r.G = min(r.U, n_cta);
    r.u0 = r.u1 = r.avail = r.c.i = 0;
    if (cta >= r.G) return r;
    int line = r.U, pieces = r.G, piece = cta, base = 0;
    if (items > 0 && 2 * items <= n_cta) {
        r.item_nt = item_units<R, UK>(p, r.pb, ahead, 0).nt;
        r.of_item = min(static_cast<uint32_t>(n_cta) / static_cast<uint32_t>(items), static_cast<uint32_t>(r.item_nt));
        r.G = items * r.of_item;
        if (cta >= r.G) {
            r.avail = 0;
            return r;
        }
        const int item = static_cast<uint32_t>(cta) / static_cast<uint32_t>(r.of_item);
        line = r.item_nt;
        pieces = r.of_item;
        piece = cta - item * r.of_item;
        base = item * r.item_nt;
    }
    r.each = static_cast<uint32_t>(line) / static_cast<uint32_t>(pieces);
    r.more = line - r.each * pieces;
    r.u0 = base + piece * r.each + min(piece, r.more);
    r.u1 = r.u0 + r.each + (piece < r.more ? 1 : 0);
    int at = incl - own;
    const bool here = at <= r.u0 && r.u0 < incl;
    const int who = __ffs(__ballot_sync(kAll, here)) - 1;
    int b = b0;
    if (per > 1 && here) {
#pragma unroll 1
        for (;; b++) {
            const int n = seq_units<R, UK, ITEMS>(p, r.pb, load_seq(p, b), r.w);
            if (r.u0 < at + n) break;
            at += n;
        }
    }
    r.c.b = __shfl_sync(kAll, b, who);
    at = __shfl_sync(kAll, at, who);
    r.c.s = load_seq(p, r.c.b);
    r.c.rb = 0;
#pragma unroll 1
    for (;; r.c.rb++) {
        r.c.u = item_units<R, UK>(p, r.pb, r.c.s, r.c.rb);
        const int n = (ITEMS ? 1 : r.c.u.nt + r.w) * p.Hkv;
        if (r.u0 < at + n) break;
        at += n;
    }
    const uint32_t rest = r.u0 - at;
    const int place = ITEMS ? 0 : rest % static_cast<uint32_t>(r.c.u.nt + r.w);
    r.c.h = ITEMS ? rest : rest / static_cast<uint32_t>(r.c.u.nt + r.w);
    r.c.i = ITEMS ? 0 : max(place - r.w, 0);
    r.avail = r.u1 - r.u0 + place - r.w;
    return r;
}

// CTA whose piece holds unit u.
__device__ __forceinline__ int cta_of(const Piece& r, int u)
{
    int first = 0;
    if (r.of_item > 0) {
        const int item = static_cast<uint32_t>(u) / static_cast<uint32_t>(r.item_nt);
        first = item * r.of_item;
        u -= item * r.item_nt;
    }
    const int longer = r.more * (r.each + 1);
    return first + (u < longer ? static_cast<uint32_t>(u) / static_cast<uint32_t>(r.each + 1)
                               : r.more + static_cast<uint32_t>(u - longer) / static_cast<uint32_t>(r.each));
}

// The table's entry for key k (k below the sequence's length), and the page that it
// stands for: one past the cache's end (which the tensor map fills with zeros) where
// the table names none of its pages.  Apart, so that an entry can be asked for well
// before it is looked at.
__device__ __forceinline__ int page_entry(const PassParams& p, int b, int k)
{
    return p.table[static_cast<int64_t>(b) * p.table_stride + (k >> p.page_shift)];
}
__device__ __forceinline__ int page_of(const PassParams& p, int entry)
{
    return entry >= 0 && entry < p.n_pages ? entry : p.n_pages;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2, int c3,
                                            int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// ---------------------------------------------------------------------------
// Joining
// ---------------------------------------------------------------------------

struct JoinParams {
    const float* part_o;
    const float2* part_ml;
    const RowInfo* info[2];   // the passes' (the second null without a prefix)
    const float* acc[2];
    const float2* acc_ml[2];
    __nv_bfloat16* o;
    int64_t o_token, o_head;
    float* lse;
    const int32_t* q_start;
    int32_t B, T, Hq;
    int32_t part_rows;        // rows of the part arrays
};

// Up to two kernels' tail rows: entry e of a kernel is row e mod R of CTA e / R.
struct TailJoinParams {
    const float* part_o;
    const float2* part_ml;
    const TailRow* tails[2];
    int32_t entries[2], shift[2];  // entries (0: none), log2 R
    int32_t part_row0[2];
    __nv_bfloat16* o;
    int64_t o_token, o_head;
    float* lse;
    int32_t Hq, rows;              // T * Hq
    int32_t part_rows;
};

// A part in which a row sees nothing.  A part whose scores are all NaN keeps its maximum of -inf too (the maximum
// drops them), but its sum is NaN: it is added, and the row is NaN whichever part it comes from.
__device__ __forceinline__ bool no_part(float2 ml) { return ml.x == -INFINITY && ml.y == 0.f; }

// A row's parts added up by one warp, E elements a lane: O = sum of O_k 2^(m_k - M)
// over L = sum of l_k 2^(m_k - M), M the largest m_k, in the order they come.
template <int D>
struct RowSum {
    static constexpr int E = D / 32;
    float acc[E];
    float M, L;
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = 0.f;
        M = -INFINITY;
        L = 0.f;
    }
    __device__ __forceinline__ void add(const float (&v)[E], float2 ml)
    {
        if (no_part(ml)) return;
        const float mn = fmaxf(M, ml.x);
        const float a = ex2_approx(M - mn), b = ex2_approx(ml.x - mn);
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = acc[e] * a + v[e] * b;
        L = L * a + ml.y * b;
        M = mn;
    }
    // parts first, second, second + stride, ...: every `step`-th from k0 on, eight in flight
    __device__ __forceinline__ void add_parts(const float* part_o, const float2* part_ml, const RowInfo& ri, int k0,
                                              int step, int lane)
    {
        constexpr int K = 8;
        for (int k1 = k0; k1 < ri.n; k1 += K * step) {
            float v[K][E];
            float2 ml[K];
#pragma unroll
            for (int j = 0; j < K; j++) {
                const int k = k1 + j * step;
                ml[j] = make_float2(-INFINITY, 0.f);
                if (k >= ri.n) continue;
                const int64_t at = k == 0 ? ri.first : ri.second + static_cast<int64_t>(k - 1) * ri.stride;
                ml[j] = part_ml[at];
#pragma unroll
                for (int e = 0; e < E; e++) v[j][e] = part_o[at * D + lane * E + e];
            }
#pragma unroll
            for (int j = 0; j < K; j++) add(v[j], ml[j]);
        }
    }
    template <class P>
    __device__ __forceinline__ void write(const P& p, uint32_t row, int lane) const
    {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const uint32_t t = row / static_cast<uint32_t>(p.Hq), h = row - t * p.Hq;
        __nv_bfloat16* dst = p.o + t * p.o_token + h * p.o_head + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        if (lane == 0) p.lse[row] = lse_of(M, log2f(L), L);
    }
};


// Rows whose result lies in parts (and, with a prefix, all rows).  WPR warps share
// a row (each takes every WPR-th part, then they are added in the order of the
// warps): one where rows are many, eight where a few rows have up to a part per CTA,
// whose loads are then in flight together.
template <int D, int WPR, bool PREFIX>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p)
{
    constexpr int kRows = 8 / WPR;
    constexpr int E = D / 32;  // elements of a lane
    wait_previous_kernel();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = warp % WPR;
    __shared__ float sh_o[8][D];
    __shared__ float sh_m[8], sh_l[8];
    const int64_t total = static_cast<int64_t>(min(max(p.q_start[p.B], 0), p.T)) * p.Hq;
    // every warp of a block makes the same number of rounds
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < total;
         row0 += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t row = row0 + warp / WPR;
        bool write = PREFIX && row < total;
        RowSum<D> sum;
        sum.clear();
        if (row < total) {
#pragma unroll
            for (int s = 0; s < (PREFIX ? 2 : 1); s++) {
                const RowInfo ri = p.info[s][row];
                if (!in_range(ri, p.part_rows)) continue;
                if (ri.n == 0) {
                    if (PREFIX && sub == 0) {
                        float v[E];
#pragma unroll
                        for (int e = 0; e < E; e++) v[e] = p.acc[s][row * D + lane * E + e];
                        sum.add(v, p.acc_ml[s][row]);
                    }
                    continue;
                }
                write = true;
                sum.add_parts(p.part_o, p.part_ml, ri, sub, WPR, lane);
            }
        }
        if constexpr (WPR > 1) {
#pragma unroll
            for (int e = 0; e < E; e++) sh_o[warp][lane * E + e] = sum.acc[e];
            if (lane == 0) {
                sh_m[warp] = sum.M;
                sh_l[warp] = sum.L;
            }
            __syncthreads();
            if (sub == 0) {
                for (int w = 1; w < WPR; w++) {
                    float v[E];
#pragma unroll
                    for (int e = 0; e < E; e++) v[e] = sh_o[warp + w][lane * E + e];
                    sum.add(v, make_float2(sh_m[warp + w], sh_l[warp + w]));
                }
            }
            __syncthreads();
        }
        if (write && sub == 0) sum.write(p, static_cast<uint32_t>(row), lane);
    }
}

// The rows of the CTAs' tail slots, eight lanes each: most have two parts, so what
// counts is how many rows' loads a warp has in flight.
template <int D>
__global__ void __launch_bounds__(256) join_tails_kernel(const TailJoinParams p)
{
    constexpr int E = D / 8, V = E / 4;  // elements and 16-byte loads of a lane (those of a load lie side by side)
    wait_previous_kernel();
    const int l = threadIdx.x % 8;
    int e = (blockIdx.x * 256 + threadIdx.x) / 8;
    const int k = e >= p.entries[0];
    if (k) e -= p.entries[0];
    if (e >= p.entries[k]) return;
    const TailRow t = p.tails[k][e];
    const int R = 1 << p.shift[k];
    const int64_t first = p.part_row0[k] + (2 * (e >> p.shift[k]) + 1) * R + (e & (R - 1));
    // part i at rows first, first + R, first + 3 R, ...
    if (t.n <= 0 || t.row < 0 || t.row >= p.rows || first + (2 * static_cast<int64_t>(t.n) - 3) * R >= p.part_rows) return;
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; i++) acc[i] = 0.f;
    float M = -INFINITY, L = 0.f;
    for (int i0 = 0; i0 < t.n; i0 += 2) {
        float4 v[2][V];
        float2 ml[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int i = i0 + j;
            ml[j] = make_float2(-INFINITY, 0.f);
            if (i >= t.n) continue;
            const int64_t at = i == 0 ? first : first + (2 * i - 1) * R;
            ml[j] = p.part_ml[at];
#pragma unroll
            for (int x = 0; x < V; x++) v[j][x] = *reinterpret_cast<const float4*>(p.part_o + at * D + (x * 8 + l) * 4);
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            if (no_part(ml[j])) continue;
            const float mn = fmaxf(M, ml[j].x);
            const float a = ex2_approx(M - mn), b = ex2_approx(ml[j].x - mn);
#pragma unroll
            for (int x = 0; x < V; x++) {
                acc[4 * x] = acc[4 * x] * a + v[j][x].x * b;
                acc[4 * x + 1] = acc[4 * x + 1] * a + v[j][x].y * b;
                acc[4 * x + 2] = acc[4 * x + 2] * a + v[j][x].z * b;
                acc[4 * x + 3] = acc[4 * x + 3] * a + v[j][x].w * b;
            }
            L = L * a + ml[j].y * b;
            M = mn;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const uint32_t tok = static_cast<uint32_t>(t.row) / static_cast<uint32_t>(p.Hq), h = t.row - tok * p.Hq;
    __nv_bfloat16* dst = p.o + tok * p.o_token + h * p.o_head + l * 4;
#pragma unroll
    for (int x = 0; x < V; x++)
        *reinterpret_cast<uint2*>(dst + x * 32) = make_uint2(pack_bf16x2(acc[4 * x] * inv, acc[4 * x + 1] * inv),
                                                             pack_bf16x2(acc[4 * x + 2] * inv, acc[4 * x + 3] * inv));
    if (l == 0) p.lse[t.row] = lse_of(M, log2f(L), L);
}

}  // namespace sa
