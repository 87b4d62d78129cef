// Attention of few rows (single tokens, a handful of tokens, small groups of
// heads) over a paged cache.
//
// Each key and value is read once for at most 32 rows: 4 bytes of cache carry 4 R
// operations, far below what the tensor cores need to be the limit, so the kernel
// is bound by memory, and small calls by latency.  Four warps of a CTA work
// without a barrier between them: each has its own ring of stages (8 KB: TK keys
// and values), loads its own tiles with one TMA per page, S = Q K^T and O += P V
// on mma.sync with R = 16 MT rows, and its own running maximum and sum; the warps
// meet only where an item ends.  A warp's loads run ahead over the borders of
// items.  Two CTAs of an SM hold 8 warps x 3 stages x 8 KB = 192 KB in flight (two
// stages for MT = 2), four times what HBM's latency asks for.  64 sequences of 550
// to 16384 tokens, 32/8 heads of 128: 204 us, 6.06 TB/s.
//
// mma.sync, not tcgen05: 16 rows fill its tile, and its operands come straight
// from registers; a 128-row tcgen05 tile would be 7/8 padding and would pay the
// trip through tensor memory for every tile of 16 keys.
//
// kLine: the line of units is cut evenly (see paged_sm100.cuh), cut items are joined
// by join_kernel.  kClusters, for items of few units: a cluster of CTAs takes whole
// items, its CTAs every n-th unit of one, and the parts are added over distributed
// shared memory, so that nothing has to follow.  kBoth: the same for two passes side by
// side, that over a prefix and that of the sequences, each by CTAs of its own, added by
// join_kernel (8 sequences behind 2043 tokens: 13.2 us on the device, one after another
// 18.2).  kWarps, for many short items: the line is cut evenly over the warps, which never
// meet, so that an item's end costs no barrier and no idle warps.
//
// Code that runs once in a launch costs about 9 cycles an instruction (it comes
// from L2: measured on the first and second pass over the same tile, 8660 and 1580
// cycles), more than the data of a small call.  So the once-run parts are short:
// rolled loops, no division, one copy of the walk over the items, which the
// loading side leaves to the other in a record per stage.
#pragma once

#include <type_traits>

#include "paged_sm100.cuh"

namespace sa {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Clusters: this CTA's place, the two halves of a barrier over all their threads
// (release, acquire), and stores to a CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_st4(uint32_t addr, uint32_t rank, float4 v)
{
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void cluster_st2(uint32_t addr, uint32_t rank, float2 v)
{
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v.x), "f"(v.y)
                 : "memory");
}

// What the loading side of a warp knows about a stage's tile.
struct alignas(16) TileRec {
    int32_t k0;            // first key of the warp's tile
    int32_t flags;         // the item's last tile of this CTA (1), its first unit is here (2), all are (4); its rows * 8
    int32_t parts;         // CTAs that share it (at the last tile, where it begins)
    int32_t hi;            // its keys end before hi
    int32_t first, rb, h;  // the sequence's first token, row block, head
    int32_t base;          // position of the sequence's first new token
};

template <int D, int MT>
struct DecodeCfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int R = 16 * MT;
    static constexpr int TK = 2048 / D;         // keys of a warp's tile (a stage of K: 4 KB)
    static constexpr int UK = TK * kWarps;      // keys of a unit: one tile per warp
    static constexpr int kStages = MT == 1 ? 3 : 2;
    static constexpr int kTileBytes = TK * D * 2;
    static constexpr int kPanel = TK * 128;     // 64 columns x TK rows
    static constexpr int kOffMerge = kWarps * kStages * 2 * kTileBytes;
    static constexpr int kOffQ = kOffMerge + 2 * R * D * 4;      // two warps' O
    static constexpr int kOffMl = kOffQ + (MT == 2 ? R * D * 2 : 0);
    static constexpr int kOffRec = kOffMl + 2 * kWarps * R * 4;  // the warps' maxima and sums
    static constexpr int kOffBar = kOffRec + kWarps * kStages * static_cast<int>(sizeof(TileRec));
    static constexpr int kSmemBytes = kOffBar + kWarps * kStages * 8;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

enum DecodeMode { kLine, kClusters, kWarps, kBoth };

template <int D, int MT, int MODE>
__global__ void __launch_bounds__(128, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ PassParams launch)
{
    using C = DecodeCfg<D, MT>;
    constexpr bool ITEMS = MODE == kClusters || MODE == kBoth, WARP = MODE == kWarps;
    constexpr int R = C::R, TK = C::TK, ST = C::kStages, NW = C::kWarps;
    constexpr int UK = WARP ? TK : C::UK;  // keys of a unit: a tile of each warp, or one tile
    static_assert(!WARP || MT == 1, "warps that never meet hold their queries in registers");
    constexpr int NF = D / 32;  // mma column tiles of a warp's quarter of the columns
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles sit on 1024 bytes
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint8_t* ring = smem + warp * ST * 2 * C::kTileBytes;
    float4* merge = reinterpret_cast<float4*>(smem + C::kOffMerge);  // [2][MT][D / 8][32 lanes]
    float* sm_m = reinterpret_cast<float*>(smem + C::kOffMl);        // [NW][R]
    float* sm_l = sm_m + NW * R;
    const uint32_t sq = smem_addr(smem + C::kOffQ);                  // MT = 2: the item's queries [R][D]
    TileRec* recs = reinterpret_cast<TileRec*>(smem + C::kOffRec) + warp * ST;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * ST;

    // what needs nothing of the kernel before: barriers, the tensor maps' way into the cache
    if (lane == 0) {
        for (int s = 0; s < ST; s++) mbar_init(&bar[s], 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncwarp();
    wait_previous_kernel();
    launch_dependents();
    // this CTA's pass, its place among the pass's CTAs and how many these are
    int rank = 0, CL = 1, cta = blockIdx.x, n_cta = gridDim.x;
    if constexpr (ITEMS) {
        rank = static_cast<int>(cluster_rank());
        CL = static_cast<int>(cluster_size());
    }
    PassParams both;
    if constexpr (MODE == kBoth) {
        both = launch;
        if (cta < launch.side_ctas) {
            n_cta = launch.side_ctas;
            both.over_prefix = 1;
            both.table = launch.side_table;
            both.table_stride = 0;
            both.info = launch.side_info;
            both.acc = launch.side_acc;
            both.acc_ml = launch.side_ml;
        } else {
            cta -= launch.side_ctas;
            n_cta -= launch.side_ctas;
            if (launch.cluster == 1) rank = 0, CL = 1;
        }
    }
    const PassParams& p = MODE == kBoth ? both : launch;
    const SeqView ahead = peek_seq(p);
    // no tail rows yet (a segment's end, where there may be some, lies behind barriers)
    if (MODE == kLine && p.tails != nullptr && tid < R) p.tails[blockIdx.x * R + tid] = TailRow{0, 0};
    const int taker = WARP ? blockIdx.x * NW + warp : blockIdx.x;  // of a piece of the line
    const Piece piece = ITEMS ? find_piece<R, UK, true>(p, ahead, cta / CL, n_cta / CL, 0)
                              : find_piece<R, UK, false>(p, ahead, taker, WARP ? gridDim.x * NW : gridDim.x, 2);
    const int n_seq = p.over_prefix ? 1 : p.B;

    // ---- loads: this warp's tile of every unit of the piece, ST tiles ahead
    constexpr int kTileShift = D == 128 ? 4 : 5;
    static_assert(TK == 1 << kTileShift, "");
    const int row_shift = min(p.page_shift, kTileShift), page_rows = 1 << row_shift;  // rows of one box
    Cursor pc = piece.c;
    if (ITEMS) pc.i = rank;
    // ITEMS: items to come; else units of the item before the piece's end (which may be more than it has)
    int left = ITEMS ? piece.u1 - piece.u0 : piece.avail;
    int issued = 0, live = 0;  // tiles, and those loaded (a warp whose wait ran out goes on without loads)
    bool dead = false;
    // The next tile is looked up one step before its loads go out, so that its page numbers are there by then.
    struct Next {
        TileRec rec;
        int nb, k, page;  // boxes to load; this lane's key and table entry
        bool any;
    } nx;
    auto look_up_next = [&]() {
        nx.any = ITEMS ? left > 0 : pc.i < left;
        if (!nx.any) return;
        const int k0 = pc.u.key(pc.i, UK) + (WARP ? 0 : warp * TK);
        // boxes that begin below the item's last key; a tile with none completes its phase at once
        nx.nb = min((pc.u.hi - k0 + page_rows - 1) >> row_shift, TK >> row_shift);
        if (nx.nb < 0 || pc.i >= pc.u.nt) nx.nb = 0;  // ITEMS: a CTA may have no unit of an item
        nx.k = k0 + lane * page_rows;
        if (lane < nx.nb) nx.page = page_entry(p, pc.b, nx.k);
        const bool last = pc.i + CL >= pc.u.nt || (!ITEMS && pc.i + 1 >= left);
        const int rows = min(pc.s.m * p.group - pc.rb * R, R);
        const int u_item = piece.u1 - left;  // where the item's units begin on the line
        const bool begins = ITEMS || u_item >= piece.u0, whole = ITEMS || (begins && pc.u.nt <= left);
        int parts = 0;
        if (!ITEMS && last && begins && !whole)
            parts = cta_of(piece, u_item + pc.u.nt - 1) - taker + 1;
        nx.rec = TileRec{nx.nb > 0 ? k0 : INT32_MAX, (last ? 1 : 0) | (begins ? 2 : 0) | (whole ? 4 : 0) | rows << 3,
                         parts, pc.u.hi, pc.s.first, pc.rb, pc.h, p.prefix_len + pc.s.p0};
        if (ITEMS && last) left--;
        pc.i += CL;
        if (pc.i >= pc.u.nt) {
            if (!ITEMS) left -= pc.u.nt + piece.w;
            if (left > 0) {
                next_item<R, UK>(p, piece.pb, pc, n_seq);
                if (ITEMS) pc.i = rank;
            } else {
                left = 0;
            }
        }
    };
    auto issue = [&]() {
        const Next now = nx;
        look_up_next();
        const int st = issued % ST;
        const bool skip = (p.debug_flags & 1) && blockIdx.x == 0 && warp == 0 && issued == 0;
        if (lane == 0) {
            recs[st] = now.rec;
            if (!dead) mbar_arrive_expect_tx(&bar[st], skip ? 16 : now.nb * page_rows * D * 4);
        }
        __syncwarp();
        if (lane < now.nb && !skip && !dead) {
            uint8_t* k_dst = ring + st * 2 * C::kTileBytes + lane * page_rows * 128;
            const int row = now.k & ((1 << p.page_shift) - 1);
            const int page = page_of(p, now.page);
            tma_load_5d(k_dst, &tmK, &bar[st], 0, row, 0, now.rec.h, page);
            tma_load_5d(k_dst + C::kTileBytes, &tmV, &bar[st], 0, row, 0, now.rec.h, page);
        }
        issued++;
        if (!dead) live = issued;
    };
    look_up_next();
    if (!nx.any) return;

    // ---- the piece's tiles
    const int rq = lane / 4, cq = (lane % 4) * 2;  // this lane's row (and row + 8) and column pair in an mma tile
    const int off = p.over_prefix ? 0 : p.prefix_len;  // position of key 0
    uint32_t qf[D / 16][4];  // MT = 1: the item's queries
    float o[MT][D / 8][4];
    float m_ref[MT][2], l_sum[MT][2];
    int row_lo[MT][2], row_hi[MT][2];  // keys this lane's rows see: row_lo .. row_hi, and those below cols
    const int cols = p.cols - off;
    TileRec it;                        // of the item
    int lo_lo = 0, lo_hi = 0, hi_lo = 0, hi_hi = 0;  // lowest and highest of the rows' bounds
    int rows_left = 0;
    bool fresh = true;
    issue();
#pragma unroll 1
    for (int j = 0; j < issued; j++) {
        const int st = j % ST;
        const bool first_tile = fresh;
        if (fresh) {
            fresh = false;
            it = recs[st];
            const int r0 = it.rb * R;
            rows_left = it.flags >> 3;
            const int p_lo = p.over_prefix ? piece.pb.lo : it.base + div_group(p, r0);
            const int p_hi = p.over_prefix ? piece.pb.hi : it.base + div_group(p, r0 + rows_left - 1);
            auto first_seen = [&](int pos) {
                return pos < p.n_global ? 0 : p.window >= 0 ? pos - p.window - off : INT32_MAX;
            };
            lo_lo = first_seen(p_lo);
            lo_hi = first_seen(p_hi);
            hi_lo = min(p_lo - off, it.hi - 1);
            hi_hi = min(p_hi - off, it.hi - 1);
            // over the prefix the rows' own positions matter unless every row sees every key
            const bool look_up = p.over_prefix && !(p_lo >= p.prefix_len - 1 && p.window >= 0 && p_hi <= p.window);
            if constexpr (MT == 2) {
                // 32 rows' fragments would take 64 registers, and what spilled was read for every tile (32 sequences
                // of up to 16384 keys, 32 rows a head: 295 us so, 134 like this; 20 to 112 bytes still spill at head
                // size 128).  To shared memory, chunks of 16
                // bytes swizzled; every warp is past the barriers of the item before.
#pragma unroll 1
                for (int c = tid; c < R * (D / 8); c += C::kThreads) {
                    const int r = c / (D / 8), ch = c % (D / 8);
                    const int rr = r0 + min(r, rows_left - 1);  // rows behind the item's last repeat it
                    const int i = div_group(p, rr);
                    const int hq = it.h * p.group + rr - i * p.group;
                    cp_async_16(sq + r * D * 2 + ((ch ^ (r & 7)) * 16),
                                p.q + (it.first + i) * p.q_token + hq * p.q_head + ch * 8);
                }
            }
            // MT = 1: Q fragments of the item's rows, straight from memory
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int r = mt * 16 + rq + 8 * x;
                    const int rr = r0 + min(r, rows_left - 1);
                    const int i = div_group(p, rr), g = rr - i * p.group;
                    const int pos = look_up ? token_position(p, it.first + i) : p.over_prefix ? p_lo : it.base + i;
                    row_lo[mt][x] = first_seen(pos);
                    row_hi[mt][x] = min(pos - off, it.hi - 1);
                    if constexpr (MT == 1) {
                        const int hq = it.h * p.group + g;
                        const __nv_bfloat16* src = p.q + (it.first + i) * p.q_token + hq * p.q_head + cq;
                        const uint32_t* pairs = reinterpret_cast<const uint32_t*>(src);
#pragma unroll
                        for (int kk = 0; kk < D / 16; kk++)
#pragma unroll
                            for (int y = 0; y < 2; y++)
                                qf[kk][x + 2 * y] = r < rows_left ? pairs[kk * 8 + y * 4] : 0u;
                    }
                    m_ref[mt][x] = -INFINITY;
                    l_sum[mt][x] = 0.f;
                }
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int i = 0; i < D / 8; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) o[mt][i][e] = 0.f;
        }
        // tiles up to ST ahead: the stage of the last one has just been read
#pragma unroll 1
        while (issued < j + ST && nx.any) issue();
        if (MT == 2 && first_tile) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
        }
        const int k0 = recs[st].k0, flags = recs[st].flags, parts = recs[st].parts;
        const bool last = flags & 1;
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar[st], (j / ST) & 1, p.timeout))) {
            dead = true;
            if (lane == 0) atomicOr(p.status, ST_PAGED_WAIT);
        }
        if (!dead && k0 < it.hi) {
            const uint32_t ks = smem_addr(ring + st * 2 * C::kTileBytes);
            const uint32_t vs = ks + C::kTileBytes;
            // is every key of the tile seen by every row?
            const int z = k0 + TK - 1;
            const bool full = z <= hi_lo && (k0 >= lo_hi || z < cols);
            // Values no row sees may be anything, and 0 x infinity is not 0: such keys' halves of the V fragments
            // are cleared (the masks are all ones in a full tile; clearing shared memory instead took longer).
            uint32_t keep[TK / 16][2];
#pragma unroll
            for (int kb = 0; kb < TK / 16; kb++)
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    const int kp = k0 + kb * 16 + y * 8 + cq;
                    const bool a = full || (kp <= hi_hi && (kp >= lo_lo || kp < cols));
                    const bool b = full || (kp + 1 <= hi_hi && (kp + 1 >= lo_lo || kp + 1 < cols));
                    keep[kb][y] = (a ? 0xffffu : 0u) | (b ? 0xffff0000u : 0u);
                }
            float s[MT][TK / 8][4];
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int nb = 0; nb < TK / 8; nb++)
#pragma unroll
                    for (int e = 0; e < 4; e++) s[mt][nb][e] = 0.f;
            // S = Q K^T: a matrix of 8 keys x 8 elements per quarter of the warp's addresses
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) {
                uint32_t a[MT][2][4];
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        if constexpr (MT == 2) {
                            const int r = mt * 16 + lane % 16, c = kk * 4 + y * 2 + lane / 16;
                            ldsm_x4(sq + r * D * 2 + ((c ^ (r & 7)) * 16), a[mt][y]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; e++) a[mt][y][e] = qf[2 * kk + y][e];
                        }
                    }
#pragma unroll
                for (int nb = 0; nb < TK / 8; nb++) {
                    const int row = nb * 8 + lane % 8;
                    const int ch = (kk * 4 + lane / 8) % 8;  // 16-byte chunk within the panel
                    uint32_t b[4];
                    ldsm_x4(ks + (kk * 32 / 64) * C::kPanel + row * 128 + ((ch ^ (row & 7)) * 16), b);
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        mma_16816(s[mt][nb], a[mt][0], b[0], b[1]);
                        mma_16816(s[mt][nb], a[mt][1], b[2], b[3]);
                    }
                }
            }
            if (!full) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int nb = 0; nb < TK / 8; nb++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int kp = k0 + nb * 8 + cq + (e & 1);
                            if (!(kp <= row_hi[mt][e >> 1] && (kp >= row_lo[mt][e >> 1] || kp < cols)))
                                s[mt][nb][e] = -INFINITY;
                        }
            }
            // running maximum (a row's four lanes agree), weights, sum
            uint32_t pf[MT][TK / 16][4];
#pragma unroll
            for (int mt = 0; mt < MT; mt++) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int nb = 0; nb < TK / 8; nb++) {
                    mx[0] = fmaxf(mx[0], fmaxf(s[mt][nb][0], s[mt][nb][1]));
                    mx[1] = fmaxf(mx[1], fmaxf(s[mt][nb][2], s[mt][nb][3]));
                }
                float al[2];
                bool scale_o = false;
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
                    mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * p.scale_log2;
                    // the reference follows the maximum only when it grows by 2^8 (as it may: O and the sum
                    // carry the same reference), so O is rarely rescaled
                    const bool grow = mx[x] > m_ref[mt][x] + 8.f;
                    al[x] = grow ? ex2_approx(m_ref[mt][x] - mx[x]) : 1.f;
                    scale_o = scale_o || (grow && m_ref[mt][x] != -INFINITY);  // before that O is 0
                    if (grow) m_ref[mt][x] = mx[x];
                    l_sum[mt][x] *= al[x];
                }
                if (__any_sync(0xffffffffu, scale_o)) {
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        o[mt][i][0] *= al[0];
                        o[mt][i][1] *= al[0];
                        o[mt][i][2] *= al[1];
                        o[mt][i][3] *= al[1];
                    }
                }
                const float mu0 = m_ref[mt][0] == -INFINITY ? 0.f : m_ref[mt][0];
                const float mu1 = m_ref[mt][1] == -INFINITY ? 0.f : m_ref[mt][1];
#pragma unroll
                for (int nb = 0; nb < TK / 8; nb++) {
                    const float e0 = ex2_approx(s[mt][nb][0] * p.scale_log2 - mu0);
                    const float e1 = ex2_approx(s[mt][nb][1] * p.scale_log2 - mu0);
                    const float e2 = ex2_approx(s[mt][nb][2] * p.scale_log2 - mu1);
                    const float e3 = ex2_approx(s[mt][nb][3] * p.scale_log2 - mu1);
                    l_sum[mt][0] += e0 + e1;
                    l_sum[mt][1] += e2 + e3;
                    // weights are rounded to bf16 for the tensor cores; the sum is of the unrounded ones
                    pf[mt][nb / 2][(nb & 1) * 2] = pack_bf16x2(e0, e1);
                    pf[mt][nb / 2][(nb & 1) * 2 + 1] = pack_bf16x2(e2, e3);
                }
            }
            // O += P V
#pragma unroll
            for (int kb = 0; kb < TK / 16; kb++)
#pragma unroll
                for (int d = 0; d < D / 16; d++) {
                    const int row = kb * 16 + (lane / 8 % 2) * 8 + lane % 8;
                    const int ch = (d * 2 + lane / 16) % 8;
                    uint32_t b[4];
                    ldsm_x4_t(vs + (d * 16 / 64) * C::kPanel + row * 128 + ((ch ^ (row & 7)) * 16), b);
#pragma unroll
                    for (int y = 0; y < 4; y++) b[y] &= keep[kb][y & 1];
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        mma_16816(o[mt][2 * d], pf[mt][kb], b[0], b[1]);
                        mma_16816(o[mt][2 * d + 1], pf[mt][kb], b[2], b[3]);
                    }
                }
        }
        __syncwarp();  // the stage is read
        if (!last) continue;

        // ---- the item's last tile here
        fresh = true;
        // An item that is not all in this piece leaves a part.
        const bool begins = flags & 2, whole = flags & 4;
        const int slot = (2 * taker + (begins ? 1 : 0)) * R;
        RowInfo ri{0, 0, 0, 0};
        if (!whole && begins)
            ri = RowInfo{p.part_row0 + slot, p.part_row0 + slot + R, parts, 2 * R};
        // columns col + 8 i, + 1 of row r; `first` where the row's sum and its entry are to be written too
        auto write = [&](auto n_const, int r, int col, auto& v, float m, float l, bool first) {
            constexpr int N = decltype(n_const)::value;
            const int rr = it.rb * R + r;
            const int i_tok = div_group(p, rr);
            const int64_t t = it.first + i_tok;
            const int hq = it.h * p.group + rr - i_tok * p.group;
            const int64_t at = t * p.Hq + hq;
            if (whole && p.acc == nullptr) {
                if (MODE == kClusters && p.pre_acc != nullptr) {  // add the row's part over the prefix, or its parts
                    auto add = [&](const float2 (&w)[N], float2 ml) {
                        const float mn = fmaxf(m, ml.x);
                        const float fo = m == -INFINITY ? 0.f : ex2_approx(m - mn);
                        const float fn = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
#pragma unroll
                        for (int i = 0; i < N; i++) {
                            v[i][0] = v[i][0] * fo + w[i].x * fn;
                            v[i][1] = v[i][1] * fo + w[i].y * fn;
                        }
                        l = l * fo + ml.y * fn;
                        m = mn;
                    };
                    RowInfo pi{0, 0, 0, 0};
                    if (p.pre_info != nullptr) pi = p.pre_info[at];
                    if (pi.n == 0) {
                        float2 w[N];
#pragma unroll
                        for (int i = 0; i < N; i++)
                            w[i] = *reinterpret_cast<const float2*>(p.pre_acc + at * D + col + i * 8);
                        add(w, p.pre_ml[at]);
                    } else if (in_range(pi, p.part_rows)) {
                        constexpr int K = N == 1 ? 4 : 2;  // in flight
#pragma unroll 1
                        for (int k0 = 0; k0 < pi.n; k0 += K) {
                            float2 ml[K], w[K][N];
#pragma unroll
                            for (int k = 0; k < K; k++) {
                                const int kk = min(k0 + k, pi.n - 1);  // past the last: not added
                                const int64_t from = kk == 0 ? pi.first : pi.second + int64_t(kk - 1) * pi.stride;
                                ml[k] = p.pre_part_ml[from];
#pragma unroll
                                for (int i = 0; i < N; i++)
                                    w[k][i] = *reinterpret_cast<const float2*>(p.pre_part_o + from * D + col + i * 8);
                            }
#pragma unroll
                            for (int k = 0; k < K; k++)
                                if (k0 + k < pi.n) add(w[k], ml[k]);
                        }
                    }
                }
                const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
                __nv_bfloat16* dst = p.o + t * p.o_token + hq * p.o_head + col;
#pragma unroll
                for (int i = 0; i < N; i++)
                    *reinterpret_cast<uint32_t*>(dst + i * 8) = pack_bf16x2(v[i][0] * inv, v[i][1] * inv);
                if (first) p.lse[at] = lse_of(m, __log2f(l), l);
            } else {
                float* dst = (whole ? p.acc + at * D : p.part_o + static_cast<int64_t>(slot + r) * D) + col;
#pragma unroll
                for (int i = 0; i < N; i++) *reinterpret_cast<float2*>(dst + i * 8) = make_float2(v[i][0], v[i][1]);
                if (first) (whole ? p.acc_ml[at] : p.part_ml[slot + r]) = make_float2(m, l);
            }
            if (MODE == kLine && first && p.tails != nullptr && begins && !whole)
                p.tails[blockIdx.x * R + r] = TailRow{static_cast<int32_t>(at), ri.n};
            if (first && p.info != nullptr && begins)
                p.info[at] = RowInfo{ri.first + (whole ? 0 : r), ri.second + (whole ? 0 : r), ri.n, ri.stride};
        };
        if constexpr (WARP) {
#pragma unroll
            for (int x = 0; x < 2; x++) {
                float l = l_sum[0][x];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                float v[D / 8][2];
#pragma unroll
                for (int i = 0; i < D / 8; i++) {
                    v[i][0] = o[0][i][2 * x];
                    v[i][1] = o[0][i][2 * x + 1];
                }
                if (rq + 8 * x < rows_left)
                    write(std::integral_constant<int, D / 8>{}, rq + 8 * x, cq, v, m_ref[0][x], l, lane % 4 == 0);
            }
        } else {
            // ---- add the four warps.  Each warp's O goes to shared memory, two warps
            // at a time, and each warp sums a quarter of the columns, weighted by 2^(its maximum - the common one).
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    l_sum[mt][x] += __shfl_xor_sync(0xffffffffu, l_sum[mt][x], 1);
                    l_sum[mt][x] += __shfl_xor_sync(0xffffffffu, l_sum[mt][x], 2);
                    if (lane % 4 == 0) {
                        sm_m[warp * R + mt * 16 + rq + 8 * x] = m_ref[mt][x];
                        sm_l[warp * R + mt * 16 + rq + 8 * x] = l_sum[mt][x];
                    }
                }
            float M[MT][2], L[MT][2], acc[MT][NF][4];
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int i = 0; i < NF; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[mt][i][e] = 0.f;
#pragma unroll 1
            for (int half = 0; half < 2; half++) {
                if (warp / 2 == half) {
#pragma unroll
                    for (int mt = 0; mt < MT; mt++)
#pragma unroll
                        for (int i = 0; i < D / 8; i++)
                            merge[(((warp & 1) * MT + mt) * (D / 8) + i) * 32 + lane] =
                                make_float4(o[mt][i][0], o[mt][i][1], o[mt][i][2], o[mt][i][3]);
                }
                __syncthreads();
                if (half == 0) {
#pragma unroll
                    for (int mt = 0; mt < MT; mt++)
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const int r = mt * 16 + rq + 8 * x;
                            M[mt][x] = fmaxf(fmaxf(sm_m[r], sm_m[R + r]), fmaxf(sm_m[2 * R + r], sm_m[3 * R + r]));
                            L[mt][x] = 0.f;
                        }
                }
#pragma unroll 1
                for (int w = 2 * half; w < 2 * half + 2; w++) {
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const int r = w * R + mt * 16 + rq + 8 * x;
                            f[x] = sm_m[r] == -INFINITY ? 0.f : ex2_approx(sm_m[r] - M[mt][x]);
                            L[mt][x] += f[x] * sm_l[r];
                        }
#pragma unroll
                        for (int i = 0; i < NF; i++) {
                            const float4 v = merge[(((w & 1) * MT + mt) * (D / 8) + warp * NF + i) * 32 + lane];
                            acc[mt][i][0] += f[0] * v.x;
                            acc[mt][i][1] += f[0] * v.y;
                            acc[mt][i][2] += f[1] * v.z;
                            acc[mt][i][3] += f[1] * v.w;
                        }
                    }
                }
                __syncthreads();
            }
            if (ITEMS && CL > 1) {
                // ---- add the CTAs of the cluster.  Of the item's F column pairs of two rows (in the order of the mma
                // tiles' lanes) CTA k takes those from k F / CL on: all send theirs to its shared memory, with the
                // rows' maxima and sums, and after one barrier it adds what came.
                constexpr int F = MT * (D / 8) * 32;
                const int shift = 31 - __clz(F) + 1 - __ffs(CL), share = 1 << shift;  // F / CL: both are powers of two
                float2* got_ml = reinterpret_cast<float2*>(merge + F);  // [CL][R]
                cluster_arrive();
                cluster_wait();  // every CTA has added its warps: their buffer is free for what comes
#pragma unroll
                for (int mt = 0; mt < MT; mt++) {
#pragma unroll
                    for (int i = 0; i < NF; i++) {
                        const int f = (mt * (D / 8) + warp * NF + i) * 32 + lane;
                        cluster_st4(smem_addr(merge + rank * share + (f & (share - 1))), f >> shift,
                                    make_float4(acc[mt][i][0], acc[mt][i][1], acc[mt][i][2], acc[mt][i][3]));
                    }
#pragma unroll
                    for (int x = 0; x < 2; x++)  // lane 4 rq + c of warp w: to CTA w + 4 (c & 1)
                        if (warp + 4 * (lane & 1) < CL && (lane & 3) < 2)
                            cluster_st2(smem_addr(got_ml + rank * R + mt * 16 + rq + 8 * x), warp + 4 * (lane & 1),
                                        make_float2(M[mt][x], L[mt][x]));
                }
                __syncwarp();
                cluster_arrive();
                cluster_wait();
#pragma unroll 1
                for (int f0 = tid; f0 < share; f0 += C::kThreads) {
                    const int f = rank * share + f0;
                    const int r = f / ((D / 8) * 32) * 16 + f % 32 / 4, col = f / 32 % (D / 8) * 8 + f % 4 * 2;
                    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, v[2][1][2] = {{{0.f, 0.f}}, {{0.f, 0.f}}};
#pragma unroll 4
                    for (int k = 0; k < CL; k++)
#pragma unroll
                        for (int x = 0; x < 2; x++) m[x] = fmaxf(m[x], got_ml[k * R + r + 8 * x].x);
#pragma unroll 4
                    for (int k = 0; k < CL; k++) {
                        const float4 a = merge[k * share + f0];
                        const float2 m0 = got_ml[k * R + r], m1 = got_ml[k * R + r + 8];
                        const float w0 = m0.x == -INFINITY ? 0.f : ex2_approx(m0.x - m[0]);
                        const float w1 = m1.x == -INFINITY ? 0.f : ex2_approx(m1.x - m[1]);
                        v[0][0][0] += w0 * a.x;
                        v[0][0][1] += w0 * a.y;
                        v[1][0][0] += w1 * a.z;
                        v[1][0][1] += w1 * a.w;
                        l[0] += w0 * m0.y;
                        l[1] += w1 * m1.y;
                    }
#pragma unroll 1
                    for (int x = 0; x < 2; x++) {
                        const bool hi = x;
                        float u[1][2] = {{hi ? v[1][0][0] : v[0][0][0], hi ? v[1][0][1] : v[0][0][1]}};
                        if (r + 8 * x < rows_left)
                            write(std::integral_constant<int, 1>{}, r + 8 * x, col, u, hi ? m[1] : m[0],
                                  hi ? l[1] : l[0], col == 0);
                    }
                }
                if (j + 1 < issued) __syncthreads();  // read, before the next item's warps write there
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int r = mt * 16 + rq + 8 * x;
                        if (r >= rows_left) continue;
                        float v[NF][2];
#pragma unroll
                        for (int i = 0; i < NF; i++) {
                            v[i][0] = acc[mt][i][2 * x];
                            v[i][1] = acc[mt][i][2 * x + 1];
                        }
                        write(std::integral_constant<int, NF>{}, r, warp * (D / 4) + cq, v, M[mt][x], L[mt][x],
                              warp == 0 && lane % 4 == 0);
                    }
            }
        }
    }
    if (dead) {
        // copies still in flight land before the CTA's memory goes away
        for (int j = max(live - ST, 0); j < live; j++) mbar_wait(&bar[j % ST], (j / ST) & 1, p.timeout);
    }
}

}  // namespace sa
