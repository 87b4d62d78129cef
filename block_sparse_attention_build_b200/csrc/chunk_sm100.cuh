// Attention of many rows (pieces of prompts, whole prompts, all sequences of a
// batch over their shared prefix) over a paged cache, on the tensor cores.
//
// An item is 256 rows: two slots of 128 (a tensor-memory lane per row) that read
// the same keys, so that a key tile serves 2 x 128 rows and the tensor cores work
// on one slot while the other slot's softmax runs.  At 256 rows a unit of 128 keys
// is 4 * 256 * 128 * D operations on 512 D bytes: the tensor cores and the
// exponentials bound it, not memory.
//
// Warp roles (384 threads, three warpgroups, with fwd_kernel's register split):
//   warp 0      producer: walks the CTA's items, describes each segment (the units
//               of an item in this CTA's piece) in a two-entry ring that the other
//               roles read, and loads K and V tiles through one ring of stages, a
//               page (or 128 places of one) per TMA, its lanes side by side
//   warp 1      allocates tensor memory; one lane issues every tcgen05.mma
//   warps 2, 3  Q of slot A, slot B: rows lie where tokens and heads put them, so
//               they are gathered with cp.async into the swizzled layout that TMA
//               would write, while the previous item's last softmax and PV still run
//   warps 4-7   softmax of slot A, warps 8-11 of slot B: a thread per row
//
// Order of the tensor cores: PV_A(j), S_A(j+1), PV_B(j), S_B(j+1), 512 cycles each
// at D = 128.  Tensor memory (512 columns): S_A, S_B (128 each; P over their first
// half), O_A, O_B (D each).  Two threads to a row (half of the keys each, the row's
// maximum exchanged) were slower: 2190 us against 2060 for 4096 new tokens behind
// 28672, 32/8 heads of 128, where the board runs at its 1000 W limit.
// Places no row sees may hold anything: scores there are replaced, and slot A's
// threads clear the tile's V rows before P V (0 x infinity is not 0).
//
// Every wait is bounded; on expiry the status word is set, all roles leave their
// loops, copies and MMAs in flight are waited for and tensor memory is freed.
#pragma once

#include "fwd_sm100.cuh"
#include "paged_sm100.cuh"

namespace sa {

// One segment, as the producer describes it.
struct Segment {
    int32_t n;                 // units here; 0: no more segments
    int32_t i, ns, bs, hi;     // first of them, and where units and keys lie (see Units)
    int32_t first, rows, rb, h, base;  // item: first token, its rows, row block, head, position of the first token
    int32_t begins, whole;     // the item's first unit is here; all of them are
    int32_t parts;             // CTAs that share it (where it begins)
    int32_t pad[3];
    __device__ __forceinline__ int key(int j) const
    {
        const int u = i + j;
        return (u < ns ? u : bs + (u - ns)) * 128;
    }
};

template <int D>
struct ChunkCfg {
    static constexpr int kThreads = 384;
    static constexpr int R = 256;
    static constexpr int UK = 128;
    static constexpr int kTileBytes = UK * D * 2;
    static constexpr int kStages = kRingBytes / kTileBytes;  // 4 (D = 128) or 8
    static constexpr int kPanel = 128 * 128;                 // 64 columns x 128 rows
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kOffRing = 2 * kQBytes;
    static constexpr int kStageRow = 80;  // 64 bytes of a row: 16-byte accesses of consecutive rows meet no bank twice
    static constexpr int kOffStage = kOffRing + kStages * kTileBytes;  // a softmax warp's 32 rows each
    static constexpr int kOffSeg = kOffStage + 8 * 32 * kStageRow;
    static constexpr int kOffBar = kOffSeg + 2 * static_cast<int>(sizeof(Segment));
    static constexpr int kNumBars = 2 * kStages + 2 * 6 + 2 * 2 + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmemUsed = kOffMisc + 16;
    // at least this much, so that one CTA owns the SM's tensor memory
    static constexpr int kSmemBytes = kSmemUsed > 120 * 1024 ? kSmemUsed : 120 * 1024;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(2 * UK + 2 * D <= 512, "tensor memory budget");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 2^x for two lanes on the FMA pipe, as exp2_poly_x2 but of degree 5 (relative error
// 2.2e-7, fitted by csrc/fit_exp2.py): the sum, which the LSE is taken from, then keeps
// 32 bits' worth.  With degree 3 the LSE of rows with few keys was off by 7e-5; the two
// terms more cost half a percent.
__device__ __forceinline__ void exp2_poly5_x2(uint64_t x2, float& p0, float& p1)
{
    constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: x + kRound rounds x to an integer
    const uint64_t t2 = f2_add(x2, f2_pack(kRound, kRound));
    const uint64_t j2 = f2_add(t2, f2_pack(-kRound, -kRound));
    const uint64_t f2 = f2_fma(j2, f2_pack(-1.f, -1.f), x2);
    uint64_t q2 = f2_fma(f2_pack(0.0013276472454890609f, 0.0013276472454890609f), f2,
                         f2_pack(0.009675540961325169f, 0.009675540961325169f));
    q2 = f2_fma(q2, f2, f2_pack(0.05550713092088699f, 0.05550713092088699f));
    q2 = f2_fma(q2, f2, f2_pack(0.24022120237350464f, 0.24022120237350464f));
    q2 = f2_fma(q2, f2, f2_pack(0.6931469440460205f, 0.6931469440460205f));
    q2 = f2_fma(q2, f2, f2_pack(1.0000001192092896f, 1.0000001192092896f));
    float x0, x1, t0, t1, q0, q1;
    f2_unpack(x2, x0, x1);
    f2_unpack(t2, t0, t1);
    // the low bits of t hold j (two's complement): shifted into the exponent field of 1 they make 2^j, by which q
    // is multiplied (added to q's own bits they would make 3.4e38 of a NaN)
    f2_unpack(f2_mul(q2, f2_pack(__int_as_float(0x3f800000 + (__float_as_int(t0) << 23)),
                                 __int_as_float(0x3f800000 + (__float_as_int(t1) << 23)))), q0, q1);
    p0 = x0 < -125.f ? 0.f : q0;
    p1 = x1 < -125.f ? 0.f : q1;
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ PassParams p)
{
    using C = ChunkCfg<D>;
    constexpr int S = C::kStages, R = C::R, UK = C::UK;
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles sit on 1024 bytes
    uint8_t* sQ = smem;
    uint8_t* ring = smem + C::kOffRing;
    Segment* segs_ring = reinterpret_cast<Segment*>(smem + C::kOffSeg);
    uint64_t* ring_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [S]
    uint64_t* ring_empty = ring_full + S;                                  // [S]
    uint64_t* q_full = ring_empty + S;     // [2]
    uint64_t* q_empty = q_full + 2;        // [2] the slot's last S MMA of the item is done
    uint64_t* s_full = q_empty + 2;        // [2]
    uint64_t* p_full = s_full + 2;         // [2]
    uint64_t* o_full = p_full + 2;         // [2]
    uint64_t* o_empty = o_full + 2;        // [2]
    uint64_t* info_full = o_empty + 2;     // [2] a segment is described
    uint64_t* info_empty = info_full + 2;  // [2] all roles are done with it
    uint64_t* drain = info_empty + 2;      // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;

    if (threadIdx.x == 64) {
        for (int i = 0; i < S; i++) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 1);
        }
        for (int x = 0; x < 2; x++) {
            mbar_init(&q_full[x], 32);
            mbar_init(&q_empty[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);    // a lane of each softmax warp of the slot
            mbar_init(&o_full[x], 1);
            mbar_init(&o_empty[x], 4);
            mbar_init(&info_full[x], 1);
            mbar_init(&info_empty[x], 1 + 2 + 8);  // a lane of the MMA, Q and softmax warps
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 96) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    wait_previous_kernel();
    launch_dependents();
    if (p.tails != nullptr && threadIdx.x < R) p.tails[blockIdx.x * R + threadIdx.x] = TailRow{0, 0};
    Piece piece;
    if (warp == 0) piece = find_piece<R, UK, false>(p, peek_seq(p), blockIdx.x, gridDim.x, 3);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const long long lim = p.timeout;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, ST_PAGED_WAIT);
    };
    // every lane polls; the outcome is made warp-uniform
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim) && !*abort_flag);
    };
    // The next segment (k-th): false at the end or when a wait ran out.
    bool ok = true;
    auto open_segment = [&](int k) -> const Segment* {
        const Segment* g = &segs_ring[k & 1];
        ok = wait(&info_full[k & 1], (k >> 1) & 1);
        return ok && g->n > 0 ? g : nullptr;
    };
    auto close_segment = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&info_empty[k & 1]);
    };
    // warp-uniform warpgroup index, so that the register split applies per branch
    const int wg = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 128, 0);

    if (wg == 0) {
        regs_dec<kRegsControl>();
        if (warp == 0) {
            // ============================================================ producer
            const int n_seq = p.over_prefix ? 1 : p.B;
            const int row_shift = min(p.page_shift, 7), page_rows = 1 << row_shift;  // rows of one box
            constexpr int P = D / 64;  // column panels
            const int box = lane / P, panel = lane % P;
            Cursor c = piece.c;
            int left = piece.avail;  // units of the item before the piece's end (which may be more than it has)
            int pos = 0, k_seg = 0;
            for (;; k_seg++) {
                // describe the segment
                if (!(ok = wait(&info_empty[k_seg & 1], ((k_seg >> 1) & 1) ^ 1))) break;
                const int n = left > c.i ? min(c.u.nt, left) - c.i : 0;
                if (lane == 0) {
                    Segment& g = segs_ring[k_seg & 1];
                    g.n = n;
                    if (n > 0) {
                        const int u_item = piece.u1 - left;  // where the item's units begin on the line
                        g.i = c.i;
                        g.ns = c.u.ns;
                        g.bs = c.u.bs;
                        g.hi = c.u.hi;
                        g.first = c.s.first;
                        g.rows = min(c.s.m * p.group - c.rb * R, R);
                        g.rb = c.rb;
                        g.h = c.h;
                        g.base = p.prefix_len + c.s.p0;
                        g.begins = u_item >= piece.u0;
                        g.whole = u_item >= piece.u0 && c.u.nt <= left;
                        g.parts = 0;
                        if (g.begins && !g.whole) g.parts = cta_of(piece, u_item + c.u.nt - 1) - static_cast<int>(blockIdx.x) + 1;
                    }
                    mbar_arrive(&info_full[k_seg & 1]);
                }
                __syncwarp();
                if (n == 0) break;
                // the pages of a tile are looked up while the one before it is loaded
                auto tile_key = [&](int j) { return c.u.key(c.i + j, UK); };
                auto boxes = [&](int k0) {
                    return min(max((c.u.hi - k0 + page_rows - 1) >> row_shift, 0), UK >> row_shift);
                };
                auto page_at = [&](int k0) { return box < boxes(k0) ? page_entry(p, c.b, k0 + box * page_rows) : 0; };
                int pg_next = page_at(tile_key(0));
                for (int j = 0; j < n && ok; j++) {
                    const int k0 = tile_key(j), nb = boxes(k0), pg = page_of(p, pg_next);
                    if (j + 1 < n) pg_next = page_at(tile_key(j + 1));
                    const int row = (k0 + box * page_rows) & ((1 << p.page_shift) - 1);
#pragma unroll 1
                    for (int v = 0; v < 2; v++) {  // K, then V
                        const int st = pos % S;
                        if (!(ok = wait(&ring_empty[st], ((pos / S) & 1) ^ 1))) break;
                        const bool skip = (p.debug_flags & 1) && blockIdx.x == 0 && pos == 0;
                        if (lane == 0) mbar_arrive_expect_tx(&ring_full[st], skip ? 16 : nb * page_rows * D * 2);
                        __syncwarp();
                        if (box < nb && !skip)
                            tma_load_5d(ring + st * C::kTileBytes + panel * C::kPanel + box * page_rows * 128,
                                        v == 0 ? &tmK : &tmV, &ring_full[st], 0, row, panel, c.h, pg);
                        __syncwarp();
                        pos++;
                    }
                }
                if (!ok) break;
                left -= c.u.nt + piece.w;
                if (left > 0)
                    next_item<R, UK>(p, piece.pb, c, n_seq);
                else
                    left = c.i = 0;
            }
            if (!ok) {
                if (lane == 0) fail();
                // copies still in flight land before the CTA's memory goes away
                for (int i = pos > S ? pos - S : 0; i < pos; i++) mbar_wait(&ring_full[i % S], (i / S) & 1, lim);
            }
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, UK, false, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t qd = smem_desc_sw128(smem_addr(sQ), 16, 1024);
            const uint64_t kd = smem_desc_sw128(smem_addr(ring), 16, 1024);
            const uint64_t vd = smem_desc_sw128(smem_addr(ring), C::kPanel, 1024);
            const uint32_t q_lo = static_cast<uint32_t>(qd), k_lo = static_cast<uint32_t>(kd);
            const uint32_t v_lo = static_cast<uint32_t>(vd), d_hi = static_cast<uint32_t>(qd >> 32);
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) tc_commit(bar);
                __syncwarp();
            };
            auto issue_s = [&](int x, int stage) {
                const uint32_t a0 = q_lo + static_cast<uint32_t>((x * C::kQBytes) >> 4);
                const uint32_t b0 = k_lo + static_cast<uint32_t>((stage * C::kTileBytes) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++) {
                        const uint32_t off = static_cast<uint32_t>(((kk / 4) * C::kPanel + (kk % 4) * 32) >> 4);
                        mma_ss(tm + x * UK, desc_from_halves(a0 + off, d_hi), desc_from_halves(b0 + off, d_hi), idesc_s,
                               kk > 0 ? 1u : 0u);
                    }
                }
                __syncwarp();
            };
            auto issue_pv = [&](int x, int stage, bool accumulate) {
                const uint32_t b0 = v_lo + static_cast<uint32_t>((stage * C::kTileBytes) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < UK / 16; kk++)
                        mma_ts(tm + 2 * UK + x * D, tm + x * UK + kk * 8,
                               desc_from_halves(b0 + static_cast<uint32_t>(kk * 128), d_hi), idesc_o,
                               (accumulate || kk > 0) ? 1u : 0u);
                }
                __syncwarp();
            };
            int steps[2] = {0, 0};  // S/P handshakes per slot
            int segs[2] = {0, 0};   // segments per slot (phases of q_full, o_full, o_empty)
            int pos = 0;
            for (int k_seg = 0;; k_seg++) {
                const Segment* g = open_segment(k_seg);
                if (!g) break;
                const int n = g->n;
                const int nx = g->rows > 128 ? 2 : 1;
                close_segment(k_seg);
                ok = wait(&ring_full[pos % S], (pos / S) & 1);
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    if (x >= nx || !ok) continue;
                    ok = wait(&q_full[x], segs[x] & 1);
                    if (!ok) break;
                    tc_fence_after_sync();
                    issue_s(x, pos % S);
                    commit(&s_full[x]);
                    if (n == 1) commit(&q_empty[x]);
                }
                if (!ok) break;
                commit(&ring_empty[pos % S]);
                for (int j = 0; j < n && ok; j++) {
                    const bool last = j == n - 1;
                    const int pv = pos + 2 * j + 1;  // V(j)
                    const int pk = pv + 1;           // K(j + 1)
                    ok = wait(&ring_full[pv % S], (pv / S) & 1);
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        if (x >= nx || !ok) continue;
                        ok = wait(&p_full[x], steps[x] & 1);
                        if (ok && j == 0 && segs[x] > 0) ok = wait(&o_empty[x], (segs[x] - 1) & 1);
                        if (!ok) break;
                        steps[x]++;
                        tc_fence_after_sync();
                        issue_pv(x, pv % S, j > 0);
                        if (last) {
                            commit(&o_full[x]);
                        } else {
                            if (x == 0 && !(ok = wait(&ring_full[pk % S], (pk / S) & 1))) break;
                            tc_fence_after_sync();
                            issue_s(x, pk % S);
                            commit(&s_full[x]);
                            if (j + 2 == n) commit(&q_empty[x]);  // the slot's last read of Q
                        }
                    }
                    if (!ok) break;
                    commit(&ring_empty[pv % S]);
                    if (!last) commit(&ring_empty[pk % S]);
                }
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 2; x++)
                    if (x < nx) segs[x]++;
                pos += 2 * n;
            }
            if (!ok && lane == 0) fail();
            // all issued tensor-core work is finished before the memory is released
            commit(drain);
            if (!__all_sync(0xffffffffu, mbar_wait(drain, 0, lim)) && lane == 0) atomicOr(p.status, ST_DRAIN_WAIT);
        } else {
            // ============================================================ Q of slot x
            const int x = warp - 2;
            constexpr int L = D / 8;        // lanes of a row, 16 bytes each
            constexpr int RW = 32 / L;      // rows of one step
            const int ch = lane % L;
            const uint32_t dst0 = smem_addr(sQ) + x * C::kQBytes + (ch / 8) * C::kPanel;
            int loads = 0;
            for (int k_seg = 0;; k_seg++) {
                const Segment* g = open_segment(k_seg);
                if (!g) break;
                const int rows = g->rows - x * 128;
                if (rows > 0) {
                    const int r0 = g->rb * R + x * 128, h0 = g->h * p.group;
                    const __nv_bfloat16* q0 = p.q + static_cast<int64_t>(g->first) * p.q_token;
                    if (!(ok = wait(&q_empty[x], (loads & 1) ^ 1))) break;
#pragma unroll 1
                    for (int b = 0; b < 128; b += 32) {
                        // where row b + lane lies; rows behind the item's last repeat it: what they compute is
                        // not written
                        const int rr = r0 + min(b + lane, rows - 1);
                        const int i = div_group(p, rr);
                        const int64_t at = i * p.q_token + (h0 + rr - i * p.group) * p.q_head;
#pragma unroll
                        for (int s = 0; s < 32; s += RW) {
                            const int r = s + lane / L;
                            const int64_t src = __shfl_sync(0xffffffffu, at, r);
                            cp_async_16(dst0 + (b + r) * 128 + (((ch % 8) ^ (r & 7)) * 16), q0 + src + ch * 8);
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    mbar_arrive(&q_full[x]);
                    loads++;
                }
                close_segment(k_seg);
            }
            if (!ok && lane == 0) fail();
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ================================================================ softmax
        const int x = wg - 1;             // slot
        const int quarter = warp & 3;     // tensor-memory lanes this warp may access
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32);
        const uint32_t t_s = tmem_addr(tmem, lane_base, static_cast<uint32_t>(x * UK));  // P is written over it
        const uint32_t t_o = tmem_addr(tmem, lane_base, static_cast<uint32_t>(2 * UK + x * D));
        uint8_t* stage = smem + C::kOffStage + (warp - 4) * 32 * C::kStageRow;
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
        const int off = p.over_prefix ? 0 : p.prefix_len;
        PassBounds bounds{0, 0};  // over the prefix: of all rows' positions
        if (p.over_prefix) bounds = pass_bounds(p);
        int steps = 0, segs = 0;
        int pos = 0;  // ring items of the segments before
        for (int k_seg = 0;; k_seg++) {
            const Segment* g = open_segment(k_seg);
            if (!g) break;
            const int n = g->n;
            const int rows = g->rows - x * 128;  // of this slot
            if (rows <= 0) {
                pos += 2 * n;
                close_segment(k_seg);
                continue;
            }
            float m_ref = -INFINITY;  // running max, log2 units of the scaled score
            float l_sum = 0.f;
            int row_lo, row_hi, lo_lo, lo_hi, hi_lo, hi_item;  // keys seen: by this row, and over the slot's rows
            {
                const int r0 = g->rb * R + x * 128;
                const int base = g->base;
                const int i_tok = div_group(p, r0 + min(row, rows - 1));
                const int p_lo = p.over_prefix ? bounds.lo : base + div_group(p, r0);
                const int p_hi = p.over_prefix ? bounds.hi : base + div_group(p, r0 + min(rows, 128) - 1);
                const int p_item = p.over_prefix ? bounds.hi : base + div_group(p, g->rb * R + g->rows - 1);
                auto first_seen = [&](int q) {
                    return q < p.n_global ? 0 : p.window >= 0 ? q - p.window - off : INT32_MAX;
                };
                const bool look_up = p.over_prefix && !(p_lo >= p.prefix_len - 1 && p.window >= 0 && p_hi <= p.window);
                const int pr = look_up ? token_position(p, g->first + i_tok) : p.over_prefix ? p_lo : base + i_tok;
                row_lo = first_seen(pr);
                row_hi = min(pr - off, g->hi - 1);
                lo_lo = first_seen(p_lo);
                lo_hi = first_seen(p_hi);
                hi_lo = min(p_lo - off, g->hi - 1);
                hi_item = min(p_item - off, g->hi - 1);
            }
            const int cols = p.cols - off;
#pragma unroll 1
            for (int j = 0; j < n; j++) {
                const int kv0 = g->key(j);
                const bool masked = !(kv0 + UK - 1 <= hi_lo && (kv0 >= lo_hi || kv0 + UK <= cols));
                if (masked && x == 0) {
                    // this thread's V row of the tile, where no row of the item sees it
                    const int kp = kv0 + row;
                    const bool seen = kp <= hi_item && (kp >= lo_lo || kp < cols);
                    if (__any_sync(0xffffffffu, !seen)) {
                        const int pv = pos + 2 * j + 1;
                        if (!(ok = wait(&ring_full[pv % S], (pv / S) & 1))) break;
                        if (!seen) {
                            uint8_t* v = ring + (pv % S) * C::kTileBytes + row * 128;
#pragma unroll 1
                            for (int q = 0; q < D / 8; q++)
                                *reinterpret_cast<uint4*>(v + (q / 8) * C::kPanel + (q % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                if (!(ok = wait(&s_full[x], steps & 1))) break;
                tc_fence_after_sync();
                float s[UK];
                {
                    uint32_t r[UK / 32][32];
#pragma unroll
                    for (int q = 0; q < UK / 32; q++) tmem_ld_32x32b_x32(t_s + 32 * q, r[q]);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < UK / 32; q++) reg_fence(r[q]);
#pragma unroll
                    for (int q = 0; q < UK; q++) s[q] = __uint_as_float(r[q / 32][q % 32]);
                }
                if (masked) {
#pragma unroll
                    for (int w = 0; w < UK / 32; w++) {
                        const int b = kv0 + 32 * w;
                        const uint32_t m = (bits_between(row_lo - b, 31) | bits_between(0, cols - 1 - b)) &
                                           bits_between(0, row_hi - b);
#pragma unroll
                        for (int q = 0; q < 32; q++) s[32 * w + q] = (m >> q) & 1u ? s[32 * w + q] : -INFINITY;
                    }
                }
                // row max: 16 independent chains of three-input max
                float mx[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    mx[i] = fmax3(s[i], s[16 + i], s[32 + i]);
                    mx[i] = fmax3(mx[i], s[48 + i], s[64 + i]);
                    mx[i] = fmaxf(fmax3(mx[i], s[80 + i], s[96 + i]), s[112 + i]);
                }
                const float m_tile =
                    fmax3(fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmax3(mx[6], mx[7], mx[8])),
                          fmax3(fmax3(mx[9], mx[10], mx[11]), fmax3(mx[12], mx[13], mx[14]), mx[15]), -INFINITY) *
                    p.scale_log2;
                // Rescale only when the max grows by more than 2^8: O and the sum carry the same reference.
                const bool grow = m_tile > m_ref + 8.f;
                float alpha = 1.f;
                if (grow) {
                    alpha = ex2_approx(m_ref - m_tile);  // 0 when m_ref = -inf
                    l_sum *= alpha;
                    m_ref = m_tile;
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                const uint64_t neg_m = f2_pack(-m_use, -m_use);
                // p = 2^(s * scale_log2 - m): 7 of every 8 pairs on the MUFU unit, 1 on the FMA pipe (2: 1 % slower)
                uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < UK; q += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const uint64_t x2 = f2_fma(f2_pack(s[q + 2 * i], s[q + 2 * i + 1]), scale2, neg_m);
                        float e0, e1;
                        if ((i & 7) < 1) {
                            exp2_poly5_x2(x2, e0, e1);
                        } else {
                            float x0, x1;
                            f2_unpack(x2, x0, x1);
                            e0 = ex2_approx(x0);
                            e1 = ex2_approx(x1);
                        }
                        acc[i & 3] = f2_add(acc[i & 3], f2_pack(e0, e1));
                        pk[i] = pack_bf16x2(e0, e1);
                    }
                    tmem_st_32x32b_x32(t_s + q / 2, pk);
                }
                {
                    float a0, a1, b0, b1;
                    f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
                    f2_unpack(f2_add(acc[2], acc[3]), b0, b1);
                    l_sum += (a0 + a1) + (b0 + b1);
                }
                if (j > 0 && __any_sync(0xffffffffu, grow)) {
                    // O_X holds every product up to tile j-1 (the commit of S_X(j) covers PV_X(j-1))
#pragma unroll 1
                    for (int q = 0; q < D; q += 32) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(t_o + q, r);
                        tmem_wait_ld();
                        reg_fence(r);
#pragma unroll
                        for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st_32x32b_x32(t_o + q, r);
                    }
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
                steps++;
            }
            if (!ok) break;
            // ---------------------------------------------------------------- end of the segment
            if (!(ok = wait(&o_full[x], segs & 1))) break;
            tc_fence_after_sync();
            const int r0 = g->rb * R + x * 128;
            const int rr = r0 + min(row, rows - 1);
            const int i_tok = div_group(p, rr);
            const int64_t t = g->first + i_tok;
            const int hq = g->h * p.group + rr - i_tok * p.group;
            const int64_t at = t * p.Hq + hq;
            const bool begins = g->begins, whole = g->whole;
            const int slot = (2 * static_cast<int>(blockIdx.x) + (begins ? 1 : 0)) * R + x * 128 + row;
            const int parts = g->parts;
            const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
            const bool write = row < rows;
            const bool final = whole && p.acc == nullptr;
            // Rows leave through a small buffer of the warp, 64 bytes of each at a time, so that a store writes
            // whole sectors of eight rows (a thread per row writes 32 half sectors: 7900 cycles for 256 rows).
            uint8_t* own = nullptr;
            if (write)
                own = final   ? reinterpret_cast<uint8_t*>(p.o + t * p.o_token + hq * p.o_head)
                      : whole ? reinterpret_cast<uint8_t*>(p.acc + at * D)
                              : reinterpret_cast<uint8_t*>(p.part_o + static_cast<int64_t>(slot) * D);
            uint8_t* dst[4];  // this lane's 16 bytes of rows lane / 4 + 8 i
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint64_t d = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(own), lane / 4 + 8 * i);
                dst[i] = d ? reinterpret_cast<uint8_t*>(d) + lane % 4 * 16 : nullptr;
            }
            auto pass_on = [&](int offset) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + (lane / 4 + 8 * i) * C::kStageRow + lane % 4 * 16);
                    if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + offset) = v;
                }
                __syncwarp();
            };
            uint4* in = reinterpret_cast<uint4*>(stage + lane * C::kStageRow);
#pragma unroll 1
            for (int q = 0; q < D; q += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(t_o + q, o);
                tmem_wait_ld();
                reg_fence(o);
                if (final) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        in[i / 8] = make_uint4(pack_bf16x2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv),
                                               pack_bf16x2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv),
                                               pack_bf16x2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv),
                                               pack_bf16x2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv));
                    pass_on(q * 2);
                } else {
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            in[i] = make_uint4(o[h + 4 * i], o[h + 4 * i + 1], o[h + 4 * i + 2], o[h + 4 * i + 3]);
                        pass_on((q + h) * 4);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[x]);  // O_X may now be overwritten
            segs++;
            if (write) {
                if (whole && p.acc == nullptr)
                    p.lse[at] = lse_of(m_ref, log2f(l_sum), l_sum);
                else
                    (whole ? p.acc_ml[at] : p.part_ml[slot]) = make_float2(m_ref, l_sum);
                if (begins && p.info != nullptr)
                    p.info[at] = whole ? RowInfo{0, 0, 0, 0}
                                       : RowInfo{p.part_row0 + slot, p.part_row0 + slot + R, parts, 2 * R};
                if (begins && !whole && p.tails != nullptr)
                    p.tails[blockIdx.x * R + x * 128 + row] = TailRow{static_cast<int32_t>(at), parts};
            }
            pos += 2 * n;
            close_segment(k_seg);
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace sa
