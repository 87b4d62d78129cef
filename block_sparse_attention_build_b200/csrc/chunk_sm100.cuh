// Attention of many rows (pieces of prompts, whole prompts, all sequences of a
// batch over their shared prefix) over a paged cache, on the tensor cores.
//
// An item is 256 rows: two slots of 128 (a tensor-memory lane per row) that read
// the same keys, so that a key tile serves 2 x 128 rows and the tensor cores work
// on one slot while the other slot's softmax runs.  At 256 rows a unit of 128 keys
// is 4 * 256 * 128 * D operations on 512 D bytes: the tensor cores and the
// exponentials bound it, not memory.
//
// Warp roles (384 threads, three warpgroups):
//   warp 0     producer: K and V tiles of the CTA's units through one ring of
//              stages, a page (or 128 places of one) per TMA, its lanes side by side
//   warp 1     allocates tensor memory; one lane issues every tcgen05.mma
//   warps 2, 3 Q of slot A, slot B: rows lie where tokens and heads put them, so
//              they are gathered with cp.async into the swizzled layout that TMA
//              would write, while the previous item's last softmax and PV still run
//   warps 4-7  softmax of slot A, warps 8-11 of slot B: a thread per row
//
// Order of the tensor cores: PV_A(j), S_A(j+1), PV_B(j), S_B(j+1).  Tensor memory
// (512 columns): S_A, S_B (128 each; P over their first half), O_A, O_B (D each).
// Places no row sees may hold anything: scores there are replaced, and slot A's
// threads clear the tile's V rows before P V (0 x infinity is not 0).
//
// Every wait is bounded; on expiry the status word is set, all roles leave their
// loops, copies and MMAs in flight are waited for and tensor memory is freed.
#pragma once

#include "fwd_sm100.cuh"
#include "paged_sm100.cuh"

namespace sa {

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
    static constexpr int kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * 6 + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmemUsed = kOffMisc + 16;
    // at least this much, so that one CTA owns the SM's tensor memory
    static constexpr int kSmemBytes = kSmemUsed > 120 * 1024 ? kSmemUsed : 120 * 1024;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(2 * UK + 2 * D <= 512, "tensor memory budget");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
    uint64_t* ring_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [S]
    uint64_t* ring_empty = ring_full + S;                                  // [S]
    uint64_t* q_full = ring_empty + S;   // [2]
    uint64_t* q_empty = q_full + 2;      // [2] the slot's last S MMA of the item is done
    uint64_t* s_full = q_empty + 2;      // [2]
    uint64_t* p_full = s_full + 2;       // [2]
    uint64_t* o_full = p_full + 2;       // [2]
    uint64_t* o_empty = o_full + 2;      // [2]
    uint64_t* drain = o_empty + 2;       // [1]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; i++) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 1);
        }
        for (int x = 0; x < 2; x++) {
            mbar_init(&q_full[x], 32);
            mbar_init(&q_empty[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 128);
            mbar_init(&o_full[x], 1);
            mbar_init(&o_empty[x], 128);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    launch_dependents();
    const Piece piece = find_piece<R, UK, false>(p, peek_seq(p), blockIdx.x, gridDim.x);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const long long lim = p.timeout;
    const int n_seq = p.over_prefix ? 1 : p.B;
    const int total = piece.u1 - piece.u0;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, ST_PAGED_WAIT);
    };
    // The CTA's segments: for each, the item and the units [c.i, c.i + n) of it.
    Cursor c = piece.c;
    int left = total;
    auto seg_len = [&]() { return min(c.u.nt - c.i, left); };
    auto seg_next = [&](int n) {
        left -= n;
        if (left > 0) next_item<R, UK>(p, piece.pb, c, n_seq);
    };
    auto rows_of_item = [&]() { return min(c.s.m * p.group - c.rb * R, R); };
    // warp-uniform warpgroup index, so that the register split applies per branch
    const int wg = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 128, 0);

    if (wg == 0) {
        regs_dec<kRegsControl>();
        if (warp == 0) {
            // ============================================================ producer
            const int page_rows = min(1 << p.page_shift, UK);
            constexpr int P = D / 64;  // column panels
            int pos = 0;
            bool dead = false;
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim));
            };
            while (left > 0 && !dead) {
                const int n = seg_len();
                for (int j = 0; j < n && !dead; j++) {
                    const int k0 = c.u.key(c.i + j, UK);
                    // boxes that begin below the item's last key, a panel each
                    const int nb = min(max((c.u.hi - k0 + page_rows - 1) / page_rows, 0), UK / page_rows);
                    const int box = lane / P, panel = lane % P;
                    const bool mine = box < nb;
                    const int k = k0 + box * page_rows;
                    const int pg = mine ? page_of(p, c.b, k) : 0;
                    const int row = k & ((1 << p.page_shift) - 1);
#pragma unroll
                    for (int v = 0; v < 2; v++) {  // K, then V
                        if (!wait(&ring_empty[pos % S], ((pos / S) & 1) ^ 1)) {
                            if (lane == 0) fail();
                            dead = true;
                            break;
                        }
                        const int st = pos % S;
                        const bool skip = (p.debug_flags & 1) && blockIdx.x == 0 && pos == 0;
                        if (lane == 0) mbar_arrive_expect_tx(&ring_full[st], skip ? 16 : nb * page_rows * D * 2);
                        __syncwarp();
                        if (mine && !skip)
                            tma_load_5d(ring + st * C::kTileBytes + panel * C::kPanel + box * page_rows * 128,
                                        v == 0 ? &tmK : &tmV, &ring_full[st], 0, row, panel, c.h, pg);
                        __syncwarp();
                        pos++;
                    }
                    if (__any_sync(0xffffffffu, *abort_flag != 0)) dead = true;
                }
                seg_next(n);
            }
            if (__any_sync(0xffffffffu, *abort_flag != 0)) {
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
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim));
            };
            int steps[2] = {0, 0};  // S/P handshakes per slot
            int segs[2] = {0, 0};   // segments per slot (phases of q_full, o_full, o_empty)
            int pos = 0;
            bool ok = true;
            while (left > 0 && ok) {
                const int n = seg_len();
                const int nx = rows_of_item() > 128 ? 2 : 1;
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
                            if (x == 0 && !wait(&ring_full[pk % S], (pk / S) & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after_sync();
                            issue_s(x, pk % S);
                            commit(&s_full[x]);
                            if (j + 2 == n) commit(&q_empty[x]);  // the slot's last read of Q
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                    if (!ok) break;
                    commit(&ring_empty[pv % S]);
                    if (!last) commit(&ring_empty[pk % S]);
                }
#pragma unroll
                for (int x = 0; x < 2; x++)
                    if (x < nx) segs[x]++;
                pos += 2 * n;
                seg_next(n);
            }
            if (!ok && lane == 0) fail();
            // all issued tensor-core work is finished before the memory is released
            commit(drain);
            if (!wait(drain, 0) && lane == 0) atomicOr(p.status, ST_DRAIN_WAIT);
        } else {
            // ============================================================ Q of slot x
            const int x = warp - 2;
            constexpr int L = D / 8;        // lanes of a row, 16 bytes each
            constexpr int RW = 32 / L;      // rows of one step
            const uint32_t dst0 = smem_addr(sQ) + x * C::kQBytes;
            int loads = 0;
            bool ok = true;
            while (left > 0 && ok) {
                const int n = seg_len();
                const int rows = rows_of_item() - x * 128;
                if (rows > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[x], (loads & 1) ^ 1, lim) && !*abort_flag);
                    if (!ok) break;
                    const int ch = lane % L;
                    for (int r = lane / L; r < 128; r += RW) {
                        // rows behind the item's last repeat it: what they compute is not written
                        const int rr = c.rb * R + x * 128 + min(r, rows - 1);
                        const int i = div_group(p, rr), g = rr - i * p.group;
                        cp_async_16(dst0 + (ch / 8) * C::kPanel + r * 128 + (((ch % 8) ^ (r & 7)) * 16),
                                    p.q + (c.s.first + i) * p.q_token + (c.h * p.group + g) * p.q_head + ch * 8);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    mbar_arrive(&q_full[x]);
                    loads++;
                }
                seg_next(n);
            }
            if (!ok && lane == 0) fail();
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ================================================================ softmax
        const int x = wg - 1;            // slot
        const int quarter = warp & 3;    // tensor-memory lanes this warp may access
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32);
        const uint32_t col_s = static_cast<uint32_t>(x * UK);
        const uint32_t col_o = static_cast<uint32_t>(2 * UK + x * D);
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
        const int off = p.over_prefix ? 0 : p.prefix_len;
        int steps = 0, segs = 0;
        int pos = 0;  // ring items of the segments before
        bool ok = true;
        while (left > 0 && ok) {
            const int n = seg_len();
            const int rows = rows_of_item() - x * 128;  // of this slot
            if (rows <= 0) {
                pos += 2 * n;
                seg_next(n);
                continue;
            }
            const int r0 = c.rb * R + x * 128;
            const int rr = r0 + min(row, rows - 1);
            const int i_tok = div_group(p, rr);
            const int base = p.prefix_len + c.s.p0;
            // the slot's lowest and highest position, this row's, and the item's (whose keys are loaded)
            const int p_lo = p.over_prefix ? piece.pb.lo : base + div_group(p, r0);
            const int p_hi = p.over_prefix ? piece.pb.hi : base + div_group(p, r0 + min(rows, 128) - 1);
            const int item_hi = p.over_prefix ? piece.pb.hi : base + div_group(p, c.rb * R + rows_of_item() - 1);
            const bool look_up = p.over_prefix && !(p_lo >= p.prefix_len - 1 && p.window >= 0 && p_hi <= p.window);
            const int pr = look_up ? token_position(p, c.s.first + i_tok) : p.over_prefix ? p_lo : base + i_tok;
            const bool row_all = pr < p.n_global;
            float m_ref = -INFINITY;  // running max, log2 units of the scaled score
            float l_sum = 0.f;
            for (int j = 0; j < n; j++) {
                const int kv0 = c.u.key(c.i + j, UK);
                const int a = kv0 + off, z = a + UK - 1;  // positions of the tile's first and last key
                const bool masked = !(kv0 + UK <= c.u.hi && z <= p_lo &&
                                      ((p.window >= 0 && p_hi - a <= p.window) || z < p.cols || p_hi < p.n_global));
                uint32_t allow[UK / 32];
                if (masked) {
                    const int dq = pr - a;
                    const int c_max = min(dq, c.u.hi - 1 - kv0);
#pragma unroll
                    for (int w = 0; w < UK / 32; w++) {
                        const int b = 32 * w;
                        uint32_t m = bits_between(0, p.cols - 1 - a - b);
                        if (p.window >= 0) m |= bits_between(dq - p.window - b, 31);
                        if (row_all) m = 0xffffffffu;
                        allow[w] = m & bits_between(0, c_max - b);
                    }
                    if (x == 0) {
                        // this thread's V row of the tile, where no row of the item sees it
                        const int kp = a + row;
                        const bool seen = kv0 + row < c.u.hi && kp <= item_hi &&
                                          (kp < p.cols || p_lo < p.n_global || (p.window >= 0 && p_lo - kp <= p.window));
                        if (__any_sync(0xffffffffu, !seen)) {
                            const int pv = pos + 2 * j + 1;
                            ok = mbar_wait(&ring_full[pv % S], (pv / S) & 1, lim);
                            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                            if (!ok) break;
                            if (!seen) {
                                uint8_t* v = ring + (pv % S) * C::kTileBytes + row * 128;
#pragma unroll
                                for (int pn = 0; pn < D / 64; pn++)
#pragma unroll
                                    for (int q = 0; q < 8; q++)
                                        *reinterpret_cast<uint4*>(v + pn * C::kPanel + q * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                        }
                    }
                }

                ok = mbar_wait(&s_full[x], steps & 1, lim);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
                tc_fence_after_sync();

                float s[UK];
                {
                    uint32_t r[UK / 32][32];
#pragma unroll
                    for (int q = 0; q < UK / 32; q++)
                        tmem_ld_32x32b_x32(tmem_addr(tmem, lane_base, col_s + 32 * q), r[q]);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < UK / 32; q++) reg_fence(r[q]);
#pragma unroll
                    for (int q = 0; q < UK; q++) s[q] = __uint_as_float(r[q / 32][q % 32]);
                }
                if (masked) {
#pragma unroll
                    for (int q = 0; q < UK; q++) s[q] = (allow[q / 32] >> (q % 32)) & 1u ? s[q] : -INFINITY;
                }
                // row max: 16 independent chains of three-input max
                float mx[16];
#pragma unroll
                for (int i = 0; i < 16; i++) mx[i] = fmax3(s[i], s[16 + i], s[32 + i]);
#pragma unroll
                for (int q = 48; q + 32 <= UK; q += 32)
#pragma unroll
                    for (int i = 0; i < 16; i++) mx[i] = fmax3(mx[i], s[q + i], s[q + 16 + i]);
#pragma unroll
                for (int i = 0; i < 16; i++) mx[i] = fmaxf(mx[i], s[UK - 16 + i]);
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
                // p = 2^(s * scale_log2 - m): 6 of every 8 pairs on the MUFU unit, 2 on the FMA pipe
                uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < UK; q += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const uint64_t x2 = f2_fma(f2_pack(s[q + 2 * i], s[q + 2 * i + 1]), scale2, neg_m);
                        float e0, e1;
                        if (((q / 2 + i) & 7) < 2) {
                            exp2_poly_x2(x2, e0, e1);
                        } else {
                            float x0, x1;
                            f2_unpack(x2, x0, x1);
                            e0 = ex2_approx(x0);
                            e1 = ex2_approx(x1);
                        }
                        acc[i & 3] = f2_add(acc[i & 3], f2_pack(e0, e1));
                        pk[i] = pack_bf16x2(e0, e1);
                    }
                    tmem_st_32x32b_x32(tmem_addr(tmem, lane_base, col_s + q / 2), pk);
                }
                {
                    float a0, a1, b0, b1, c0, c1, d0, d1;
                    f2_unpack(acc[0], a0, a1);
                    f2_unpack(acc[1], b0, b1);
                    f2_unpack(acc[2], c0, c1);
                    f2_unpack(acc[3], d0, d1);
                    l_sum += ((a0 + a1) + (b0 + b1)) + ((c0 + c1) + (d0 + d1));
                }
                if (j > 0 && __any_sync(0xffffffffu, grow)) {
                    // O_X holds every product up to tile j-1 (the commit of S_X(j) covers PV_X(j-1))
#pragma unroll
                    for (int q = 0; q < D; q += 32) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(tmem_addr(tmem, lane_base, col_o + q), r);
                        tmem_wait_ld();
                        reg_fence(r);
#pragma unroll
                        for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st_32x32b_x32(tmem_addr(tmem, lane_base, col_o + q), r);
                    }
                }
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(&p_full[x]);
                steps++;
            }
            if (!ok) break;
            // ---------------------------------------------------------------- end of the segment
            ok = mbar_wait(&o_full[x], segs & 1, lim);
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            uint32_t o[D / 32][32];
            tc_fence_after_sync();
#pragma unroll
            for (int q = 0; q < D / 32; q++) tmem_ld_32x32b_x32(tmem_addr(tmem, lane_base, col_o + 32 * q), o[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < D / 32; q++) reg_fence(o[q]);
            tc_fence_before_sync();
            mbar_arrive(&o_empty[x]);
            segs++;
            if (row < rows) {
                const int u_item = piece.u0 + (total - left) - c.i;
                const bool begins = u_item >= piece.u0, whole = begins && u_item + c.u.nt <= piece.u1;
                const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0)) * R + x * 128 + row;
                const int64_t t = c.s.first + i_tok;
                const int hq = c.h * p.group + rr - i_tok * p.group;
                const int64_t at = t * p.Hq + hq;
                if (begins) {
                    RowInfo ri{0, 0, 0, 0};
                    if (!whole) {
                        const int n_parts = cta_of(piece, u_item + c.u.nt - 1) - static_cast<int>(blockIdx.x) + 1;
                        ri = RowInfo{p.part_row0 + static_cast<int32_t>(slot), p.part_row0 + static_cast<int32_t>(slot) + R,
                                     n_parts, 2 * R};
                    }
                    p.info[at] = ri;
                }
                if (whole && p.acc == nullptr) {
                    const float inv = l_sum > 0.f ? 1.f / l_sum : 0.f;
                    uint4* dst = reinterpret_cast<uint4*>(p.o + t * p.o_token + hq * p.o_head);
#pragma unroll
                    for (int q = 0; q < D; q += 8) {
                        const uint32_t* oc = &o[q / 32][q % 32];
                        uint4 v;
                        v.x = pack_bf16x2(__uint_as_float(oc[0]) * inv, __uint_as_float(oc[1]) * inv);
                        v.y = pack_bf16x2(__uint_as_float(oc[2]) * inv, __uint_as_float(oc[3]) * inv);
                        v.z = pack_bf16x2(__uint_as_float(oc[4]) * inv, __uint_as_float(oc[5]) * inv);
                        v.w = pack_bf16x2(__uint_as_float(oc[6]) * inv, __uint_as_float(oc[7]) * inv);
                        dst[q / 8] = v;
                    }
                    p.lse[at] = l_sum > 0.f ? (m_ref + log2f(l_sum)) * 0.69314718055994530942f : -INFINITY;
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(whole ? p.acc + at * D : p.part_o + slot * D);
#pragma unroll
                    for (int q = 0; q < D; q += 4) {
                        const uint32_t* oc = &o[q / 32][q % 32];
                        dst[q / 4] = make_uint4(oc[0], oc[1], oc[2], oc[3]);
                    }
                    (whole ? p.acc_ml[at] : p.part_ml[slot]) = make_float2(m_ref, l_sum);
                }
            }
            pos += 2 * n;
            seg_next(n);
        }
        if (!ok) fail();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    wait_previous_kernel();
}

}  // namespace sa
