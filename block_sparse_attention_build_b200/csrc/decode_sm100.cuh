// Attention of few rows (single tokens, a handful of tokens, small groups of
// heads) over a paged cache.
//
// Each key and value is read once for at most 32 rows: 4 bytes of cache carry 4 R
// operations, far below what the tensor cores need to be the limit, so the kernel
// is bound by memory and everything serves to keep loads in flight.  Four warps
// of a CTA work without a barrier between them: each has its own ring of stages
// (8 KB: TK keys and values), loads its own tiles with one TMA per page, S = Q K^T
// and O += P V on mma.sync with R = 16 MT rows, and its own running maximum and
// sum; the warps meet only where an item ends.  A warp's loads run ahead over the
// borders of items.  Two CTAs of an SM hold 8 warps x 3 stages x 8 KB = 192 KB in
// flight (two stages for MT = 2), four times what HBM's latency asks for.
//
// mma.sync, not tcgen05: 16 rows fill its tile, and its operands come straight
// from registers; a 128-row tcgen05 tile would be 7/8 padding and would pay the
// trip through tensor memory for every tile of 16 keys.
#pragma once

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
    static constexpr int kOffMl = kOffMerge + 2 * R * D * 4;  // two warps' O
    static constexpr int kOffScan = kOffMl + 2 * kWarps * R * 4;
    static constexpr int kOffBar = kOffScan + 16 * 8;
    static constexpr int kSmem = kOffBar + kWarps * kStages * 8;
    static constexpr int kSmemBytes = kSmem;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int D, int MT>
__global__ void __launch_bounds__(128, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ PassParams p)
{
    using C = DecodeCfg<D, MT>;
    constexpr int R = C::R, TK = C::TK, UK = C::UK, ST = C::kStages, NW = C::kWarps;
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles sit on 1024 bytes
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint8_t* ring = smem + warp * ST * 2 * C::kTileBytes;
    float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
    float* sm_m = reinterpret_cast<float*>(smem + C::kOffMl);  // [NW][R]
    float* sm_l = sm_m + NW * R;
    int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kOffScan);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * ST;

    if (lane == 0) {
        for (int s = 0; s < ST; s++) mbar_init(&bar[s], 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncwarp();
    launch_dependents();
    const Piece piece = find_piece<R, UK, C::kThreads>(p, 1, scan);
    const int n = static_cast<int>(piece.u1 - piece.u0);
    if (n <= 0) {
        wait_previous_kernel();
        return;
    }
    const int n_seq = p.over_prefix ? 1 : p.B;

    // ---- loads: this warp's tile of every unit of the piece, ST units ahead
    const int page_rows = min(1 << p.page_shift, TK);  // rows of one box
    const int boxes = TK / page_rows;
    Cursor pc = piece.c;
    int issued = 0;
    bool dead = false;
    auto issue = [&]() {
        const int st = issued % ST;
        uint8_t* k_dst = ring + st * 2 * C::kTileBytes;
        const int k0 = pc.u.key(pc.i, UK) + warp * TK;
        // boxes that begin below the item's last key; a tile with none completes its phase at once
        const int nb = min(max((pc.u.hi - k0 + page_rows - 1) / page_rows, 0), boxes);
        const bool skip = (p.debug_flags & 1) && blockIdx.x == 0 && warp == 0 && issued == 0;
        if (lane == 0) mbar_arrive_expect_tx(&bar[st], skip ? 16 : nb * page_rows * D * 4);
        __syncwarp();
        if (lane < nb && !skip) {
            const int k = k0 + lane * page_rows;
            const int pg = page_of(p, pc, k);
            const int row = k & ((1 << p.page_shift) - 1);
            tma_load_5d(k_dst + lane * page_rows * 128, &tmK, &bar[st], 0, row, 0, pc.h, pg);
            tma_load_5d(k_dst + C::kTileBytes + lane * page_rows * 128, &tmV, &bar[st], 0, row, 0, pc.h, pg);
        }
        issued++;
        if (++pc.i >= pc.u.nt) next_item<R, UK>(p, piece.pb, pc, n_seq);
    };
    for (int j = 0; j < ST && j < n; j++) issue();

    // ---- the piece's units
    Cursor c = piece.c;
    const int rq = lane / 4, cq = (lane % 4) * 2;  // this lane's row (and row + 8) and column pair in an mma tile
    uint32_t qf[MT][D / 16][4];
    float o[MT][D / 8][4];
    float m_ref[MT][2], l_sum[MT][2];
    int pos[MT][2];           // positions of this lane's rows
    int p_lo = 0, p_hi = 0;   // the item's lowest and highest
    int rows_left = 0;
    const int off = p.over_prefix ? 0 : p.prefix_len;
    bool fresh = true;
    for (int j = 0; j < n; j++) {
        if (fresh) {
            // Q fragments of the item's rows, straight from memory
            const int r0 = c.rb * R;
            rows_left = min(c.s.m * p.group - r0, R);
            const int base = p.prefix_len + c.s.p0;
            p_lo = p.over_prefix ? piece.pb.lo : base + r0 / p.group;
            p_hi = p.over_prefix ? piece.pb.hi : base + (r0 + rows_left - 1) / p.group;
            // over the prefix the rows' own positions matter unless every row sees every key
            const bool look_up = p.over_prefix && !(p_lo >= p.prefix_len - 1 && p.window >= 0 && p_hi <= p.window);
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int r = mt * 16 + rq + 8 * x;
                    const int rr = r0 + min(r, rows_left - 1);
                    const int i = rr / p.group, g = rr % p.group;
                    pos[mt][x] = look_up ? token_position(p, c.s.first + i) : p.over_prefix ? p_lo : base + i;
                    const __nv_bfloat16* src = p.q + (c.s.first + i) * p.q_token + (c.h * p.group + g) * p.q_head + cq;
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++)
#pragma unroll
                        for (int y = 0; y < 2; y++)
                            qf[mt][kk][x + 2 * y] =
                                r < rows_left ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + y * 8)) : 0u;
                    m_ref[mt][x] = -INFINITY;
                    l_sum[mt][x] = 0.f;
                }
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int i = 0; i < D / 8; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) o[mt][i][e] = 0.f;
            fresh = false;
        }
        const int st = j % ST;
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar[st], (j / ST) & 1, p.timeout))) {
            dead = true;
            if (lane == 0) atomicOr(p.status, ST_PAGED_WAIT);
        }
        const int k0 = c.u.key(c.i, UK) + warp * TK;
        if (!dead && k0 < c.u.hi) {
            const uint32_t ks = smem_addr(ring + st * 2 * C::kTileBytes);
            const uint32_t vs = ks + C::kTileBytes;
            // positions of the tile's first and last key; is every key seen by every row?
            const int a = k0 + off, z = a + TK - 1;
            const bool full = k0 + TK <= c.u.hi && z <= p_lo &&
                              ((p.window >= 0 && p_hi - a <= p.window) || z < p.cols || p_hi < p.n_global);
            if (!full) {
                // values no row sees may be anything, and 0 x infinity is not 0: clear them
                const bool mine = lane < TK;
                const int kp = a + lane;
                const bool seen = k0 + lane < c.u.hi && kp <= p_hi &&
                                  (kp < p.cols || p_lo < p.n_global || (p.window >= 0 && p_lo - kp <= p.window));
                if (mine && !seen) {
                    uint8_t* v = ring + st * 2 * C::kTileBytes + C::kTileBytes + lane * 128;
#pragma unroll
                    for (int pn = 0; pn < D / 64; pn++)
#pragma unroll
                        for (int x = 0; x < 8; x++)
                            *reinterpret_cast<uint4*>(v + pn * C::kPanel + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();  // before the copy that refills the stage
                __syncwarp();
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
            for (int kk = 0; kk < D / 32; kk++)
#pragma unroll
                for (int nb = 0; nb < TK / 8; nb++) {
                    const int row = nb * 8 + lane % 8;
                    const int ch = (kk * 4 + lane / 8) % 8;  // 16-byte chunk within the panel
                    uint32_t b[4];
                    ldsm_x4(ks + (kk * 32 / 64) * C::kPanel + row * 128 + ((ch ^ (row & 7)) * 16), b);
#pragma unroll
                    for (int mt = 0; mt < MT; mt++) {
                        mma_16816(s[mt][nb], qf[mt][2 * kk], b[0], b[1]);
                        mma_16816(s[mt][nb], qf[mt][2 * kk + 1], b[2], b[3]);
                    }
                }
            if (!full) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int nb = 0; nb < TK / 8; nb++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int kk = nb * 8 + cq + (e & 1);
                            const int kp = a + kk, pr = pos[mt][e >> 1];
                            const bool seen = k0 + kk < c.u.hi && kp <= pr &&
                                              (kp < p.cols || pr < p.n_global || (p.window >= 0 && pr - kp <= p.window));
                            if (!seen) s[mt][nb][e] = -INFINITY;
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
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
                    mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * p.scale_log2;
                }
                // the reference follows the maximum only when it grows by 2^8 (as it may: O and the
                // sum carry the same reference), so O is rarely rescaled
                const bool grow = mx[0] > m_ref[mt][0] + 8.f || mx[1] > m_ref[mt][1] + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    float al[2];
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const float mn = fmaxf(m_ref[mt][x], mx[x]);
                        al[x] = mn == -INFINITY ? 1.f : ex2_approx(m_ref[mt][x] - mn);
                        m_ref[mt][x] = mn;
                        l_sum[mt][x] *= al[x];
                    }
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
                    for (int mt = 0; mt < MT; mt++) {
                        mma_16816(o[mt][2 * d], pf[mt][kb], b[0], b[1]);
                        mma_16816(o[mt][2 * d + 1], pf[mt][kb], b[2], b[3]);
                    }
                }
        }
        __syncwarp();  // the stage is read: refill it
        if (issued < n && !dead) issue();

        const bool item_end = c.i + 1 >= c.u.nt;
        if (item_end || j + 1 == n) {
            // ---- join the warps: common maximum, then the O's over two rounds
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
            __syncthreads();
            float M[MT][2], L[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int r = mt * 16 + rq + 8 * x;
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < NW; w++) mm = fmaxf(mm, sm_m[w * R + r]);
                    float ll = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; w++) {
                        const float mw = sm_m[w * R + r];
                        if (mw != -INFINITY) ll += sm_l[w * R + r] * ex2_approx(mw - mm);
                    }
                    M[mt][x] = mm;
                    L[mt][x] = ll;
                    const float f = m_ref[mt][x] == -INFINITY ? 0.f : ex2_approx(m_ref[mt][x] - mm);
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        o[mt][i][2 * x] *= f;
                        o[mt][i][2 * x + 1] *= f;
                    }
                }
            auto put = [&](float* dst) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int i = 0; i < D / 8; i++)
                        *reinterpret_cast<float4*>(dst + ((mt * (D / 8) + i) * 32 + lane) * 4) =
                            make_float4(o[mt][i][0], o[mt][i][1], o[mt][i][2], o[mt][i][3]);
            };
            auto add = [&](const float* src) {
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        const float4 v =
                            *reinterpret_cast<const float4*>(src + ((mt * (D / 8) + i) * 32 + lane) * 4);
                        o[mt][i][0] += v.x;
                        o[mt][i][1] += v.y;
                        o[mt][i][2] += v.z;
                        o[mt][i][3] += v.w;
                    }
            };
            if (warp >= 2) put(merge + (warp - 2) * R * D);
            __syncthreads();
            if (warp < 2) add(merge + warp * R * D);
            if (warp == 1) put(merge + R * D);
            __syncthreads();
            if (warp == 0) {
                add(merge + R * D);
                // the item's units are [u_item, u_item + nt); is it all in this piece?
                const int64_t u_now = piece.u0 + j;
                const int64_t u_item = u_now - c.i;
                const int c_first = cta_of(piece, u_item), c_last = cta_of(piece, u_item + c.u.nt - 1);
                const bool whole = c_first == c_last;
                const bool begins = c_first == static_cast<int>(blockIdx.x);
                const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0)) * R;
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int r = mt * 16 + rq + 8 * x;
                        if (r >= rows_left) continue;
                        const int rr = c.rb * R + r;
                        const int64_t t = c.s.first + rr / p.group;
                        const int hq = c.h * p.group + rr % p.group;
                        const int64_t at = t * p.Hq + hq;
                        if (begins && lane % 4 == 0) {
                            RowInfo ri{0, 0, 0, 0};
                            if (!whole)
                                ri = RowInfo{p.part_row0 + static_cast<int32_t>(slot) + r,
                                             p.part_row0 + (2 * c_first + 2) * R + r, c_last - c_first + 1, 2 * R};
                            p.info[at] = ri;
                        }
                        if (whole && p.acc == nullptr) {
                            const float inv = L[mt][x] > 0.f ? 1.f / L[mt][x] : 0.f;
                            __nv_bfloat16* dst = p.o + t * p.o_token + hq * p.o_head + cq;
#pragma unroll
                            for (int i = 0; i < D / 8; i++)
                                *reinterpret_cast<uint32_t*>(dst + i * 8) =
                                    pack_bf16x2(o[mt][i][2 * x] * inv, o[mt][i][2 * x + 1] * inv);
                            if (lane % 4 == 0)
                                p.lse[at] = L[mt][x] > 0.f ? (M[mt][x] + log2f(L[mt][x])) * 0.69314718055994530942f
                                                           : -INFINITY;
                        } else {
                            float* dst = (whole ? p.acc + at * D : p.part_o + (slot + r) * D) + cq;
#pragma unroll
                            for (int i = 0; i < D / 8; i++)
                                *reinterpret_cast<float2*>(dst + i * 8) =
                                    make_float2(o[mt][i][2 * x], o[mt][i][2 * x + 1]);
                            if (lane % 4 == 0)
                                (whole ? p.acc_ml[at] : p.part_ml[slot + r]) = make_float2(M[mt][x], L[mt][x]);
                        }
                    }
            }
            // the merge buffers are written again only after the next item's first barrier
            fresh = true;
        }
        if (item_end) {
            if (j + 1 < n) next_item<R, UK>(p, piece.pb, c, n_seq);
        } else {
            c.i++;
        }
    }
    if (dead) {
        // copies still in flight land before the CTA's memory goes away
        for (int j = max(issued - ST, 0); j < issued; j++) mbar_wait(&bar[j % ST], (j / ST) & 1, p.timeout);
    }
    wait_previous_kernel();
}

}  // namespace sa
