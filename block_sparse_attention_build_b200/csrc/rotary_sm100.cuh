// Rotation of queries and keys by their positions, and the append of a batch's
// new keys and values to a paged cache with the rotation applied on the way.
//
// Pair j of a row turns by the angle pos[axis_j] * freq_j: (a, b) -> (a cos - b
// sin, b cos + a sin).  Every element is read and written once, so the kernel is
// bound by memory; what it has to keep small besides is the trigonometry.  The
// angles depend on the token alone, so one thread owns the same few pairs of one
// token in every head of its share: it takes their sines and cosines once, keeps
// them in registers and walks the heads with nothing but wide loads, the
// rotation and wide stores.  No shared memory, no barrier.
//
// The angle counts in turns, as a 64-bit fraction: position times fraction wraps
// around at a whole turn by itself and is exact (a 32-bit product would be off by
// 0.03 radians at position 10^6), and its upper 32 bits go to sincospif.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_sm100.cuh"

namespace sa {

constexpr int kMaxPairs = 64;  // D / 2
constexpr int kMaxAxes = 4;

struct RotSpec {
    uint64_t turns[kMaxPairs];  // turns per position, modulo 1: a fraction of 64 bits
    uint8_t axis[kMaxPairs];
    int32_t n_pairs;
};

struct RotView {
    __nv_bfloat16* p;
    int64_t batch, head, token;
};

struct RotParams {
    RotView q, k, v;    // inputs; v only with a cache
    RotView qo, ko;     // outputs; with a cache ko, vo are its pages (batch = page stride)
    __nv_bfloat16* vo;
    int32_t Hq, Hk, Hv; // heads rotated to qo, rotated to ko, copied to vo
    int32_t heads_per;  // heads of one thread
    int64_t rows;       // tokens: B * N, or T
    int32_t N;          // tokens of a sequence (whole sequences)
    const int32_t* pos; // null: the place in the cache + pos_offset
    int64_t pos_axis, pos_batch;
    float sign;         // -1: backward
    // cache
    int32_t B, n_pages, page_shift, max_pages, pos_offset;
    int64_t table_stride;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x c + y s of a word's two elements, rounded once to bf16.
__device__ __forceinline__ uint32_t turn_word(uint32_t x, uint32_t y, float c0, float c1, float s0, float s1)
{
    return pack_bf16x2(bf_lo(x) * c0 + bf_lo(y) * s0, bf_hi(x) * c1 + bf_hi(y) * s1);
}

// How a thread holds its part of a row:
//   kHalves      (j, j + n_pairs), n_pairs a multiple of 8: two chunks of 16 bytes, n_pairs apart,
//                of 8 pairs
//   kInterleaved (2j, 2j + 1): two neighbouring chunks of 4 pairs each
//   kShuffled    (j, j + n_pairs), any n_pairs: one chunk of 8 bytes, whose partners lie in other
//                lanes' chunks at any offset
enum RotLayout { kHalves, kInterleaved, kShuffled };

template <int W>
struct Words {  // one access of W words
    uint32_t w[W];
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x;
            w[1] = x.y;
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const
    {
        if constexpr (W == 4)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};

// Turn a kShuffled chunk: words 2 l, 2 l + 1 of a row that L lanes hold.  `cs`, `sn`
// belong to the chunk's four elements (sn with the sign that the element's place in
// its pair wants): x cos + partner sn.
template <int L>
__device__ __forceinline__ void turn_shuffled(Words<2>& x, int P, int lane, const float (&cs)[8], const float (&sn)[8])
{
    const int base = lane & ~(L - 1), l = lane & (L - 1);
    const int S = P >> 1;
    if ((P & 1) == 0) {
        // The partner of word w is word w + S in the first half, w - S in the second: register (i + S) mod 2
        // of some lane either way, so one shuffle per word serves both halves.
        const bool swap = S & 1;
        const uint32_t r0 = swap ? x.w[1] : x.w[0], r1 = swap ? x.w[0] : x.w[1];
        uint32_t y[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int w = 2 * l + i;
            const int src = w < S ? w + S : w - S;
            y[i] = __shfl_sync(0xffffffffu, i ? r1 : r0, base + ((src >> 1) & (L - 1)));
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t r = turn_word(x.w[i], y[i], cs[2 * i], cs[2 * i + 1], sn[2 * i], sn[2 * i + 1]);
            x.w[i] = 2 * l + i < P ? r : x.w[i];
        }
    } else {
        // partners straddle words: elements e + P begin in the high half of word w + S, e - P in the high half of
        // word w - S - 1
        const uint32_t x0 = x.w[0], x1 = x.w[1];
        auto word = [&](int w) {  // of the row; both registers are offered, the asker picks
            const int src = base + ((w >> 1) & (L - 1));
            const uint32_t a = __shfl_sync(0xffffffffu, x0, src), b = __shfl_sync(0xffffffffu, x1, src);
            return w & 1 ? b : a;
        };
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int w = 2 * l + i, e = 2 * w;
            const uint32_t up = __funnelshift_r(word(w + S), word(w + S + 1), 16);
            const uint32_t dn = __funnelshift_r(word(w - S - 1), word(w - S), 16);
            const uint32_t v = i ? x1 : x0;
            const uint32_t y = __byte_perm(e < P ? up : dn, e + 1 < P ? up : dn, 0x7610);
            const uint32_t r = turn_word(v, y, cs[2 * i], cs[2 * i + 1], sn[2 * i], sn[2 * i + 1]);
            x.w[i] = w < P ? r : v;
        }
    }
}

constexpr int kRotThreads = 128;
// Heads whose loads one thread has in flight, and blocks of an SM (which bound the registers), both
// swept on 16 + 16 heads of 128 at 8192 tokens and 64 + 8 heads of 64 at 2 x 16384: 4 heads of 32 bytes
// with 6 blocks, 8 of 8 bytes with 8.
__host__ __device__ constexpr int rot_unroll(RotLayout l) { return l == kShuffled ? 8 : 4; }
__host__ __device__ constexpr int rot_blocks(RotLayout l) { return l == kShuffled ? 8 : 6; }

template <int D, RotLayout LAYOUT, bool PAGED>
__global__ void __launch_bounds__(kRotThreads, rot_blocks(LAYOUT)) rotary_kernel(const __grid_constant__ RotSpec spec,
                                                             const __grid_constant__ RotParams p)
{
    constexpr int kChunks = LAYOUT == kShuffled ? 1 : 2;    // of one thread
    constexpr int W = LAYOUT == kShuffled ? 2 : 4;          // words of a chunk
    constexpr int kItems = D / (2 * W * kChunks);           // threads of one token
    constexpr int kTok = 32 / kItems;                       // tokens of one warp
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
    const int64_t t = gid / kItems;
    const int item = static_cast<int>(gid % kItems);
    const int lane = threadIdx.x % 32;

    // The pairs' turns and axes, from parameters to shared memory: a warp's lanes index them apart, which
    // constant memory would serve one lane at a time (64 + 8 heads of 64, 30 pairs: 133 us so).
    __shared__ uint64_t sh_turns[kMaxPairs];
    __shared__ uint8_t sh_axis[kMaxPairs];
    for (int i = threadIdx.x; i < spec.n_pairs; i += kRotThreads) {
        sh_turns[i] = spec.turns[i];
        sh_axis[i] = spec.axis[i];
    }
    wait_previous_kernel();
    launch_dependents();
    __syncthreads();
    constexpr int U = rot_unroll(LAYOUT);
    const int h_begin = static_cast<int>(blockIdx.y) * p.heads_per, h_end = h_begin + p.heads_per;
    if constexpr (PAGED) {
        // finding the token's sequence, position and page takes several loads one after another: have the
        // first rows on their way to L2 meanwhile
        if (t < p.rows) {
            const __nv_bfloat16* q = p.q.p + t * p.q.token + item * (D / kItems);
#pragma unroll
            for (int u = 0; u < U; u++)
                if (h_begin + u < p.Hq) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (h_begin + u) * p.q.head));
        }
    }

    // where the token stands, and where its key and value go
    bool have;  // lanes without a token stay: others may shuffle with them
    int64_t b = 0, n = 0;
    int64_t page_off = -1;
    int place = 0;
    if constexpr (PAGED) {
        // the sequence of each of the warp's tokens: how many sequences start at or before it
        const int64_t t0 = (gid - lane) / kItems;
        const int mine = static_cast<int>(t - t0);
        int cnt = 0;
        for (int c = 0; c < p.B; c += 32) {
            const int s = c + lane < p.B ? p.q_start[c + lane] : INT32_MAX;
#pragma unroll
            for (int k = 0; k < kTok; k++) {
                const int m = __popc(__ballot_sync(0xffffffffu, s <= t0 + k));
                if (k == mine) cnt += m;
            }
        }
        have = t < p.rows && cnt > 0 && t < p.q_start[p.B];
        b = max(cnt - 1, 0);
        const int first = p.q_start[b], next = p.q_start[b + 1];
        n = t;
        place = tokens_of(p.kv_len[b]) - (next - first) + static_cast<int>(t - first);
        const int pi = place >> p.page_shift;
        if (have && place >= 0 && pi < p.max_pages) {
            const int page = p.table[b * p.table_stride + pi];
            if (page >= 0 && page < p.n_pages)
                page_off = page * p.ko.batch + (place & ((1 << p.page_shift) - 1)) * p.ko.token;
        }
    } else {
        have = t < p.rows;
        b = t / p.N;
        n = t % p.N;
    }

    // this thread's chunks and the pair of each of its 8 elements or pairs (-1: stays as it is)
    const int P = spec.n_pairs;
    int off_a, off_b = 0, pair0 = 0, n_rot = 0;
    if constexpr (LAYOUT == kInterleaved) {
        off_a = 16 * item;
        off_b = off_a + 8;
        pair0 = 8 * item;
        n_rot = min(max(P - pair0, 0), 8);
    } else if constexpr (LAYOUT == kHalves) {
        const int turning = P / 8;
        if (item < turning) {
            off_a = 8 * item;
            off_b = P + off_a;
            pair0 = off_a;
            n_rot = 8;
        } else {
            off_a = 2 * P + 16 * (item - turning);
            off_b = off_a + 8;
        }
    } else {
        off_a = 4 * item;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        int j = i < n_rot ? pair0 + i : -1;
        float sign = p.sign;
        if constexpr (LAYOUT == kShuffled) {  // an element is x cos + partner sn: minus in the first of a pair
            const int e = off_a + i;
            j = i >= 2 * W ? -1 : e < P ? e : e < 2 * P ? e - P : -1;
            if (e < P) sign = -sign;
        }
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (j >= 0 && have) {
            int pos;
            if (PAGED && p.pos == nullptr)
                pos = place + p.pos_offset;
            else
                pos = p.pos[sh_axis[j] * p.pos_axis + (PAGED ? t : b * p.pos_batch + n)];
            // the angle modulo a turn: the low 64 bits of the product, of which the upper 32 are kept
            const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * sh_turns[j];
            sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
            sn[i] *= sign;
        }
    }
    auto turn_own = [&](Words<W> (&x)[kChunks]) {  // kHalves, kInterleaved
        Words<W>& a = x[0];
        Words<W>& c = x[kChunks - 1];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t wa = a.w[i], wc = c.w[i];
            if constexpr (LAYOUT == kInterleaved) {
                const uint32_t ra = turn_word(wa, __byte_perm(wa, 0, 0x1032), cs[i], cs[i], -sn[i], sn[i]);
                const uint32_t rc = turn_word(wc, __byte_perm(wc, 0, 0x1032), cs[i + 4], cs[i + 4], -sn[i + 4], sn[i + 4]);
                a.w[i] = i < n_rot ? ra : wa;
                c.w[i] = i + 4 < n_rot ? rc : wc;
            } else {
                const int j = 2 * i;
                a.w[i] = turn_word(wa, wc, cs[j], cs[j + 1], -sn[j], -sn[j + 1]);
                c.w[i] = turn_word(wc, wa, cs[j], cs[j + 1], sn[j], sn[j + 1]);
            }
        }
    };

    int first = 0;  // heads before this kind's
#pragma unroll 1
    for (int kind = 0; kind < (PAGED ? 3 : 2); kind++) {  // queries, keys, values (copied)
        const RotView& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
        const RotView& out = kind == 0 ? p.qo : p.ko;
        const int heads = kind == 0 ? p.Hq : kind == 1 ? p.Hk : p.Hv;
        const int h0 = max(h_begin - first, 0), h1 = min(h_end - first, heads);
        first += heads;
        const bool paged = PAGED && kind > 0;
        const bool mine = have && (!paged || page_off >= 0);
        const __nv_bfloat16* src = in.p + (PAGED ? 0 : b * in.batch) + n * in.token + h0 * in.head + off_a;
        __nv_bfloat16* dst = (kind == 2 ? p.vo : out.p) + (paged ? page_off : (PAGED ? 0 : b * out.batch) + n * out.token) +
                             h0 * out.head + off_a;
        const int d_b = off_b - off_a;
        const int64_t s_in = in.head, s_out = out.head;
        auto turn = [&](Words<W> (&x)[kChunks]) {
            if constexpr (LAYOUT == kShuffled)
                turn_shuffled<kItems>(x[0], P, lane, cs, sn);
            else if (n_rot > 0)
                turn_own(x);
        };
        // whole batches of heads, then the rest one by one; lanes without work read nothing and shuffle along
        int h = h0;
        for (; h + U <= h1; h += U) {
            Words<W> x[U][kChunks];
            if (mine) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    x[u][0].load(src);
                    if constexpr (kChunks == 2) x[u][1].load(src + d_b);
                    src += s_in;
                }
            }
            if (kind < 2) {
#pragma unroll
                for (int u = 0; u < U; u++) turn(x[u]);
            }
            if (mine) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    x[u][0].store(dst);
                    if constexpr (kChunks == 2) x[u][1].store(dst + d_b);
                    dst += s_out;
                }
            }
        }
        for (; h < h1; h++) {
            Words<W> x[kChunks];
            if (mine) {
                x[0].load(src);
                if constexpr (kChunks == 2) x[1].load(src + d_b);
            }
            if (kind < 2) turn(x);
            if (mine) {
                x[0].store(dst);
                if constexpr (kChunks == 2) x[1].store(dst + d_b);
            }
            src += s_in;
            dst += s_out;
        }
    }
}

}  // namespace sa
