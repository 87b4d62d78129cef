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
// The angle is a 64-bit product in turns (positions times freq / 2 pi), reduced
// to [-1/2, 1/2] before it is rounded to 32 bits: at position 10^6 a 32-bit
// product would be off by 0.03 radians.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sa {

constexpr int kMaxPairs = 64;  // D / 2
constexpr int kMaxAxes = 4;

struct RotSpec {
    double turns[kMaxPairs];  // freq / 2 pi
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

// One access of V bf16 elements.
template <int V>
struct Chunk;
template <>
struct Chunk<8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    __device__ __forceinline__ void set_word(int i, uint32_t x)
    {
        if (i == 0) w.x = x;
        else if (i == 1) w.y = x;
        else if (i == 2) w.z = x;
        else w.w = x;
    }
};
template <>
struct Chunk<2> {
    uint32_t w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = w; }
    __device__ __forceinline__ uint32_t word(int) const { return w; }
    __device__ __forceinline__ void set_word(int, uint32_t x) { w = x; }
};
template <>
struct Chunk<1> {
    uint32_t w;  // the low half holds the element
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint16_t*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const
    {
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w);
    }
    __device__ __forceinline__ uint32_t word(int) const { return w; }
    __device__ __forceinline__ void set_word(int, uint32_t x) { w = x; }
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Rotate one thread's part of a row in place.  Halves layout: a and b hold the V
// elements x and x + n_pairs of V pairs.  Interleaved (V = 8): a and b are
// neighbouring chunks of four pairs each, and `n` counts the pairs that turn.
template <int V, bool INTER>
__device__ __forceinline__ void rotate_chunks(Chunk<V>& a, Chunk<V>& b, const float (&cs)[8], const float (&sn)[8],
                                              int n)
{
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            Chunk<V>& c = i < 4 ? a : b;
            const uint32_t w = c.word(i & 3);
            const float x = bf_lo(w), y = bf_hi(w);
            const uint32_t r = pack_bf16x2(x * cs[i] - y * sn[i], y * cs[i] + x * sn[i]);
            c.set_word(i & 3, i < n ? r : w);
        }
    } else {
        constexpr int W = V == 8 ? 4 : 1;
#pragma unroll
        for (int i = 0; i < W; i++) {
            const uint32_t wa = a.word(i), wb = b.word(i);
            const float x0 = bf_lo(wa), y0 = bf_lo(wb);
            const int j = 2 * i;
            float a1 = 0.f, b1 = 0.f;
            if constexpr (V > 1) {
                const float x1 = bf_hi(wa), y1 = bf_hi(wb);
                a1 = x1 * cs[j + 1] - y1 * sn[j + 1];
                b1 = y1 * cs[j + 1] + x1 * sn[j + 1];
            }
            a.set_word(i, pack_bf16x2(x0 * cs[j] - y0 * sn[j], a1));
            b.set_word(i, pack_bf16x2(y0 * cs[j] + x0 * sn[j], b1));
        }
    }
}

constexpr int kRotThreads = 128;
constexpr int kRotUnroll = 4;  // heads whose loads one thread has in flight

// V: elements of one access (8 when the halves start on 16 bytes or pairs are
// interleaved, else 2 for an even and 1 for an odd number of pairs); the row of D
// elements is D / (2 V) items of two accesses each.
template <int D, int V, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotSpec spec,
                                                             const __grid_constant__ RotParams p)
{
    constexpr int kItems = D / (2 * V);                     // threads of one token
    constexpr int kTok = kItems >= 32 ? 1 : 32 / kItems;    // tokens of one warp
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
    const int64_t t = gid / kItems;
    const int item = static_cast<int>(gid % kItems);
    const int lane = threadIdx.x % 32;

    // where the token stands, and where its key and value go
    int64_t b = 0, n = 0;
    int64_t page_off = -1;
    int place = 0;
    if constexpr (PAGED) {
        // the sequence of each of the warp's tokens: how many sequences start at or before it
        const int64_t t0 = (gid - lane) / kItems;
        const int mine = static_cast<int>(t - t0);
        int cnt = 0;
        for (int c = 0; c < p.B; c += 32) {
            const int s = c + lane < p.B ? __ldg(&p.q_start[c + lane]) : INT32_MAX;
#pragma unroll
            for (int k = 0; k < kTok; k++) {
                const int m = __popc(__ballot_sync(0xffffffffu, s <= t0 + k));
                if (k == mine) cnt += m;
            }
        }
        if (t >= p.rows || cnt == 0 || t >= __ldg(&p.q_start[p.B])) return;
        b = cnt - 1;
        const int first = __ldg(&p.q_start[b]), next = __ldg(&p.q_start[b + 1]);
        n = t;
        place = __ldg(&p.kv_len[b]) - (next - first) + static_cast<int>(t - first);
        const int pi = place >> p.page_shift;
        if (place >= 0 && pi < p.max_pages) {
            const int page = __ldg(&p.table[b * p.table_stride + pi]);
            if (page >= 0 && page < p.n_pages)
                page_off = page * p.ko.batch + (place & ((1 << p.page_shift) - 1)) * p.ko.token;
        }
    } else {
        if (t >= p.rows) return;
        b = t / p.N;
        n = t % p.N;
    }

    // this item's two accesses and the pairs they hold
    const int P = spec.n_pairs;
    int off_a, off_b, n_rot, pair0;
    if constexpr (INTER) {
        off_a = 2 * V * item;
        off_b = off_a + V;
        pair0 = V * item;
        n_rot = min(max(P - pair0, 0), 8);
    } else {
        const int turning = P / V;
        if (item < turning) {
            off_a = V * item;
            off_b = P + off_a;
            pair0 = off_a;
            n_rot = V;
        } else {
            off_a = 2 * P + 2 * V * (item - turning);
            off_b = off_a + V;
            pair0 = 0;
            n_rot = 0;
        }
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (i < V && i < n_rot) {
            const int j = pair0 + i;
            const int ax = spec.axis[j];
            int pos;
            if (PAGED && p.pos == nullptr)
                pos = place + p.pos_offset;
            else
                pos = __ldg(&p.pos[ax * p.pos_axis + (PAGED ? t : b * p.pos_batch + n)]);
            const double turns = static_cast<double>(pos) * spec.turns[j];
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn[i], &cs[i]);
            sn[i] *= p.sign;
        }
    }

    const int h_end = min(p.Hq + p.Hk + p.Hv, static_cast<int>(blockIdx.y + 1) * p.heads_per);
    for (int h0 = blockIdx.y * p.heads_per; h0 < h_end; h0 += kRotUnroll) {
        Chunk<V> a[kRotUnroll], c[kRotUnroll];
        __nv_bfloat16* dst[kRotUnroll];
#pragma unroll
        for (int u = 0; u < kRotUnroll; u++) {
            const int h = h0 + u;
            dst[u] = nullptr;
            if (h >= h_end) continue;
            const __nv_bfloat16* src;
            if (h < p.Hq) {
                src = p.q.p + (PAGED ? 0 : b * p.q.batch) + h * p.q.head + n * p.q.token;
                dst[u] = p.qo.p + (PAGED ? 0 : b * p.qo.batch) + h * p.qo.head + n * p.qo.token;
            } else if (h < p.Hq + p.Hk) {
                const int hk = h - p.Hq;
                src = p.k.p + (PAGED ? 0 : b * p.k.batch) + hk * p.k.head + n * p.k.token;
                if constexpr (PAGED) {
                    if (page_off >= 0) dst[u] = p.ko.p + page_off + hk * p.ko.head;
                } else {
                    dst[u] = p.ko.p + b * p.ko.batch + hk * p.ko.head + n * p.ko.token;
                }
            } else {
                const int hv = h - p.Hq - p.Hk;
                src = p.v.p + hv * p.v.head + n * p.v.token;
                if (page_off >= 0) dst[u] = p.vo + page_off + hv * p.ko.head;
            }
            if (dst[u] == nullptr) continue;
            a[u].load(src + off_a);
            c[u].load(src + off_b);
        }
#pragma unroll
        for (int u = 0; u < kRotUnroll; u++) {
            if (dst[u] == nullptr) continue;
            if (n_rot > 0 && (!PAGED || h0 + u < p.Hq + p.Hk)) rotate_chunks<V, INTER>(a[u], c[u], cs, sn, n_rot);
            a[u].store(dst[u] + off_a);
            c[u].store(dst[u] + off_b);
        }
    }
}

}  // namespace sa
