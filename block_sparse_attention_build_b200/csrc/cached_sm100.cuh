// Attention of new tokens over a paged cache, plain form: one block per row and
// query head, one thread per key for the scores, one per element of the output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace sa {

struct CachedParams {
    const __nv_bfloat16* q;
    int64_t q_token, q_head;
    __nv_bfloat16* o;
    int64_t o_token, o_head;
    float* lse;  // [T, Hq]
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t page_stride, head_stride, token_stride;
    int32_t n_pages, page_shift, max_pages;
    int64_t table_stride;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    const int32_t* prefix_table;
    int32_t prefix_len;
    int32_t B, T, Hq, group;
    int32_t window, cols, n_global;  // cols = max(sinks, n_global)
    float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(128) cached_plain_kernel(const CachedParams p)
{
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    if (t >= __ldg(&p.q_start[p.B])) return;
    int b = 0;
    while (b + 1 < p.B && __ldg(&p.q_start[b + 1]) <= t) b++;
    const int first = p.q_start[b], next = p.q_start[b + 1];
    const int len = min(p.kv_len[b], p.max_pages << p.page_shift);
    const int pos = p.prefix_len + len - (next - first) + (t - first);
    __shared__ float sq[D], sp[128], red[4], stat[2];
    if (tid < D) sq[tid] = __bfloat162float(p.q[t * p.q_token + h * p.q_head + tid]);
    if (tid == 0) {
        stat[0] = -INFINITY;
        stat[1] = 0.f;
    }
    __syncthreads();
    float acc = 0.f;
    const int hk = h / p.group;
    const int end = pos + 1;
    auto row_of = [&](int kv) -> int64_t {
        const bool pre = kv < p.prefix_len;
        const int i = pre ? kv : kv - p.prefix_len;
        const int pg = pre ? p.prefix_table[i >> p.page_shift] : p.table[b * p.table_stride + (i >> p.page_shift)];
        if (pg < 0 || pg >= p.n_pages) return -1;
        return pg * p.page_stride + hk * p.head_stride + (i & ((1 << p.page_shift) - 1)) * p.token_stride;
    };
    auto sees = [&](int kv) {
        return kv < end && (kv < p.cols || pos < p.n_global || (p.window >= 0 && pos - kv <= p.window));
    };
    for (int kv0 = 0; kv0 < end; kv0 += 128) {
        const int kv = kv0 + tid;
        float s = -INFINITY;
        if (sees(kv)) {
            const int64_t r = row_of(kv);
            s = 0.f;
            if (r >= 0)
                for (int d = 0; d < D; d++) s += sq[d] * __bfloat162float(p.k[r + d]);
            s *= p.scale_log2;
        }
        float m = s;
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (tid % 32 == 0) red[tid / 32] = m;
        __syncthreads();
        const float m_old = stat[0];
        m = fmaxf(m_old, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float mu = m == -INFINITY ? 0.f : m;
        const float e = exp2f(s - mu);
        const float a = m_old == -INFINITY ? 0.f : exp2f(m_old - mu);
        sp[tid] = e;
        float l = e;
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        __syncthreads();
        if (tid % 32 == 0) red[tid / 32] = l;
        __syncthreads();
        if (tid == 0) {
            stat[0] = m;
            stat[1] = stat[1] * a + red[0] + red[1] + red[2] + red[3];
        }
        if (tid < D) {
            acc *= a;
            for (int j = 0; j < 128; j++) {
                if (!sees(kv0 + j)) continue;
                const int64_t r = row_of(kv0 + j);
                if (r >= 0) acc += sp[j] * __bfloat162float(p.v[r + tid]);
            }
        }
        __syncthreads();
    }
    const float l = stat[1];
    if (tid < D) p.o[t * p.o_token + h * p.o_head + tid] = __float2bfloat16(l > 0.f ? acc / l : 0.f);
    if (tid == 0)
        p.lse[static_cast<int64_t>(t) * p.Hq + h] = l > 0.f ? (stat[0] + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace sa
