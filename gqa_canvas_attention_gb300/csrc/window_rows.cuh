// window_rows.cuh -- one attention row by one warp, reading only the keys the row sees: the plainest
// right form of the operator.
//
// out = sum_j e^(z_j - m) v_j / sum_j e^(z_j - m), z_j = scale q.k_j, m the running maximum; sums in
// fp32.  A row that sees no key, or only keys of score -inf, is 0.
#pragma once
#include "serving.cuh"

#include <cuda_fp8.h>

namespace dg {

__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    const uint32_t m = code & 7u;
    const float v = m < 4 ? 0.5f * m : (m < 6 ? (float)m - 2.f : 2.f * m - 8.f);
    return (code & 8u) ? -v : v;
}

__device__ __forceinline__ float e4m3_value(unsigned char b)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

__device__ __forceinline__ float half_value(const void *p, long long i, bool bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                : __half2float(static_cast<const __half *>(p)[i]);
}

// A lane's elements lane * N .. + N - 1 of one key's K (side 0) or V (side 1) row, as they lie: N 16-bit
// values, or N codes and the byte of their scale.
template <int HD, bool KV4> struct KeyPart {
    static constexpr int N = HD / 32, BYTES = KV4 ? N / 2 : 2 * N;
    uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
    unsigned char scale;

    __device__ __forceinline__ void load(const WindowParams &p, int side, int b, int g, int j, int lane)
    {
        if constexpr (KV4) {
            const long long cell = ((long long)b * p.nkv + g) * p.S + j;
            const unsigned char *at = (side ? p.kv4.v : p.kv4.k) + cell * (HD / 2) + lane * BYTES;
            scale = (side ? p.kv4.v_scale : p.kv4.k_scale)[cell * (HD / 16) + lane * N / 16];
            if constexpr (BYTES == 1) w[0] = *at;
            else if constexpr (BYTES == 2) w[0] = *reinterpret_cast<const unsigned short *>(at);
            else w[0] = *reinterpret_cast<const uint32_t *>(at);
        } else {
            const Rows &r = side ? p.v : p.k;
            const char *at = static_cast<const char *>(r.data) + 2 * (b * r.batch + j * r.token + g * r.head) + lane * BYTES;
            if constexpr (BYTES == 4) w[0] = *reinterpret_cast<const uint32_t *>(at);
            else if constexpr (BYTES == 8) {
                const uint2 x = *reinterpret_cast<const uint2 *>(at);
                w[0] = x.x; w[1] = x.y;
            } else {
                const uint4 x = *reinterpret_cast<const uint4 *>(at);
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void widen(float *x, bool bf16) const
    {
        const float s = KV4 ? e4m3_value(scale) : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (KV4) {
                x[i] = e2m1_value(w[0] >> (4 * i)) * s;
            } else {
                const unsigned short h = (unsigned short)(w[i / 2] >> (16 * (i & 1)));
                x[i] = bf16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
            }
        }
    }
};

// The whole warp computes row (b, t, h) into out.  The faster kernels call it for rows that end as NaN, up to
// every row of a call where K or V holds one: 500 rows of 8 heads over 4500 keys of 256 take 27 ms with a NaN
// in V (one key at a time, an element a load: 90), 0.17 with one in K, which ends a row at once.
constexpr int kAtOnce = 8;
template <int HD, bool KV4>
__device__ __noinline__ void attend_row(const WindowParams &p, int b, int t, int h, int nq, int nk)
{
    constexpr int N = HD / 32;
    const int lane = threadIdx.x & 31;
    const int g = h / p.G;
    const Visible see = visible_keys(p, nq, nk, t);
    const long long qa = b * p.q.batch + t * p.q.token + h * p.q.head + lane * N;
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = half_value(p.q.data, qa + i, p.bf16);
        o[i] = 0.f;
    }
    const int sink = min(p.sinks, see.lo);           // sink keys below the window
    const int n = sink + see.hi - see.lo;
    // kAtOnce keys under way at once: a step is the latency of their loads and of 5 shuffles
    for (int step = 0; step < n; step += kAtOnce) {
        KeyPart<HD, KV4> k[kAtOnce], v[kAtOnce];
        float x[N], w[kAtOnce], top = m;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = min(step + u, n - 1), j = i < sink ? i : see.lo + i - sink;
            k[u].load(p, 0, b, g, j, lane);
            v[u].load(p, 1, b, g, j, lane);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            k[u].widen(x, p.bf16);
            w[u] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) w[u] = fmaf(q[i], x[i], w[u]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) w[u] += __shfl_xor_sync(0xffffffffu, w[u], d);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            w[u] = step + u < n ? w[u] * p.scale : -INFINITY;
            top = fmaxf(top, w[u]);
        }
        const float keep = l == 0.f ? 0.f : expf(m - top);
        m = top;
        l *= keep;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= keep;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            w[u] = w[u] == -INFINITY ? 0.f : expf(w[u] - top);      // a score of -inf has weight 0
            l += w[u];
            if (step + u < n) {
                v[u].widen(x, p.bf16);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fmaf(w[u], x[i], o[i]);
            }
        }
        if (l != l) break;                           // NaN, whatever follows
    }
    const bool none = l == 0.f;                      // no key has a weight (l is 1 at the least after one that has)
    const float inv = 1.0f / l;
    const long long oa = b * p.out.batch + t * p.out.token + h * p.out.head + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = none ? 0.f : o[i] * inv;
        if (p.bf16) static_cast<__nv_bfloat16 *>(p.out.data)[oa + i] = __float2bfloat16_rn(y);
        else static_cast<__half *>(p.out.data)[oa + i] = __float2half_rn(y);
    }
}

// Row `row` (t * G + h mod G) of kv head g over 4-bit keys, which ended as NaN in a kernel that reads every key
// that the rows first .. last see: once more, if there are keys that it does not see, or if no key has a weight
// (`empty`).  Its NaN is its own otherwise: a 4-bit V holds no infinity that a weight rounded to 0 would make one.
template <int HD>
__device__ __noinline__ void mend_row_kv4(const WindowParams &p, int b, int g, int row, int nq, int nk, int first, int last,
                                          bool empty)
{
    const Visible v = visible_keys(p, nq, nk, row / p.G);
    if (empty || v.lo != visible_keys(p, nq, nk, first / p.G).lo ||
        v.hi != visible_keys(p, nq, nk, min(last, nq * p.G - 1) / p.G).hi)
        attend_row<HD, true>(p, b, row / p.G, g * p.G + row % p.G, nq, nk);
}

// Lengths of sequence b, held to the buffers.
__device__ __forceinline__ int query_count(const WindowParams &p, int b)
{
    return p.q_len ? min(max(p.q_len[b], 0), p.T) : p.T;
}
__device__ __forceinline__ int key_count(const WindowParams &p, int b)
{
    return p.kv_len ? min(max(p.kv_len[b], 0), p.S) : p.S;
}

}  // namespace dg
