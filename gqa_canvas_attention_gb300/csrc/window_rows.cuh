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

// Elements lane * N .. + N - 1 of one key's K (side 0) or V (side 1) row.
template <int HD, bool KV4>
__device__ __forceinline__ void key_row(const WindowParams &p, int side, int b, int g, int j, int lane, float *x)
{
    constexpr int N = HD / 32;
    if constexpr (KV4) {
        const long long cell = ((long long)b * p.nkv + g) * p.S + j;
        const unsigned char *codes = (side ? p.kv4.v : p.kv4.k) + cell * (HD / 2);
        const float s = e4m3_value((side ? p.kv4.v_scale : p.kv4.k_scale)[cell * (HD / 16) + lane * N / 16]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = lane * N + i;
            x[i] = e2m1_value(codes[e / 2] >> (4 * (e & 1))) * s;
        }
    } else {
        const Rows &r = side ? p.v : p.k;
        const long long at = b * r.batch + j * r.token + g * r.head + lane * N;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = half_value(r.data, at + i, p.bf16);
    }
}

// The whole warp computes row (b, t, h) into out.
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
    for (int step = 0; step < sink + see.hi - see.lo; ++step) {
        const int j = step < sink ? step : see.lo + step - sink;
        float x[N], z = 0.f;
        key_row<HD, KV4>(p, 0, b, g, j, lane, x);
#pragma unroll
        for (int i = 0; i < N; ++i) z = fmaf(q[i], x[i], z);
#pragma unroll
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        z *= p.scale;
        // a score of -inf has weight 0
        const float top = fmaxf(m, z), keep = l == 0.f ? 0.f : expf(m - top);
        const float w = z == -INFINITY ? 0.f : expf(z - top);
        m = top;
        l = l * keep + w;
        key_row<HD, KV4>(p, 1, b, g, j, lane, x);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(w, x[i], o[i] * keep);
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
