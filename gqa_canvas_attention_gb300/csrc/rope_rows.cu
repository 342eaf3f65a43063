// rope_rows.cu -- rotary positions, and per-head RMS norms with the rotation in the same pass, on
// [batch, T, heads, hd] rows of f32, f16 or bf16.
//
// Pair (a, b) of a head at position p turns by the angle p * f_i:  a' = (a cos - b sin) m,
// b' = (b cos + a sin) m; the pairs are (x[i], x[i + rot/2]) in the half layout and
// (x[2i], x[2i+1]) in the interleaved one, the elements from rot on pass through.  With norms,
// x = x (mean x^2 + eps)^-1/2 w first (v: no weight, no rotation), all in fp32 and rounded once.
//
// The angle: f_i / 2 pi is held as a 64-bit fraction of a turn, so p * f_i modulo one turn is one
// wrapping 64-bit integer product, off by less than |p| 2^-64 turns (of the double f_i); its upper 32
// bits give the argument of sincospi.  cos and sin are made once a token and shared by its heads.
//
// Bound by memory, and next by instruction issue (60 to 65% of the slots): a block takes a few tokens
// for as many heads as it has groups of hd/8 lanes; a group keeps its head, so that pointers and weights
// stay in registers, and walks the tokens, whose rows are all in flight (asynchronous copies that only
// the lane reads).  A lane's 8 elements are chosen so that both ends of a pair are its own.
// Measured: 262 MB (4 prompts of 4001 tokens, 16 + 8 + 8 heads of 128, norms) in 51.4 us, 5.1 TB/s, 75%
// of a copy; 101 MB (a prompt of 8192, 16 + 8 heads of 128, half of each turned) in 20.5 us, 73%; a
// step of single tokens takes 7.7 us, the host's, and 2.1 us in a graph.
#include "serving.cuh"

#include <atomic>

namespace dg {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;       // tokens of a block at most: the rows a lane has in flight

template <bool B> struct Flag {
    static constexpr bool value = B;
};

template <bool WIDE> struct Raw;
template <> struct Raw<true> { using T = float4; };
template <> struct Raw<false> { using T = uint2; };

__device__ __forceinline__ void widen(float *x, float4 r, bool)
{
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
}
__device__ __forceinline__ void widen(float *x, uint2 r, bool bf16)
{
    if (bf16) {
        x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xffff0000u);
        x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xffff0000u);
    } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
}
__device__ __forceinline__ void narrow(const float *x, float4 &r, bool)
{
    r = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void narrow(const float *x, uint2 &r, bool bf16)
{
    if (bf16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        r = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
        r = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

template <int B> __device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
}
// Waits until at most `pending` (a constant after unrolling) of the copy groups are on their way.
__device__ __forceinline__ void wait_copies(int pending)
{
    switch (pending) {
    case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    }
}

// Packed pairs of fp32.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

template <int HD, bool IN_WIDE, bool OUT_WIDE, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads, IN_WIDE ? 3 : 5) rope_rows_kernel(const __grid_constant__ RopeRowsParams p)
{
    constexpr int LPR = HD / 8;                  // lanes of a row
    constexpr int NS = kThreads / LPR;           // heads of the block
    constexpr int IN_B = IN_WIDE ? 4 : 2, OUT_B = OUT_WIDE ? 4 : 2;
    using InT = typename Raw<IN_WIDE>::T;
    using OutT = typename Raw<OUT_WIDE>::T;
    // [tokens][cos(rot/2) | sin(rot/2)], then the lanes' rows on their way: [token][half][thread]
    extern __shared__ float4 smem4[];
    float *cs = reinterpret_cast<float *>(smem4);
    constexpr int PART = 4 * IN_B;                   // bytes of a lane's half of a row
    const char *const mine = reinterpret_cast<const char *>(cs + p.tokens_per_block * p.rot);
    const uint32_t mine32 = (uint32_t)__cvta_generic_to_shared(mine);

    const int t0 = blockIdx.x * p.tokens_per_block, ntok = min(p.tokens_per_block, p.T - t0);
    const int l = threadIdx.x % LPR, half_rot = p.rot / 2;
    int head = blockIdx.y * NS + threadIdx.x / LPR, which = 0;
    const bool live = head < p.H;
    if (head >= p.heads[0]) { head -= p.heads[0]; which = 1; if (head >= p.heads[1]) { head -= p.heads[1]; which = 2; } }
    if (!live) which = head = 0;
    // the lane's elements e0..e0+3 and e1..e1+3; rotated lanes hold 4 whole pairs
    const bool turns = which < 2 && l < p.rot / 8;
    int e0 = 8 * l, e1 = 8 * l + 4;
    if (l < p.rot / 8 && !INTERLEAVED) { e0 = 4 * l; e1 = half_rot + 4 * l; }
    const bool in_bf16 = p.in_type == kRowBf16, out_bf16 = p.out_type == kRowBf16;
    float2 w[4] = {{1.f, 1.f}, {1.f, 1.f}, {1.f, 1.f}, {1.f, 1.f}};
    if (NORM && which < 2 && p.w[which]) {
        const float4 a = *reinterpret_cast<const float4 *>(p.w[which] + e0);
        const float4 c = *reinterpret_cast<const float4 *>(p.w[which] + e1);
        w[0] = make_float2(a.x, a.y); w[1] = make_float2(a.z, a.w);
        w[2] = make_float2(c.x, c.y); w[3] = make_float2(c.z, c.w);
    }
    const Rows &in = p.in[which], &out = p.out[which];
    const long long in_step = in.token * IN_B, out_step = out.token * OUT_B;

    for (int b = blockIdx.z; b < p.batch; b += gridDim.z) {
        const char *src = static_cast<const char *>(in.data) + (b * in.batch + t0 * in.token + head * in.head) * IN_B;
        char *dst = static_cast<char *>(out.data) + (b * out.batch + t0 * out.token + head * out.head) * OUT_B;
        // every row of the lane is asked for at once (cp.async: no registers wait for them)
        for (int u = 0; u < kTokens; ++u) {
            if (live && u < ntok) {
                const char *x = src + u * in_step;
                if constexpr (INTERLEAVED && !IN_WIDE) {         // 8 elements in a row
                    copy_async<16>(mine32 + (u * kThreads + threadIdx.x) * 16, x + e0 * IN_B);
                } else {
                    copy_async<PART>(mine32 + (2 * u * kThreads + threadIdx.x) * PART, x + e0 * IN_B);
                    copy_async<PART>(mine32 + ((2 * u + 1) * kThreads + threadIdx.x) * PART, x + e1 * IN_B);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }

        const long long pos0 = (long long)b * p.T + t0;
        __syncthreads();                             // the batch before is done with cs
        for (int i = threadIdx.x; i < ntok * half_rot; i += kThreads) {
            const int tk = i / half_rot, f = i - tk * half_rot;
            const long long pos = p.pos64 ? static_cast<const long long *>(p.positions)[pos0 + tk]
                                          : static_cast<const int *>(p.positions)[pos0 + tk];
            const unsigned long long turn = (unsigned long long)pos * p.turn[f] + 0x80000000ull;
            float sn, cn;
            sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cn);
            cs[tk * p.rot + f] = cn * p.magnitude;
            cs[tk * p.rot + half_rot + f] = sn * p.magnitude;
        }
        __syncthreads();

#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (u < ntok) {                          // the whole block
                wait_copies(kTokens - 1 - u);
                InT raw[2];
                if constexpr (INTERLEAVED && !IN_WIDE) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(mine + (u * kThreads + threadIdx.x) * 16);
                    raw[0] = make_uint2(v.x, v.y);
                    raw[1] = make_uint2(v.z, v.w);
                } else {
                    raw[0] = *reinterpret_cast<const InT *>(mine + (2 * u * kThreads + threadIdx.x) * PART);
                    raw[1] = *reinterpret_cast<const InT *>(mine + ((2 * u + 1) * kThreads + threadIdx.x) * PART);
                }
                float2 x[4];
                widen(&x[0].x, raw[0], in_bf16);
                widen(&x[2].x, raw[1], in_bf16);
                if constexpr (NORM) {
                    float2 ss = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
                    float sum = ss.x + ss.y;
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float inv = rsqrtf(sum * (1.0f / HD) + p.eps);
                    const float2 ii = make_float2(inv, inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(x[i], ii), w[i]);
                }
                if (turns) {
                    const float *row = cs + u * p.rot + 4 * l;
                    const float4 c = *reinterpret_cast<const float4 *>(row);
                    const float4 n = *reinterpret_cast<const float4 *>(row + half_rot);
                    if constexpr (INTERLEAVED) {
                        // pair i of the lane: x[i].x, x[i].y
                        const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = make_float2(x[i].x * cc[i] - x[i].y * nn[i], x[i].y * cc[i] + x[i].x * nn[i]);
                    } else {
                        // x[0], x[1] against x[2], x[3]
                        const float2 cc[2] = {{c.x, c.y}, {c.z, c.w}}, nn[2] = {{n.x, n.y}, {n.z, n.w}};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 a = x[i], d = x[i + 2];
                            x[i] = fma2(make_float2(-d.x, -d.y), nn[i], mul2(a, cc[i]));
                            x[i + 2] = fma2(a, nn[i], mul2(d, cc[i]));
                        }
                    }
                }
                if (live) {
                    char *y = dst + u * out_step;
                    OutT o0, o1;
                    narrow(&x[0].x, o0, out_bf16);
                    narrow(&x[2].x, o1, out_bf16);
                    if constexpr (INTERLEAVED && !OUT_WIDE) {
                        *reinterpret_cast<uint4 *>(y + e0 * OUT_B) = make_uint4(o0.x, o0.y, o1.x, o1.y);
                    } else {
                        *reinterpret_cast<OutT *>(y + e0 * OUT_B) = o0;
                        *reinterpret_cast<OutT *>(y + e1 * OUT_B) = o1;
                    }
                }
            }
        }
    }
}

// SMs of the current device, asked for once a device.
cudaError_t sm_count(int &n)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    n = e == cudaSuccess && device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
    if (e != cudaSuccess || n > 0) return e;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess && device < kDevices) known[device].store(n, std::memory_order_relaxed);
    return e;
}

template <int HD>
cudaError_t launch_hd(RopeRowsParams &p, cudaStream_t s)
{
    constexpr int NS = kThreads / (HD / 8);
    int sms = 0;
    cudaError_t e = sm_count(sms);
    if (e != cudaSuccess) return e;
    if (p.T == 1) {
        // single tokens: the batch is the run of tokens
        p.T = p.batch;
        p.batch = 1;
        for (int i = 0; i < 3; ++i) {
            p.in[i].token = p.in[i].batch;
            p.out[i].token = p.out[i].batch;
        }
    }
    // 8 tokens a block, fewer (down to one) while that leaves SMs without work.  us with 1, 2, 4, 8: the prompt
    // of 8192 43, 29, 22.5, 20.5, norms of 4 x 4001 tokens 102, 70, 57, 52, 512 fp32 tokens 11.7, 10.1, 12.5,
    // 10.4; a single one of 16 heads 7.3, 7.3, 7.8, 8.3.  The half layout alone, whose copies are of 8 bytes,
    // takes 4: 8192 tokens of 32 heads of 128 with events around them 30 against 34 with 8, 64 of 64 30
    // against 33.
    const int groups = (p.H + NS - 1) / NS;
    long long rows = (long long)p.batch * p.T * groups;
    p.tokens_per_block = p.norm || p.interleaved ? kTokens : kTokens / 2;
    while (p.tokens_per_block > 1 && rows / p.tokens_per_block < 2 * sms) p.tokens_per_block /= 2;
    const dim3 grid((p.T + p.tokens_per_block - 1) / p.tokens_per_block, groups, p.batch < 65535 ? p.batch : 65535);
    const bool iw = p.in_type == kRowF32, ow = p.out_type == kRowF32;
    const size_t smem = (size_t)p.tokens_per_block * (p.rot * sizeof(float) + kThreads * (iw ? 32 : 16));
    auto launch = [&](auto kernel) {
        // beyond 48 KB: fp32 rows of 8 tokens
        if (smem > 49152) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) kernel<<<grid, kThreads, smem, s>>>(p);
    };
    auto typed = [&](auto inter, auto norm) {
        constexpr bool I = decltype(inter)::value, N = decltype(norm)::value;
        if (iw) ow ? launch(rope_rows_kernel<HD, true, true, I, N>) : launch(rope_rows_kernel<HD, true, false, I, N>);
        else ow ? launch(rope_rows_kernel<HD, false, true, I, N>) : launch(rope_rows_kernel<HD, false, false, I, N>);
    };
    if (p.interleaved) p.norm ? typed(Flag<true>(), Flag<true>()) : typed(Flag<true>(), Flag<false>());
    else p.norm ? typed(Flag<false>(), Flag<true>()) : typed(Flag<false>(), Flag<false>());
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_rope_rows(RopeRowsParams &p, int hd, cudaStream_t s)
{
    switch (hd) {
    case 32: return launch_hd<32>(p, s);
    case 64: return launch_hd<64>(p, s);
    case 128: return launch_hd<128>(p, s);
    case 256: return launch_hd<256>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dg
