// window_few.cu -- attention with a sliding window and sink tokens for few query rows of a kv head
// (single tokens): at most 8 (hd 256: 4) over 16-bit keys and values, 16 (8) over 4-bit ones.
//
// With the G query heads of a kv head as rows, K and V are read once for all of them and the time
// is the time of that read; the products run on mma.sync, whose 16-row operand is the cache side:
//   S^T = K Q^T   (16 keys x 8 rows a step),   O^T += V^T P^T   (16 channels x 8 rows a step).
// Both contractions may run over channels and keys in any order, so the order is chosen for the loads.
//   16-bit: a warp copies K and V tiles of 16 keys in turn into its ring in shared memory (cp.async),
//     eight lanes 128 bytes of a row, to where the threads' fragments are read without conflicts.  With
//     each thread copying its own pieces, eight lanes met four rows of V: 3.6 TB/s where this order
//     reads 5.7 (copies alone, 537 MB).
//   4-bit: a warp copies tiles of 32 keys as they lie (dense rows), in an order of rows and 16-byte units
//     by which the reads of fragments meet no bank twice.  Codes become f16 pairs in registers, times
//     their scale (exactly: 2 bits times 4 bits).  V needs pairs of keys: the nibbles of two keys' words
//     are laced first (4 operations for 16 values), then converted.
//
// Softmax: the row's reference m moves only when a score passes it by kSlack (then O is rescaled),
// P = 2^(z - m + kLift) is rounded to V's type, and the denominator sums the rounded values.  kLift
// keeps f16's subnormals 2^-29 and more below the largest weight.
//
// Work: the key tiles of all sequences and kv heads stand in one line, which is cut into equal runs,
// one a CTA, whose four warps take tiles in turn.  Every CTA reads the lengths and finds its run, so
// ragged batches fill the GPU once and evenly.  Where a run ends inside a pair (sequence, kv head), its
// (m, l, O) goes to the plan's scratch; the last CTA of the pair to arrive merges the pieces in their
// order, so results do not depend on which one it is.
//
// Bound by the read of K and V.  16-bit, 135 MB (32 sequences, windows of 1024, 4 kv heads of 256): 31.1
// us, of which the same copies with nothing else take 30.4; at 537 MB the rate grows by 6.1 TB/s.  4-bit,
// 449 MB (16 sequences of up to 32768, 8 kv heads of 128): 88.4 us, 5.1 TB/s, 75% of a copy; its
// unpacking issues in 60% of the slots.  Runs cut at the ends of pairs, fewer and uneven, took as long
// (39.1 against 38.5) or longer (102 against 88).
#include "window_rows.cuh"

namespace dg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kSlack = 8.0f, kLift = 5.0f;       // log2 units
constexpr float kLog2e = 1.4426950408889634f;

enum KvKind : int { kF16 = 0, kBf16 = 1, kKv4 = 2 };

template <int HD, int KV> struct Piece {
    static constexpr bool Q4 = KV == kKv4;
    static constexpr int MT = Q4 ? 2 : 1, TK = 16 * MT;      // 16-key steps and keys of a tile
    // K: a thread of a quad has KP pieces of KB bytes (KE elements) of a row; V: a thread of eight VP
    // pieces of VB bytes (VE elements)
    static constexpr int KB = Q4 ? (HD == 64 ? 8 : 16) : 16;
    static constexpr int KE = Q4 ? 2 * KB : KB / 2;
    static constexpr int KP = HD / 4 / KE;
    static constexpr int VB = Q4 ? HD / 16 : 16;
    static constexpr int VE = Q4 ? 2 * VB : VB / 2;
    static constexpr int VP = HD / 8 / VE;
    // 16-bit: a stage is a K or a V tile; 4-bit: K and V codes and their scales
    static constexpr int ROW = HD / 2, SROW = HD / 16;       // bytes of a row of codes, of scales
    static constexpr int STAGE = Q4 ? 2 * TK * (ROW + SROW) : TK * HD * 2;
    static constexpr int STAGES = Q4 ? (HD == 256 ? 3 : 4) : (HD == 64 ? 5 : 3);
    static constexpr int RING = STAGE * STAGES * kWarps;
    // CTAs an SM is to hold
    static constexpr int CTAS = HD == 256 ? (Q4 ? 2 : 2) : HD == 128 ? 3 : 4;
};
template <int HD, int KV, int NT> constexpr int smem_bytes()
{
    constexpr int staged = kWarps * 8 * NT * (HD + 4) * 4;
    return Piece<HD, KV>::RING > staged ? Piece<HD, KV>::RING : staged;
}

template <int B> __device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool live)
{
    const int n = live ? B : 0;                     // 0: zeros
    if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(B)
                     : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int B> __device__ __forceinline__ void load_shared(uint32_t addr, uint32_t *w)
{
    if constexpr (B == 16)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else if constexpr (B == 8)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

template <int KV>
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (KV == kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight e2m1 values (one word), a pair a byte, times a pair of scales, as four f16 pairs.
__device__ __forceinline__ void widen_e2m1(uint32_t w, uint32_t scale2, uint32_t *d)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(w));
    const __half2 s = *reinterpret_cast<const __half2 *>(&scale2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&d[i]), s);
        d[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
}
// Two e4m3 scales (the low 16 bits) as an f16 pair.
__device__ __forceinline__ uint32_t widen_scales(uint32_t two)
{
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(two));
    return d;
}
__device__ __forceinline__ uint32_t load_shared_u16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_shared_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u8 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// a * b / c, with 32-bit division where that is enough
__device__ __noinline__ long long scaled_wide(unsigned long long n, unsigned long long c) { return (long long)(n / c); }
__device__ __forceinline__ long long scaled(long long a, long long b, long long c)
{
    const unsigned long long n = (unsigned long long)a * (unsigned long long)b;
    if ((n | (unsigned long long)c) >> 32) return scaled_wide(n, (unsigned long long)c);
    return (unsigned)n / (unsigned)c;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Rows that see no key are zeros.
template <int HD> __device__ __noinline__ void clear_rows(const WindowParams &p, int b, int gh)
{
    const int nq = query_count(p, b);
    for (int i = threadIdx.x; i < nq * p.G * (HD / 8); i += kThreads) {
        const int r = i / (HD / 8), t = r / p.G, h = gh * p.G + r % p.G;
        *reinterpret_cast<uint4 *>(static_cast<char *>(p.out.data) +
                                   2 * (b * p.out.batch + t * p.out.token + h * p.out.head) +
                                   16 * (i % (HD / 8))) = make_uint4(0, 0, 0, 0);
    }
}

template <int HD, int KV, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 && Piece<HD, KV>::CTAS > 2 ? 2 : Piece<HD, KV>::CTAS)
window_few_kernel(const __grid_constant__ WindowParams p)
{
    using P = Piece<HD, KV>;
    constexpr int ROWS = 8 * NT;
    constexpr int KSTEPS = HD / 16;
    constexpr int MT = P::MT, TK = P::TK;
    constexpr bool Q4 = KV == kKv4;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 ml[kWarps][ROWS];
    __shared__ int last_here, mend[ROWS];
    __shared__ int seq_tiles[kFewSequences];
    __shared__ long long scan[2];                     // units before the run's sequence, that sequence

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;

    // tiles of a sequence's keys that some row sees
    auto tiles_of = [&](int b) {
        const int nq = query_count(p, b), nk = key_count(p, b);
        const int lo = visible_keys(p, nq, nk, 0).lo, hi = visible_keys(p, nq, nk, nq - 1).hi;
        const int n = (min(p.sinks, lo) + TK - 1) / TK + (hi - lo + TK - 1) / TK;
        return nq ? n : 0;
    };
    long long unit, unit_end, units = 0, runs = 1;
    int b, gh, t_first;                               // where the run starts: pair and tile
    auto cut = [&](long long pairs) {
        // as many runs as CTAs, but of 4 warps' 2 tiles or more, and no more pieces of a pair than the merge is
        // worth: it reads rows * hd * 4 bytes a piece at ~60 bytes a clock, a tile takes ~150 clocks
        runs = 1;
        if (units > 0) {
            const float each = __fdividef((float)units, (float)pairs);
            const long long most = pairs * max(1, (int)sqrtf(each * __fdividef(9000.0f / (HD * 4), (float)p.rows_cap)));
            runs = min(min((long long)gridDim.x, max(1ll, units >> 3)), most);
        }
        unit = blockIdx.x < runs ? scaled(blockIdx.x, units, runs) : units;
        unit_end = blockIdx.x < runs ? scaled(blockIdx.x + 1, units, runs) : units;
    };
    if (p.batch <= 32) {
        // every warp for itself: a lane a sequence
        const int mine = lane < p.batch ? tiles_of(lane) : 0;
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += x;
        }
        const unsigned some = __ballot_sync(0xffffffffu, mine > 0);
        units = (long long)__shfl_sync(0xffffffffu, before, 31) * p.nkv;
        before -= mine;
        cut((long long)__popc(some) * p.nkv);
        // sequences without a visible key, dealt to the CTAs
        for (unsigned none = ~some & (0xffffffffu >> (32 - p.batch)); none; none &= none - 1)
            for (int k = blockIdx.x; k < p.nkv; k += gridDim.x) clear_rows<HD>(p, __ffs(none) - 1, k);
        if (unit >= unit_end) return;
        const unsigned at = __ballot_sync(0xffffffffu, mine > 0 && (long long)before * p.nkv <= unit);
        b = 31 - __clz(at);
        const int tiles = __shfl_sync(0xffffffffu, mine, b);
        const long long in = unit - (long long)__shfl_sync(0xffffffffu, before, b) * p.nkv;
        gh = (int)scaled(in, 1, tiles);
        t_first = (int)(in - (long long)gh * tiles);
    } else if (p.batch <= kFewSequences) {
        for (int i = threadIdx.x; i < p.batch; i += kThreads) seq_tiles[i] = tiles_of(i);
        __syncthreads();
        // a lane sums a stretch of sequences; a scan over the lanes finds the run's start
        const int per = (p.batch + 31) / 32;
        long long mine = 0, before;
        int live = 0;
        for (int i = lane * per; i < min(p.batch, (lane + 1) * per); ++i) {
            mine += seq_tiles[i];
            live += seq_tiles[i] > 0;
        }
        before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += x;
            live += __shfl_xor_sync(0xffffffffu, live, d);
        }
        units = __shfl_sync(0xffffffffu, before, 31) * p.nkv;
        before -= mine;
        cut((long long)live * p.nkv);
        if (warp == 0 && unit < unit_end && unit >= before * p.nkv && unit < (before + mine) * p.nkv) {
            int i = lane * per;
            while ((before + seq_tiles[i]) * p.nkv <= unit) before += seq_tiles[i++];
            scan[0] = before * p.nkv;
            scan[1] = i;
        }
        for (int i = blockIdx.x; i < p.batch * p.nkv; i += gridDim.x)
            if (seq_tiles[i / p.nkv] == 0) clear_rows<HD>(p, i / p.nkv, i % p.nkv);
        __syncthreads();
        if (unit >= unit_end) return;
        b = (int)scan[1];
        const long long in = unit - scan[0];
        gh = (int)scaled(in, 1, seq_tiles[b]);
        t_first = (int)(in - (long long)gh * seq_tiles[b]);
    } else {
        // a batch this large fills the GPU with one CTA a pair
        b = blockIdx.x / p.nkv;
        gh = blockIdx.x % p.nkv;
        t_first = 0;
        unit = 0;
        unit_end = tiles_of(b);
        if (unit_end == 0) {
            clear_rows<HD>(p, b, gh);
            return;
        }
    }
    const long long unit_begin = unit;
    uint8_t *const ring_at = smem + warp * (P::STAGE * P::STAGES);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_at);
    // 4-bit: the order of 8 keys that makes the V reads of a thread's keys c, c + 4 (rows 2c, 2c + 1 of the
    // product) and the K reads of rows g meet every bank once
    const int order_g = (g >> 1) + 4 * (g & 1);       // key of product row g

    while (true) {
    const int nq = query_count(p, b), nk = key_count(p, b);
    const int rows = nq * p.G;
    // the keys that some row sees: sinks [0, sk) and [lo, hi); those every row sees: [lo_all, hi_all)
    const Visible first = visible_keys(p, nq, nk, 0), final = visible_keys(p, nq, nk, nq - 1);
    const int lo = first.lo, hi = final.hi, lo_all = final.lo, hi_all = first.hi;
    const int sk = min(p.sinks, lo);
    const int sink_tiles = (sk + TK - 1) / TK, tiles = sink_tiles + (hi - lo + TK - 1) / TK;
    const int tile0 = t_first, tile1 = (int)min((long long)tiles, t_first + (unit_end - unit));
    const bool whole_pair = tile0 == 0 && tile1 == tiles;

    // visible ranges of the rows in this thread's score columns
    int row_lo[NT][2], row_hi[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * c + e;
            const Visible v = r < rows ? visible_keys(p, nq, nk, r / p.G) : Visible{0, 0};
            row_lo[n][e] = v.lo;
            row_hi[n][e] = v.hi;
        }
    auto tile_key = [&](int tile) { return tile < sink_tiles ? TK * tile : lo + TK * (tile - sink_tiles); };
    auto tile_left = [&](int tile) { return (tile < sink_tiles ? sk : hi) - tile_key(tile); };   // live rows, 1 and more

    // sources: row 0 of the sequence
    const char *k_src, *v_src;
    const unsigned char *ks_src = nullptr, *vs_src = nullptr;
    long long k_row, v_row;
    if constexpr (Q4) {
        const long long cell = ((long long)b * p.nkv + gh) * p.S;
        k_row = v_row = P::ROW;
        k_src = reinterpret_cast<const char *>(p.kv4.k) + cell * P::ROW;
        v_src = reinterpret_cast<const char *>(p.kv4.v) + cell * P::ROW;
        ks_src = p.kv4.k_scale + cell * P::SROW;
        vs_src = p.kv4.v_scale + cell * P::SROW;
    } else {
        k_row = 2 * p.k.token;
        v_row = 2 * p.v.token;
        k_src = static_cast<const char *>(p.k.data) + 2 * (b * p.k.batch + gh * p.k.head);
        v_src = static_cast<const char *>(p.v.data) + 2 * (b * p.v.batch + gh * p.v.head);
    }
    // 4-bit stage: K codes, V codes, K scales, V scales of 32 keys
    constexpr int V_AT = TK * P::ROW, KS_AT = 2 * TK * P::ROW, VS_AT = KS_AT + TK * P::SROW;
    constexpr int UPR = P::ROW / 16, CP = TK * UPR / 32;      // 16-byte units of a row, copies of a lane
    auto issue4 = [&](int tile, int stage) {
        __syncwarp();                                 // every lane has read what stood there
        if (tile >= tile0 && tile < tile1) {
            const int left = tile_left(tile);
            const long long k0 = tile_key(tile);
            const uint32_t at = ring + stage * P::STAGE;
            const char *kt = k_src + k0 * P::ROW, *vt = v_src + k0 * P::ROW;
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                const int x = 32 * i + lane, row = x / UPR, unit16 = x % UPR;
                const bool live = row < left;
                const int from = live ? 16 * x : 0;
                // K row r of 8 stands in the place of its product row; hd 256: units of odd places are swapped
                const int place = (row & ~7) + 2 * (row & 3) + (row >> 2 & 1);
                const int ku = HD == 256 ? unit16 ^ ((place & 1) << 2) : unit16;
                const int vu = HD == 256 ? unit16 ^ ((row & 3) << 1) : HD == 128 ? unit16 ^ (row & 2) : unit16;
                copy_async<16>(at + place * P::ROW + 16 * ku, kt + from, live);
                copy_async<16>(at + V_AT + row * P::ROW + 16 * vu, vt + from, live);
            }
            const bool live = lane < left;
            const int from = live ? lane * P::SROW : 0;
            copy_async<P::SROW>(at + KS_AT + lane * P::SROW, ks_src + k0 * P::SROW + from, live);
            copy_async<P::SROW>(at + VS_AT + lane * P::SROW, vs_src + k0 * P::SROW + from, live);
        }
        commit_copies();
    };
    // 16-bit stages: K of the n-th tile of the warp is stage 2 n, its V stage 2 n + 1.  Eight lanes copy 128
    // bytes of a row.  A stage holds a thread's pieces 512 bytes apart, and within 512 bytes the 32 lanes' in
    // an order by which neither the copies nor the reads meet a bank twice.
    constexpr int UPT = HD / 8;                       // 16-byte units of a 16-bit row
    auto issue16 = [&](int tile, int stage, const char *src, long long pitch, bool is_v) {
        __syncwarp();                                 // every lane has read what stood there
        if (tile < tile1) {
            const int left = tile_left(tile);
            const char *from = src + tile_key(tile) * pitch + 16 * (lane % UPT);
            const uint32_t at = ring + stage * P::STAGE;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const int row = (32 * k + lane) / UPT, u = (32 * k + lane) % UPT;
                const bool live = row < left;
                uint32_t to;
                if (is_v) {
                    // row 2c, 2c + 1 (+ 8) of the tile and unit 8 i + g go to thread (g, c)
                    const int r = (row & 1) + 2 * (row >> 3), tc = row >> 1 & 3, i = u >> 3;
                    to = (r * P::VP + i) * 32 + tc * 8 + ((u & 7) ^ (2 * tc));
                } else {
                    // row g (+ 8) and unit 4 i + c
                    const int i = u >> 2;
                    to = ((row >> 3) * P::KP + i) * 32 + (((row & 7) * 4 + (u & 3)) ^ (4 * (i & 1)));
                }
                copy_async<16>(at + 16 * to, from + (live ? row : 0) * pitch, live);
            }
        }
        commit_copies();
    };
    auto issue_k = [&](int tile, int stage) { issue16(tile, stage, k_src, k_row, false); };
    auto issue_v = [&](int tile, int stage) { issue16(tile, stage, v_src, v_row, true); };
    // Q as operand fragments, in the channel order of the K pieces; z = score * zscale in log2 units
    uint32_t qf[NT][KSTEPS][2];
    float zscale[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        const int t = r / p.G, h = gh * p.G + r % p.G;
        const char *src = static_cast<const char *>(p.q.data) + 2 * (b * p.q.batch + t * p.q.token + h * p.q.head);
#pragma unroll
        for (int i = 0; i < P::KP; ++i)
#pragma unroll
            for (int e = 0; e < P::KE / 8; ++e) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < rows) w = *reinterpret_cast<const uint4 *>(src + 2 * ((4 * i + c) * P::KE + 8 * e));
                const int ks = (i * P::KE + 8 * e) / 4;
                qf[n][ks][0] = w.x; qf[n][ks][1] = w.y;
                qf[n][ks + 1][0] = w.z; qf[n][ks + 1][1] = w.w;
            }
        float own = p.scale * kLog2e;
        if constexpr (Q4) {
            if (p.bf16) {
                // bf16 rows into f16, the row's largest element brought to [1, 2) by a power of two: what
                // is lost lies 2^-25 and more below it
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[n][k][e] << 16)),
                                               fabsf(__uint_as_float(qf[n][k][e] & 0xffff0000u))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = top > 0.f && top <= 3.402823466e38f ? ilogbf(top) : 0;
                const float up = exp2f((float)(-ex / 2)), down = exp2f((float)(-ex - -ex / 2));
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __half2 x = __floats2half2_rn(__uint_as_float(qf[n][k][e] << 16) * up * down,
                                                            __uint_as_float(qf[n][k][e] & 0xffff0000u) * up * down);
                        qf[n][k][e] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                own = ldexpf(own, ex);
            }
        }
        zscale[n][0] = __shfl_sync(0xffffffffu, own, 8 * c);       // row 2c is held by lanes with g = 2c
        zscale[n][1] = __shfl_sync(0xffffffffu, own, 8 * c + 4);
    }

    float o[NT][HD / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }

    int stage = 0;
    // one stage on: where to read, and where the copies of STAGES - 1 stages ahead go
    auto advance = [&](int &ahead) {
        const int now = stage;
        ahead = stage == 0 ? P::STAGES - 1 : stage - 1;
        if (++stage == P::STAGES) stage = 0;
        return now;
    };
    // the ring is filled by the loop's own copies, in turns before the first tile: code that runs once
    // waits for its instructions
    constexpr int FILL = Q4 ? P::STAGES - 1 : P::STAGES / 2;
#pragma unroll 1
    for (int tile = tile0 + warp - FILL * kWarps; tile < tile1; tile += kWarps) {
        const bool turn = tile >= tile0;
        // scores: rows of s are the product rows g and g + 8 of each 16 keys, columns query rows 2c, 2c + 1
        float s[NT][MT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < MT; ++t) s[n][t][0] = s[n][t][1] = s[n][t][2] = s[n][t][3] = 0.f;
        int ahead, now = advance(ahead);
        if constexpr (Q4) {
            issue4(tile + (P::STAGES - 1) * kWarps, ahead);
            if (!turn) continue;
            wait_copies<P::STAGES - 1>();
            __syncwarp();
            const uint32_t at = ring + now * P::STAGE;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                // this thread's scales: of pieces i, two (hd 64: one) a row
                uint32_t two[2][P::KP];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < P::KP; ++i) {
                        const uint32_t sa = at + KS_AT + (16 * t + 8 * r + order_g) * P::SROW + (4 * i + c) * P::KE / 16;
                        if constexpr (HD == 64) two[r][i] = load_shared_u8(sa) * 0x101u;
                        else two[r][i] = load_shared_u16(sa);
                        two[r][i] = widen_scales(two[r][i]);
                    }
#pragma unroll
                for (int i = 0; i < P::KP; ++i) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int place = 16 * t + 8 * r + g;
                        const int u = HD == 256 ? (4 * i + c) ^ ((g & 1) << 2) : 4 * i + c;
                        load_shared<P::KB>(at + place * P::ROW + u * P::KB, w[r]);
                    }
#pragma unroll
                    for (int v = 0; v < P::KB / 4; ++v) {
                        uint32_t d[2][4];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            widen_e2m1(w[r][v], __byte_perm(two[r][i], 0, v / 2 ? 0x3232 : 0x1010), d[r]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ks = (i * P::KE + 8 * v) / 4 + e;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma<KV>(s[n][t], d[0][2 * e], d[1][2 * e], d[0][2 * e + 1], d[1][2 * e + 1],
                                        qf[n][ks][0], qf[n][ks][1]);
                        }
                    }
                }
            }
        } else {
            constexpr int AHEAD = P::STAGES - 1;      // even: two stages a tile
            issue_k(tile + AHEAD / 2 * kWarps, ahead);
            if (!turn) {
                now = advance(ahead);
                issue_v(tile + AHEAD / 2 * kWarps, ahead);
                continue;
            }
            wait_copies<P::STAGES - 1>();
            __syncwarp();
            const uint32_t at = ring + now * P::STAGE;
#pragma unroll
            for (int i = 0; i < P::KP; ++i) {
                uint32_t w[2][4];
                const uint32_t mine = at + 16 * (lane ^ (4 * (i & 1)));
                load_shared<P::KB>(mine + i * 32 * P::KB, w[0]);
                load_shared<P::KB>(mine + (P::KP + i) * 32 * P::KB, w[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma<KV>(s[n][0], w[0][2 * e], w[1][2 * e], w[0][2 * e + 1], w[1][2 * e + 1], qf[n][2 * i + e][0],
                                qf[n][2 * i + e][1]);
            }
        }

        // masks: only tiles at the ends of the rows' ranges
        const bool sink = tile < sink_tiles;
        const int k0 = tile_key(tile);
        const bool whole = sink ? k0 + TK <= min(sk, hi_all) : (k0 >= lo_all && k0 + TK <= min(hi, hi_all));
        float top[NT][2];
        bool moves = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][t][e] *= zscale[n][e & 1];
            if (!whole) {
                const int end = sink ? sk : hi;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = k0 + 16 * t + 8 * (e >> 1) + (Q4 ? order_g : g);
                        const bool see = j < end && j < row_hi[n][e & 1] && (j >= row_lo[n][e & 1] || j < p.sinks);
                        if (!see) s[n][t][e] = -INFINITY;
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[n][e] = fmaxf(s[n][0][e], s[n][0][e + 2]);
                if constexpr (MT == 2) top[n][e] = fmaxf(top[n][e], fmaxf(s[n][1][e], s[n][1][e + 2]));
                moves = moves || top[n][e] > m[n][e] + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = top[n][e];
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                    t = fmaxf(m[n][e], t);
                    const float keep = m[n][e] == -INFINITY ? 0.f : exp2_fast(m[n][e] - t);
                    m[n][e] = t;
                    l[n][e] *= keep;
#pragma unroll
                    for (int i = 0; i < HD / 16; ++i) {
                        o[n][i][e] *= keep;
                        o[n][i][e + 2] *= keep;
                    }
                }
        }
        uint32_t pf[NT][MT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float ref[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) ref[e] = (m[n][e] == -INFINITY ? 0.f : m[n][e]) - kLift;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = exp2_fast(s[n][t][2 * e] - ref[0]), d = exp2_fast(s[n][t][2 * e + 1] - ref[1]);
                    float2 r;
                    uint32_t pair;
                    if constexpr (KV == kBf16) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(a, d);
                        r = __bfloat1622float2(x);
                        pair = *reinterpret_cast<const uint32_t *>(&x);
                    } else {
                        const __half2 x = __floats2half2_rn(a, d);
                        r = __half22float2(x);
                        pair = *reinterpret_cast<const uint32_t *>(&x);
                    }
                    l[n][0] += r.x;
                    l[n][1] += r.y;
                    pf[n][t][e] = transpose8(pair);   // row g; product rows 2c, 2c + 1 (+ 8 e)
                }
        }

        // O^T += V^T P^T
        if constexpr (Q4) {
            const uint32_t at = ring + now * P::STAGE;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                // keys c, c + 4, c + 8, c + 12 of the 16: the product rows 2c, 2c + 1, 2c + 8, 2c + 9
                uint32_t w[4][4], sc[2][P::VB > 8 ? 2 : 1];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 16 * t + 4 * r + c;
                    uint32_t va = at + V_AT + key * P::ROW;
                    if constexpr (HD == 256) va += 16 * (g ^ ((key & 3) << 1));
                    else if constexpr (HD == 128) va += 16 * ((g >> 1) ^ (key & 2)) + 8 * (g & 1);
                    else va += 4 * g;
                    load_shared<P::VB>(va, w[r]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    // scales of the two keys of a pair, for each 16 channels
                    const uint32_t sa = at + VS_AT + (16 * t + 8 * r + c) * P::SROW + g * (HD / 8) / 16;
                    if constexpr (HD == 256) {
                        const uint32_t x = load_shared_u16(sa), y = load_shared_u16(sa + 4 * P::SROW);
                        sc[r][0] = widen_scales(__byte_perm(x, y, 0x40));
                        sc[r][1] = widen_scales(__byte_perm(x, y, 0x51));
                    } else {
                        sc[r][0] = widen_scales(load_shared_u8(sa) | load_shared_u8(sa + 4 * P::SROW) << 8);
                    }
                }
#pragma unroll
                for (int v = 0; v < P::VB / 4; ++v) {
                    // pairs of keys, channels 0 2 4 6 and 1 3 5 7 of the word
                    uint32_t d[2][2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t x = w[2 * r][v], y = w[2 * r + 1][v];
                        widen_e2m1((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), sc[r][v / 2], d[r][0]);
                        widen_e2m1(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), sc[r][v / 2], d[r][1]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma<KV>(o[n][4 * v + e], d[0][0][e], d[0][1][e], d[1][0][e], d[1][1][e], pf[n][t][0],
                                    pf[n][t][1]);
                }
            }
        } else {
            now = advance(ahead);
            issue_v(tile + (P::STAGES - 1) / 2 * kWarps, ahead);
            wait_copies<P::STAGES - 1>();
            __syncwarp();
            const uint32_t at = ring + now * P::STAGE + 16 * (c * 8 + (g ^ (2 * c)));
#pragma unroll
            for (int i = 0; i < P::VP; ++i) {
                uint32_t w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) load_shared<P::VB>(at + (r * P::VP + i) * 32 * P::VB, w[r]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t a0 = __byte_perm(w[0][v], w[1][v], 0x5410), a1 = __byte_perm(w[0][v], w[1][v], 0x7632);
                    const uint32_t a2 = __byte_perm(w[2][v], w[3][v], 0x5410), a3 = __byte_perm(w[2][v], w[3][v], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma<KV>(o[n][4 * i + v], a0, a1, a2, a3, pf[n][0][0], pf[n][0][1]);
                }
            }
        }
    }
    wait_copies<0>();

    // the warps' results: m and l of each row, then O, through shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
            if (g == 0) ml[warp][8 * n + 2 * c + e] = make_float2(m[n][e], l[n][e]);
        }
    __syncthreads();                                 // every warp is done with its ring
    float *staged = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
            // product i: channels ch, ch + 1
            const int ch = Q4 ? g * (HD / 8) + 2 * i : (8 * (i / 4) + g) * 8 + 2 * (i % 4);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2 *>(staged + (warp * ROWS + 8 * n + 2 * c + e) * (HD + 4) + ch) =
                    make_float2(o[n][i][e], o[n][i][e + 2]);
        }
    if (threadIdx.x < ROWS) mend[threadIdx.x] = 0;
    __syncthreads();

    const long long pair = (long long)b * p.nkv + gh;
    auto write_row4 = [&](int r, int ch, float4 x, float sum) {
        // a row that sees keys and has no weight, or any NaN, goes the plain way: what it does not see
        // may have reached it as 0 * NaN
        const int t = r / p.G, h = gh * p.G + r % p.G;
        const Visible v = visible_keys(p, nq, nk, t);
        const bool any = v.hi > v.lo || min(p.sinks, v.lo) > 0;
        const float inv = any ? 1.0f / sum : 0.f;
        x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
        if (!any) x = make_float4(0.f, 0.f, 0.f, 0.f);
        const float all = x.x + x.y + x.z + x.w;
        if (any && !(fabsf(all) <= 3.402823466e38f)) mend[r] = sum == 0.f ? 2 : 1;
        uint2 u;
        if (p.bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), d = __floats2bfloat162_rn(x.z, x.w);
            u = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&d));
        } else {
            const __half2 a = __floats2half2_rn(x.x, x.y), d = __floats2half2_rn(x.z, x.w);
            u = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&d));
        }
        *reinterpret_cast<uint2 *>(static_cast<char *>(p.out.data) +
                                   2 * (b * p.out.batch + t * p.out.token + h * p.out.head + ch)) = u;
    };
    for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
        const int r = i / (HD / 4), ch = 4 * (i % (HD / 4));
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][r].x);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 one = ml[w][r];
            // a warp whose scores were all -inf, or that had no tile, has no weight; its NaN stay
            const float f = one.x == -INFINITY ? (one.y == one.y ? 0.f : one.y) : exp2_fast(one.x - top);
            const float4 y = *reinterpret_cast<const float4 *>(staged + (w * ROWS + r) * (HD + 4) + ch);
            x.x = fmaf(f, y.x, x.x); x.y = fmaf(f, y.y, x.y); x.z = fmaf(f, y.z, x.z); x.w = fmaf(f, y.w, x.w);
            sum = fmaf(f, one.y, sum);
        }
        if (whole_pair) {
            write_row4(r, ch, x, sum);
        } else {
            // a CTA has two unfinished pairs at most: the one its run starts in, the one it ends in
            const long long at = (2ll * blockIdx.x + (unit != unit_begin)) * p.rows_cap + r;
            *reinterpret_cast<float4 *>(p.part_o + at * HD + ch) = x;
            if (ch == 0) p.part_ml[at] = make_float2(top, sum);
        }
    }
    if (!whole_pair) {
        // the runs that hold the pair's units
        const long long u0 = unit - tile0, u1 = u0 + tiles;
        int run0 = blockIdx.x, run1 = blockIdx.x;
        if (u0 < unit_begin) {
            run0 = (int)scaled(u0, runs, units);
            while (scaled(run0 + 1, units, runs) <= u0) ++run0;
        }
        if (u1 > unit_end) {
            run1 = (int)scaled(u1 - 1, runs, units);
            while (scaled(run1 + 1, units, runs) < u1) ++run1;
        }
        const int pieces = run1 - run0 + 1;
        // piece k's place: its run's first, but for a first piece that its run starts before
        const int slot0 = 2 * run0 + (scaled(run0, units, runs) < u0);
        auto slot_of = [&](int k) { return k == 0 ? (long long)slot0 : 2ll * (run0 + k); };
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last_here = atomicAdd(&p.arrived[pair], 1u) == (unsigned)pieces - 1;
        __syncthreads();
        if (last_here) {
            __threadfence();
            if (threadIdx.x == 0) p.arrived[pair] = 0;
            // 4 channels of a row a thread, eight pieces' loads in flight, in the order of the pieces
            for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
                const int r = i / (HD / 4), ch = 4 * (i % (HD / 4));
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                float top = -INFINITY, sum = 0.f;
                for (int k0 = 0; k0 < pieces; k0 += 8) {
                    float2 one[8];
                    float4 y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        one[k] = make_float2(-INFINITY, 0.f);
                        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (k0 + k < pieces) {
                            const long long at = slot_of(k0 + k) * p.rows_cap + r;
                            one[k] = __ldcg(&p.part_ml[at]);
                            y[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + at * HD + ch));
                        }
                    }
                    float next = top;
#pragma unroll
                    for (int k = 0; k < 8; ++k) next = fmaxf(next, one[k].x);
                    const float keep = top == -INFINITY ? (sum == sum ? 0.f : sum) : exp2_fast(top - next);
                    x.x *= keep; x.y *= keep; x.z *= keep; x.w *= keep;
                    sum *= keep;
                    top = next;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // a piece whose scores were all -inf has no weight; its NaN stay
                        const float f = one[k].x == -INFINITY ? (one[k].y == one[k].y ? 0.f : one[k].y)
                                                              : exp2_fast(one[k].x - top);
                        x.x = fmaf(f, y[k].x, x.x); x.y = fmaf(f, y[k].y, x.y);
                        x.z = fmaf(f, y[k].z, x.z); x.w = fmaf(f, y[k].w, x.w);
                        sum = fmaf(f, one[k].y, sum);
                    }
                }
                write_row4(r, ch, x, sum);
            }
        }
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kWarps)
        if (mend[r]) {
            if constexpr (Q4) mend_row_kv4<HD>(p, b, gh, r, nq, nk, 0, rows - 1, mend[r] == 2);
            else attend_row<HD, Q4>(p, b, r / p.G, gh * p.G + r % p.G, nq, nk);
        }
    // on to the next pair of the run
    unit += tile1 - tile0;
    if (unit >= unit_end) break;
    t_first = 0;
    if (++gh == p.nkv) {
        gh = 0;
        do ++b;
        while (tiles_of(b) == 0);
    }
    __syncthreads();                                  // the ring is free again
    }
}

template <int HD, int KV, int NT> cudaError_t prepare()
{
    return cudaFuncSetAttribute(window_few_kernel<HD, KV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_bytes<HD, KV, NT>());
}
template <int HD> cudaError_t prepare_hd()
{
    cudaError_t e = prepare<HD, kF16, 1>();
    if (e == cudaSuccess) e = prepare<HD, kBf16, 1>();
    if (e == cudaSuccess) e = prepare<HD, kKv4, 1>();
    if constexpr (HD < 256)
        if (e == cudaSuccess) e = prepare<HD, kKv4, 2>();
    return e;
}

template <int HD, int KV, int NT> void launch(const WindowParams &p, cudaStream_t s)
{
    window_few_kernel<HD, KV, NT><<<p.chunks, kThreads, smem_bytes<HD, KV, NT>(), s>>>(p);
}
template <int HD> cudaError_t launch_hd(const WindowParams &p, bool kv4, cudaStream_t s)
{
    const bool two = (long long)p.T * p.G > 8;           // 4-bit, hd 64 and 128
    if (!kv4) p.bf16 ? launch<HD, kBf16, 1>(p, s) : launch<HD, kF16, 1>(p, s);
    else if (HD < 256 && two) launch<HD, kKv4, HD < 256 ? 2 : 1>(p, s);
    else launch<HD, kKv4, 1>(p, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_window_few()
{
    for (cudaError_t e : {prepare_hd<64>(), prepare_hd<128>(), prepare_hd<256>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

int few_ctas_per_sm(int hd, bool two, bool kv4)
{
    int n = 0;
    cudaError_t e = cudaErrorInvalidValue;
    auto ask = [&](auto kernel, int smem) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem);
    };
    if (two && kv4 && hd < 256)
        hd == 64 ? ask(window_few_kernel<64, kKv4, 2>, smem_bytes<64, kKv4, 2>())
                 : ask(window_few_kernel<128, kKv4, 2>, smem_bytes<128, kKv4, 2>());
    else if (hd == 64)
        kv4 ? ask(window_few_kernel<64, kKv4, 1>, smem_bytes<64, kKv4, 1>())
            : ask(window_few_kernel<64, kBf16, 1>, smem_bytes<64, kBf16, 1>());
    else if (hd == 128)
        kv4 ? ask(window_few_kernel<128, kKv4, 1>, smem_bytes<128, kKv4, 1>())
            : ask(window_few_kernel<128, kBf16, 1>, smem_bytes<128, kBf16, 1>());
    else if (hd == 256)
        kv4 ? ask(window_few_kernel<256, kKv4, 1>, smem_bytes<256, kKv4, 1>())
            : ask(window_few_kernel<256, kBf16, 1>, smem_bytes<256, kBf16, 1>());
    if (e != cudaSuccess) return 0;
    return n < kFewCtasPerSm ? n : kFewCtasPerSm;
}

cudaError_t launch_window_few(const WindowParams &p, int hd, bool kv4, cudaStream_t s)
{
    switch (hd) {
    case 64: return launch_hd<64>(p, kv4, s);
    case 128: return launch_hd<128>(p, kv4, s);
    case 256: return launch_hd<256>(p, kv4, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dg
