// window_tiles.cuh -- attention with a sliding window and sink tokens for many query rows (prompts,
// canvases) on the tcgen05 tensor cores, over 16-bit or 4-bit keys and values.
//
// Rows R = t * G + h mod G of a kv head are cut into tiles of 128, one TMEM lane and one softmax
// thread a row.  Keys come in tiles of 64: first those of the sinks below the window, then those of the
// window of the block's rows.  Unit u of a CTA is one row tile against one key tile: QK(u) fills score
// buffer u % 2, the softmax turns it into weights in place, PV(u) reads them.  One warp issues
// QK(0) QK(1) | PV(0) QK(2) | PV(1) QK(3) | ...: the softmax of a unit runs beside the products of its
// neighbours, and QK(u + 2) may overwrite the scores whose weights PV(u) reads because the pipe runs in
// order.
//   16-bit, hd 64, 128: two CTAs an SM share its tensor pipe, so that one's set-up and epilogue hide
//             behind the other's loop;
//   4-bit, hd 64, 128: two row tiles share each K and V tile (unpacked once for 256 rows); u % 2 is
//             the row tile;
//   hd 256:   O of one row tile takes half of TMEM.  Two CTAs that share one product of 256 rows
//             (cta_group::2), each with half of every K and V tile, were slower: 170 us where single ones
//             take 139 (4-bit, one partition), since weights and tiles then arrive across the cluster.
// Q is the A operand from TMEM (from shared memory, a 64-key product is bound by reading it: 48 clocks
// an MMA and not 32), but for 16-bit hd 128, whose two CTAs fill TMEM with O and scores.
//
// 16-bit K and V arrive by TMA (any strides); 4-bit ones are turned into f16 tiles by two warpgroups
// (exact: 2 bits times 4 bits), and Q is brought to f16 (bf16 rows by a power of two, what is lost lies
// 2^-25 below the row's largest element).
//
// Softmax: the reference moves when a score passes it by tile_slack(), weights are rounded to V's type
// and summed as rounded.  Key partitions of a row tile, when there are fewer row tiles than SMs, form a
// cluster and merge through distributed shared memory.  A row that ends as NaN is computed again
// the plain way, since 0 * NaN of a key that it does not see may have reached it; V rows behind the
// last visible key are zeroed.
//
// A padded batch of up to 32 sequences is dealt to the clusters by the kernel itself (deal_tiles): every
// CTA reads the lengths, and the sequences with the most tiles split theirs over a cluster while the
// others' row tiles take a CTA each, by the threshold that ends first.  3 canvases of 500 over 4500 keys,
// 72 to 80 row tiles in use: split all or none, 68 and 53 us; dealt 49 us (51.3 by now, with weights from 2^5).
//
// What bounds it: the chain of a unit, not the pipe.  hd 256, 16-bit: a tile's products take 1024 clocks,
// its softmax 960 (the wait for the scores 240, their load and maximum 310, exponentials 360, stores 60)
// and, in about two tiles of five, O's move to another reference 780: 1600 a tile together; 4-bit
// tiles, whose unpacking shares the issue slots, 2000.  Two threads a row halve neither (the exchange of
// their maxima costs what they save), and registers in place of the ring for 4-bit codes change nothing.
// hd 128: the products of two CTAs an SM (640 clocks a tile each, since Q comes from shared memory) hold
// their loops at 1360 clocks a tile; a CTA's start and end, 14 k clocks of 38 k, leave the pipe to the other
// one alone; and there are four rounds of CTAs where 3.4 are full.
// Measured: 8192 tokens of 16 heads of 128, window 1024: 77.5 us (0.83 PFLOP/s); 3 canvases of 500 over
// 4500 keys at hd 256: 51.3 us; 512 over 8704 4-bit keys at hd 256: 51.4 us (0.71 PFLOP/s), of which the
// start takes 13 k clocks of 95 k and the merge 14 k.
#pragma once
#include "sm103_ptx.cuh"
#include "window_rows.cuh"

namespace dg {

struct WindowMaps {
    CUtensorMap k, v;                // [batch][nkv][S][hd], box {64, KT, 1, 1}, 128-byte swizzle
    int k_head, k_seq, v_head, v_seq;   // 1, or 0 where all heads or sequences share their keys (a map of one)
};

namespace {

enum TileKind : int { kTileF16 = 0, kTileBf16 = 1, kTileKv4 = 2 };

template <int HD, int KIND> struct TileCfg {
    static constexpr bool Q4 = KIND == kTileKv4;
    static constexpr int NQT = Q4 && HD < 256 ? 2 : 1;               // row tiles of a CTA
    static constexpr int CTAS = !Q4 && HD < 256 ? 2 : 1;             // CTAs of an SM
    static constexpr bool Q_TMEM = Q4 || HD != 128;                  // Q in TMEM, else in shared memory
    static constexpr int KT = 64;                                    // keys of a tile
    static constexpr int PANELS = HD / 64;
    static constexpr int PANEL_BYTES = KT * 128;
    static constexpr int STAGE = PANELS * PANEL_BYTES;               // K or V tile in 16 bits
    static constexpr int KST = Q4 ? (HD == 256 ? 2 : 4) : HD == 128 ? 2 : 4;
    static constexpr int VST = Q4 ? (HD == 256 ? 2 : 4) : HD == 256 ? 3 : HD == 128 ? 2 : 4;
    static constexpr int Q_BYTES = Q_TMEM ? 0 : 128 * HD * 2;
    // 4-bit tiles on their way, K's and V's: a thread's 16-byte pieces of codes and the words of their scales
    static constexpr int PIECES = Q4 ? KT * HD / 32 / 128 : 0;
    static constexpr int FETCH = PIECES * 128 * 20;
    static constexpr int DEPTH = Q4 ? (HD == 256 ? 4 : HD == 128 ? 6 : 8) : 0;
    static constexpr int K_OFF = Q_BYTES, V_OFF = K_OFF + KST * STAGE, F_OFF = V_OFF + VST * STAGE;
    // merge of a cluster's partitions, in the place of all this: a CTA's own rows from every partition (O,
    // then m and l), weights, rows to mend, output rows; a share rounds up to one row more in each of 8
    // partitions; and 32 x 32 values of each warp on their way to their owners
    static constexpr int SLOTS = NQT * 128 + 8;
    static constexpr int ML_OFF = SLOTS * HD * 4;
    static constexpr int WGT_OFF = ML_OFF + SLOTS * 8;
    static constexpr int SEND_OFF = WGT_OFF + SLOTS * (8 * 4 + 4 + 8), MERGE_END = SEND_OFF + NQT * 4 * 4096;
    static constexpr int F_END = F_OFF + 2 * DEPTH * FETCH, BAR_OFF = F_END > MERGE_END ? F_END : MERGE_END;
    static_assert(SEND_OFF % 16 == 0 && BAR_OFF % 8 == 0, "alignment");
    static constexpr int NBARS = 2 * KST + 2 * VST + 6 + NQT + 1;
    static constexpr int SMEM = BAR_OFF + NBARS * 8 + 32 + 1024;
    static constexpr int CONV = 4 + 4 * NQT;                         // first converting warp (K's; V's 4 on)
    static constexpr int THREADS = 128 * (1 + NQT + (Q4 ? 2 : 0));
    // TMEM columns
    static constexpr int O_COL = 0, Q_COL = NQT * HD, S_COL = Q_COL + (Q_TMEM ? NQT * HD / 2 : 0);
    static constexpr int TMEM = CTAS == 2 ? 256 : 512;
    static_assert(S_COL + 2 * KT <= TMEM, "tensor memory");
    static_assert(!Q_TMEM || VST * STAGE >= NQT * 128 * HD * 2, "Q passes through the V ring");
    static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory");
    // registers of a thread at launch, and of the softmax, converting and other warpgroups: by
    // warpgroup they sum up to the launch's at most
    static constexpr int REGS = THREADS == 256 ? (CTAS == 2 ? 128 : 248) : THREADS == 512 ? 128 : 96;
    static constexpr int SOFT_REGS = THREADS == 256 ? (CTAS == 2 ? 152 : 248) : THREADS == 512 ? 200 : 144;
    static constexpr int CONV_REGS = THREADS == 512 ? 104 : 64;
    static constexpr int REST_REGS = THREADS == 256 ? (CTAS == 2 ? 104 : 248) : THREADS == 512 ? 104 : 64;
    static_assert(SOFT_REGS * NQT + (Q4 ? 2 * CONV_REGS : 0) + REST_REGS <= REGS * (THREADS / 128), "register pool");
};

// A row's reference is set so that its largest weight so far is 2^tile_lift(), and stays until a weight
// would pass 2^tile_slack().  f16 weights, over f16 or 4-bit V, reach from 2^15 down to steps of 2^-24: with
// the largest at 2^-6, keys 13 nats under a leading one (a sink token's lead) weighed nothing, and 8192 of
// those were half of a result.  From 2^5 on a small weight is off by 2^-30 of the largest, as in the
// few-row kernel.  The price: O moves in more tiles where scores spread by tens of log2 units (scale 1 at
// hd 256, partitions of 34 tiles: in 14 of them, 5 with the largest at 2^-6; simulated).  us with lifts of
// -6, 0, 3, 5 and 8: 3 f16 canvases 47.6, 49.6, 51.2, 51.3, 52.6, the 4-bit one 48, 50.4, 51.2, 51.4, 53.2.
// bf16 weights have exponents to spare on both sides.
template <int KIND> constexpr float tile_lift() { return KIND == kTileBf16 ? -6.0f : 5.0f; }
template <int KIND> constexpr float tile_slack() { return KIND == kTileBf16 ? 60.0f : 15.0f; }

__device__ __forceinline__ void fence_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int x, int y, int z, int w)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// l += the two bf16 values of h2, each widened exactly
__device__ __forceinline__ void add_bf16x2_to_f32x2(float2 &l, uint32_t h2)
{
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(l.x), "+f"(l.y) : "r"(h2));
}
template <int N> __device__ __forceinline__ void set_max_registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void set_max_registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Stores into a CTA of the cluster (addresses from dsmem_map).
__device__ __forceinline__ void dsmem_st_f2(uint32_t addr, float x, float y)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void dsmem_st_u4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Byte offset of 16-byte unit `unit` (0 .. HD/8 - 1) of row `row` in a tile of 64-element panels with
// the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int row, int unit, int panel_bytes)
{
    return (uint32_t)((unit >> 3) * panel_bytes + row * 128 + (((unit & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight e2m1 values (one word) times a scale pair, as one 16-byte unit of f16.
__device__ __forceinline__ uint4 widen_unit(uint32_t w, uint32_t scale2)
{
    uint32_t d[4];
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
    return make_uint4(d[0], d[1], d[2], d[3]);
}

// One CTA's share of a padded batch: sequence, kv head, row tile and partitions of its keys; false: none.
// For a warp, a lane a sequence; row tiles are of `block` rows, all CTAs of a cluster get the same `parts`.
struct Deal {
    int b, g, tile, parts;
};
__device__ __forceinline__ bool deal_tiles(const WindowParams &p, int block, int kt, Deal &deal)
{
    const int lane = threadIdx.x & 31, P = p.chunks, cluster = blockIdx.x / P, rank = blockIdx.x % P;
    int mine = 0, tiles = 0, blocks = 0;                 // row tiles of the sequence, key tiles of its last one
    if (lane < p.batch) {
        const int nq = query_count(p, lane), nk = key_count(p, lane), rows = nq * p.G;
        blocks = (rows + block - 1) / block;
        mine = blocks * p.nkv;
        if (rows) {
            const int lo = visible_keys(p, nq, nk, (blocks - 1) * block / p.G).lo, hi = visible_keys(p, nq, nk, nq - 1).hi;
            tiles = (min(p.sinks, lo) + kt - 1) / kt + (hi - lo + kt - 1) / kt;
        }
    }
    // the time if the sequences with as many tiles as this lane's, and more, are split; a lane without a
    // sequence: if none are
    const int from = mine ? tiles : 0x7fffffff;
    int whole = 0, split = 0, most_whole = 0, most_split = 0;
    for (int j = 0; j < p.batch; ++j) {
        const int n = __shfl_sync(0xffffffffu, mine, j), t = __shfl_sync(0xffffffffu, tiles, j);
        if (t >= from) {
            split += n;
            most_split = max(most_split, n ? t : 0);
        } else {
            whole += n;
            most_whole = max(most_whole, n ? t : 0);
        }
    }
    auto time = [&](int split_, int whole_, int most_split_, int most_whole_) {
        const int waves = (split_ + (whole_ + P - 1) / P + p.cluster_slots - 1) / p.cluster_slots;
        const float one = split_ ? (most_split_ + P - 1) / P * p.tile_clocks + p.merge_clocks : 0.f;
        return waves * (8000.f + fmaxf(one, most_whole_ * p.tile_clocks));
    };
    const float clocks = time(split, whole, most_split, most_whole);
    const float none = time(0, split + whole, 0, max(most_split, most_whole));
    float least = clocks;
#pragma unroll
    for (int d = 16; d; d >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
    const unsigned at = __ballot_sync(0xffffffffu, clocks == least);
    const int threshold = none <= least ? 0x7fffffff : __shfl_sync(0xffffffffu, from, __ffs(at) - 1);
    const bool splits = tiles >= threshold;
    // sequences in their order, the split ones' row tiles first
    int before_split = splits ? mine : 0, before_whole = splits ? 0 : mine;
    const int own_split = before_split, own_whole = before_whole;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before_split, d), y = __shfl_up_sync(0xffffffffu, before_whole, d);
        if (lane >= d) { before_split += x; before_whole += y; }
    }
    const int all_split = __shfl_sync(0xffffffffu, before_split, 31);
    before_split -= own_split;
    before_whole -= own_whole;
    const bool by_split = cluster < all_split;
    const int index = by_split ? cluster : (cluster - all_split) * P + rank;
    const int first = by_split ? before_split : before_whole, n = by_split ? own_split : own_whole;
    const unsigned here = __ballot_sync(0xffffffffu, index >= first && index < first + n);
    if (!here) return false;
    deal.b = __ffs(here) - 1;
    const int in = index - __shfl_sync(0xffffffffu, first, deal.b), of = __shfl_sync(0xffffffffu, blocks, deal.b);
    deal.g = in / of;
    deal.tile = in - deal.g * of;
    deal.parts = by_split ? P : 1;
    return true;
}

template <int HD, int KIND, bool DEAL>
__global__ void __launch_bounds__(TileCfg<HD, KIND>::THREADS, TileCfg<HD, KIND>::CTAS)
window_tiles_kernel(const __grid_constant__ WindowMaps maps, const __grid_constant__ WindowParams p)
{
    using C = TileCfg<HD, KIND>;
    constexpr bool Q4 = C::Q4;
    constexpr int NQT = C::NQT, KT = C::KT, KST = C::KST, VST = C::VST;
    // unit u = i * NQT + q uses score buffer u % 2, in the buffer's use u / 2
    constexpr uint32_t fmt = KIND == kTileBf16 ? 1 : 0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *k_empty = k_full + KST, *v_full = k_empty + KST, *v_empty = v_full + VST;
    uint64_t *s_full = v_empty + VST, *p_full = s_full + 2, *pv_done = p_full + 2;
    uint64_t *q_ready = pv_done + 2, *drain = q_ready + NQT;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns;

    // the block's rows, the keys that some row of them sees, and its share of their tiles
    // (dealt ones lie in shared memory: held in registers through the loops they spill)
    int *const given = reinterpret_cast<int *>(tmem_slot) + 1;
    auto given_at = [&](int i) {
        int v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(smem_u32(given + i)));
        return v;
    };
    if constexpr (DEAL) {
        if (warp == 0) {
            Deal deal = {0, 0, 0, 0};
            deal_tiles(p, NQT * 128, KT, deal);
            if (lane == 0) {
                given[0] = deal.b; given[1] = deal.g; given[2] = deal.tile; given[3] = deal.parts;
            }
        }
        __syncthreads();
        if (given_at(3) == 0) return;                    // a cluster with other CTAs at work has no barriers
    }
    const int own_b = DEAL ? 0 : blockIdx.y / p.nkv, own_g = DEAL ? 0 : blockIdx.y % p.nkv;
    auto sequence = [&]() { return DEAL ? given_at(0) : own_b; };
    auto kv_head = [&]() { return DEAL ? given_at(1) : own_g; };
    auto partitions = [&]() { return DEAL ? given_at(3) : p.chunks; };
    const int all_parts = partitions(), part = !DEAL ? blockIdx.z : all_parts > 1 ? cluster_ctarank() : 0;
    const int nq = query_count(p, sequence()), nk = key_count(p, sequence());
    const int rows = nq * p.G, row0 = (DEAL ? given_at(2) : (int)blockIdx.x) * (NQT * 128);
    if (row0 >= rows) return;                            // the whole cluster
    const int row1 = min(rows, row0 + NQT * 128) - 1;
    const Visible first = visible_keys(p, nq, nk, row0 / p.G), final = visible_keys(p, nq, nk, row1 / p.G);
    const int lo = first.lo, hi = final.hi, lo_all = final.lo, hi_all = first.hi;
    const int sk = min(p.sinks, lo);
    const int sink_tiles = (sk + KT - 1) / KT, tiles = sink_tiles + (hi - lo + KT - 1) / KT;
    // tiles < 2^24 (lengths up to 2^28) and parts <= 8: 32 bits are enough
    const int t0 = all_parts == 1 ? 0 : (unsigned)part * tiles / (unsigned)all_parts;
    const int n = (all_parts == 1 ? tiles : (unsigned)(part + 1) * tiles / (unsigned)all_parts) - t0;    // may be 0
    auto tile_start = [&](int i) { return t0 + i < sink_tiles ? (t0 + i) * KT : lo + (t0 + i - sink_tiles) * KT; };
    auto tile_end = [&](int i) { return t0 + i < sink_tiles ? sk : hi; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < KST; ++i) { mbar_init(&k_full[i], Q4 ? 128 : 1); mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < VST; ++i) { mbar_init(&v_full[i], Q4 ? 128 : 1); mbar_init(&v_empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < NQT; ++i) mbar_init(&q_ready[i], 4);
        mbar_init(drain, 1);
        fence_mbar_init();
        if (!Q4 && n > 0) { prefetch_tmap(&maps.k); prefetch_tmap(&maps.v); }      // S = 0: there are none
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp < 4) {
        if constexpr (C::REST_REGS < C::REGS) set_max_registers_down<C::REST_REGS>();
        if (!Q4 && (warp == 0 || warp == 2)) {
            // ------------------------------------------------------------ TMA of K (warp 0), V (warp 2)
            if (lane == 0) {
                const int stages = warp == 0 ? KST : VST;
                uint64_t *full = warp == 0 ? k_full : v_full, *empty = warp == 0 ? k_empty : v_empty;
                const CUtensorMap *map = warp == 0 ? &maps.k : &maps.v;
                uint8_t *ring = smem + (warp == 0 ? C::K_OFF : C::V_OFF);
                const int b = sequence() * (warp == 0 ? maps.k_seq : maps.v_seq);
                const int g = kv_head() * (warp == 0 ? maps.k_head : maps.v_head);
                bool ok = true;
                int issued = 0;
                // the V ring holds Q on its way into TMEM
                if (C::Q_TMEM && warp == 2 && n > 0) ok = mbar_wait_bounded(&q_ready[0], 0, limit);
                for (int i = 0; ok && i < n; ++i) {
                    const int s = i % stages;
                    if (i >= stages && !mbar_wait_bounded(&empty[s], ((i / stages) - 1) & 1, limit)) {
                        ok = false;
                        break;
                    }
                    // Q comes ahead of all but the first K tile
                    if (C::Q_TMEM && warp == 0 && i == 1 && !mbar_wait_bounded(&q_ready[0], 0, limit)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], C::STAGE);
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        tma_load_4d(ring + s * C::STAGE + pn * C::PANEL_BYTES, map, &full[s], pn * 64, tile_start(i), g,
                                    b);
                    issued = i + 1;
                }
                if (!ok) atomicOr(p.status, 1u);
                // every load has landed before the CTA can exit
                for (int i = max(0, issued - stages); i < issued; ++i)
                    mbar_wait_bounded(&full[i % stages], (i / stages) & 1, limit);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            const uint32_t leader = elect_one_sync();
            constexpr uint32_t idesc_qk = make_idesc(fmt, 0, 0, 128, KT);
            constexpr uint32_t idesc_pv = make_idesc(fmt, 0, 1, 128, HD);
            const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + C::K_OFF), 16, 1024);
            const uint64_t vdesc = smem_desc_sw128(smem_u32(smem + C::V_OFF), C::PANEL_BYTES, 1024);
            const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
            // The tile counts go through lane 0, which makes them, and with them stages and descriptors,
            // warp-uniform values for the compiler: with the counts as plain loaded values, eight MMAs took
            // 700 clocks to issue and 512 to run.
            const int un = __shfl_sync(0xffffffffu, n, 0);
            const int usink = __shfl_sync(0xffffffffu, sink_tiles - t0, 0);      // the first tile of the window
            const int last_valid = __shfl_sync(0xffffffffu, n > 0 ? min(KT, tile_end(n - 1) - tile_start(n - 1)) : KT, 0);
            const int sink_valid = __shfl_sync(0xffffffffu, sk - (sink_tiles - 1) * KT, 0);
            const uint32_t ubase = __shfl_sync(0xffffffffu, tbase, 0);
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit));
                tc_fence_after();
                return ok;
            };
            int ks = 0, kphase = 0, vs = 0, vphase = 0;
            // scores of the K tile of stage ks for row tile q into buffer buf
            auto issue_qk = [&](int q, int buf) {
                const uint32_t d = ubase + C::S_COL + buf * KT;
                const uint64_t kd = kdesc + (uint64_t)((ks * C::STAGE) >> 4);
                const uint64_t qd = qdesc + (uint64_t)((q * (128 * HD * 2)) >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const int pn = kk >> 2, sub = kk & 3;
                    const uint64_t kb = kd + (uint64_t)((pn * C::PANEL_BYTES + sub * 32) >> 4);
                    if constexpr (C::Q_TMEM)
                        mma_bf16_ts_by(leader, d, ubase + C::Q_COL + q * (HD / 2) + kk * 8, kb, idesc_qk, kk > 0);
                    else
                        mma_bf16_ss_by(leader, d, qd + (uint64_t)((pn * (128 * 128) + sub * 32) >> 4), kb, idesc_qk,
                                       kk > 0);
                }
                if (q == NQT - 1) mma_commit_by(leader, &k_empty[ks]);
                mma_commit_by(leader, &s_full[buf]);
            };
            auto issue_pv = [&](int q, int buf, int i, int valid) {
                const uint32_t d = ubase + C::O_COL + q * HD, a = ubase + C::S_COL + buf * KT;
                const uint64_t vd = vdesc + (uint64_t)((vs * C::STAGE) >> 4);
                if (valid == KT) {
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        mma_bf16_ts_by(leader, d, a + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                                       i > 0 || kk > 0);
                } else {
                    // the last tile of a range: MMAs of 16 keys up to its end
#pragma unroll 1
                    for (int kk = 0; 16 * kk < valid; ++kk)
                        mma_bf16_ts_by(leader, d, a + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                                       i > 0 || kk > 0);
                }
                if (q == NQT - 1) mma_commit_by(leader, &v_empty[vs]);
                mma_commit_by(leader, &pv_done[buf]);
            };
            if (un > 0) {
                // the scores of the first units, one a buffer
                ok = wait(&q_ready[0], 0) && wait(&k_full[0], 0);
                if (ok) issue_qk(0, 0);
                if (NQT == 2) {
                    if (ok && wait(&q_ready[NQT - 1], 0)) issue_qk(1, 1);
                } else if (un > 1) {
                    ks = 1;
                    if (ok && wait(&k_full[1 % KST], 0)) issue_qk(0, 1);
                }
                if (++ks == KST) { ks = 0; kphase = 1; }
                auto valid_of = [&](int i) { return i == un - 1 ? last_valid : i + 1 == usink ? sink_valid : KT; };
                // V of tile i is there, and its rows behind the last visible key, up to the MMA's 16, are zeros
                auto take_v = [&](int i, bool there) {
                    if (!there && !wait(&v_full[vs], vphase)) return;
                    const int valid = valid_of(i);
                    if (!Q4 && (valid & 15)) {
                        for (int j = lane; j < (16 - (valid & 15)) * (HD / 8); j += 32)
                            *reinterpret_cast<uint4 *>(smem + C::V_OFF + vs * C::STAGE +
                                                       swizzled(valid + j / (HD / 8), j % (HD / 8), C::PANEL_BYTES)) =
                                make_uint4(0, 0, 0, 0);
                        fence_async_shared();
                        __syncwarp();
                    }
                };
                if (ok) take_v(0, false);
                for (int i = 0; ok && i < un; ++i) {
                    const bool again = i + 2 / NQT < un;
#pragma unroll
                    for (int q = 0; q < NQT; ++q) {
                        const int u = i * NQT + q, buf = u % 2;
                        if (!ok || !wait(&p_full[buf], (u / 2) & 1)) break;
                        issue_pv(q, buf, i, valid_of(i));
                        // the pipe holds the product just issued while this warp waits (a wait on a barrier
                        // that is already complete takes ~150 clocks)
                        if (q == NQT - 1) {
                            if (++vs == VST) { vs = 0; vphase ^= 1; }
                            // both asked for at once: each answer takes ~150 clocks
                            const bool k_there = NQT == 1 && again && mbar_test(&k_full[ks], kphase);
                            const bool v_there = i + 1 < un && mbar_test(&v_full[vs], vphase);
                            const bool both = __all_sync(0xffffffffu, k_there && v_there);
                            if (both) tc_fence_after();
                            if (NQT == 1 && again && !both) ok = wait(&k_full[ks], kphase);
                            if (ok && i + 1 < un) take_v(i + 1, both);
                        } else if (again) {
                            ok = wait(&k_full[ks], kphase);
                        }
                        if (ok && again) issue_qk(q, buf);
                    }
                    if (++ks == KST) { ks = 0; kphase ^= 1; }
                }
            }
            if (!ok && leader) atomicOr(p.status, 2u);
            // no tcgen05 operation of this warp still runs when TMEM is released
            mma_commit_by(leader, drain);
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(drain, 0, limit)) && leader) atomicOr(p.status, 8u);
            __syncwarp();
        }
    } else if (warp < 4 + 4 * NQT) {
        // ---------------------------------------------------------------- softmax
        if constexpr (C::SOFT_REGS > C::REGS) set_max_registers_up<C::SOFT_REGS>();
        const int q = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;                       // row of the tile, TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const int row = row0 + q * 128 + r;
        const bool mine = row < rows;
        const int t = (mine ? row : row1) / p.G;
        const Visible see = visible_keys(p, nq, nk, t);
        // scores enter as s * zs; a negative scale goes into Q
        float zs = fabsf(p.scale) * 1.4426950408889634f;

        // Q into shared memory, or through the V ring's place into TMEM (a thread its row), in short loops: the
        // code of this phase runs once and comes from L2, 32 unrolled loads of it took 13 k clocks.  A warp
        // copies whole rows, LPR lanes each: with a row a thread, 32 lines a load, it took 5 k.
        auto row_of_out = [&]() {
            return static_cast<char *>(p.out.data) +
                   2 * (sequence() * p.out.batch + t * p.out.token + (kv_head() * p.G + (mine ? row % p.G : 0)) * p.out.head);
        };
        char *const early = DEAL ? nullptr : row_of_out();
        auto out_row = [&]() { return DEAL ? row_of_out() : early; };
        constexpr int LPR = HD / 8, RPI = 32 / LPR;              // lanes of a row, rows of a load
        // (a partition without keys leaves Q: nothing would hold its merge data back until every warp had
        // staged its rows in the same place)
        if (n > 0) {
            const int h = kv_head() * p.G + (mine ? row % p.G : 0);
            const char *own = static_cast<const char *>(p.q.data) +
                              2 * (sequence() * p.q.batch + t * p.q.token + h * p.q.head);
            const unsigned long long at = mine ? reinterpret_cast<unsigned long long>(own) : 0;
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
            uint8_t *const stage = C::Q_TMEM ? smem + C::V_OFF + (q * 128 + quarter * 32) * (HD * 2) : smem;
#pragma unroll 4
            for (int j = 0; j < HD / 8; ++j) {
                const int rr = j * RPI + lane / LPR, unit = lane % LPR;
                const unsigned long long src = __shfl_sync(0xffffffffu, at, rr);
                uint8_t *const dst = C::Q_TMEM ? stage + rr * (HD * 2) + ((unit ^ (rr & 7)) << 4)
                                               : stage + swizzled(quarter * 32 + rr, unit, 128 * 128);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
                             "l"(src ? src + 16 * unit : reinterpret_cast<unsigned long long>(p.q.data)),
                             "r"(src ? 16 : 0) : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            // the row's unit v
            auto unit_of = [&](int v) {
                return reinterpret_cast<uint4 *>(C::Q_TMEM ? stage + lane * (HD * 2) + ((v ^ (lane & 7)) << 4)
                                                           : stage + swizzled(r, v, 128 * 128));
            };
            // bf16 into f16 by a power of two that brings the row's largest element to [1, 2)
            int ex = 0;
            if (Q4 && p.bf16) {
                float top = 0.f;
#pragma unroll 4
                for (int v = 0; v < HD / 8; ++v) {
                    const uint4 x = *unit_of(v);
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = fmax3(top, fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u)));
                }
                if (top > 0.f && top <= 3.402823466e38f) ex = ilogbf(top);
            }
            const float up = exp2f((float)(-ex / 2)), down = exp2f((float)(-ex - -ex / 2));
            // the smallest normal at the least: a masked score stays -inf, and scale 0 gives finite scores no weight
            zs = fmaxf(ldexpf(zs, ex), 1.17549435e-38f);
            if constexpr (C::Q_TMEM) {
#pragma unroll 1
                for (int v0 = 0; v0 < HD / 8; v0 += 8) {
                    uint32_t u[32];
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint4 x = *unit_of(v0 + v);
                        u[4 * v] = x.x ^ flip; u[4 * v + 1] = x.y ^ flip; u[4 * v + 2] = x.z ^ flip; u[4 * v + 3] = x.w ^ flip;
                    }
                    if (Q4 && p.bf16)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            u[e] = pack_half2(__uint_as_float(u[e] << 16) * up * down,
                                              __uint_as_float(u[e] & 0xffff0000u) * up * down);
                    tmem_st32(tbase + lane_off + C::Q_COL + q * (HD / 2) + v0 * 4, u);
                }
                tmem_wait_st();
                tc_fence_before();
            } else if (flip) {
#pragma unroll 1
                for (int v = 0; v < HD / 8; ++v) {
                    uint4 x = *unit_of(v);
                    x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
                    *unit_of(v) = x;
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[q]);
        }

        bool ok = true;
        float m = -INFINITY, best = -INFINITY;                   // the reference, the largest score so far
        float2 l2 = make_float2(0.f, 0.f);
        for (int i = 0; i < n; ++i) {
            const int u = i * NQT + q, buf = u % 2;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[buf], (u / 2) & 1, limit));
            if (!ok) break;
            tc_fence_after();
            const uint32_t ts = tbase + lane_off + C::S_COL + buf * KT;
            uint32_t sr[KT / 32][32];
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) tmem_ld32(ts + 32 * c, sr[c]);
            tmem_wait_ld();
            const int k0 = tile_start(i), end = tile_end(i);
            const bool sink = t0 + i < sink_tiles;
            const bool whole = sink ? k0 + KT <= min(sk, hi_all) : (k0 >= lo_all && k0 + KT <= min(hi, hi_all));
            if (!whole) {
                const int c_hi = min(see.hi, end) - k0, c_lo = see.lo - k0, c_sk = p.sinks - k0;
#pragma unroll
                for (int c = 0; c < KT / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int x = 32 * c + e;
                        if (!(x < c_hi && (x >= c_lo || x < c_sk))) sr[c][e] = __float_as_uint(-INFINITY);
                    }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < KT / 32; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
            float top = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * zs;
            float keep = 1.0f;
            bool rescale = false;
            if (KIND != kTileBf16 && NQT == 1 && i == 0 && n > 1) {
                // the first reference looks at the second tile too (its scores are there already)
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[1], 0, limit));
                if (!ok) break;
                tc_fence_after();
                const int k1 = tile_start(1), c_hi = min(see.hi, tile_end(1)) - k1, c_lo = see.lo - k1, c_sk = p.sinks - k1;
                float m1 = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < KT / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tbase + lane_off + C::S_COL + KT + 32 * c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int col = 32 * c + e;
                        if (col < c_hi && (col >= c_lo || col < c_sk)) m1 = fmaxf(m1, __uint_as_float(x[e]));
                    }
                }
                top = fmaxf(top, m1 * zs);
            }
            best = fmaxf(best, top);
            if (__any_sync(0xffffffffu, top > m + tile_slack<KIND>())) {
                // every row of the warp moves to its largest score so far: scaling O costs the warp the same
                const float m_new = fmaxf(m, best - tile_lift<KIND>());
                keep = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
                l2 = mul_f32x2(l2, make_float2(keep, keep));
                m = m_new;
                rescale = i > 0;
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const float2 zz = make_float2(zs, zs), rr = make_float2(-ref, -ref);
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
                uint32_t pw[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 z = fma_f32x2(
                        make_float2(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), zz, rr);
                    const float a = ex2_approx(z.x), d = ex2_approx(z.y);
                    if constexpr (KIND == kTileBf16) {
                        pw[e] = pack_bf162(a, d);
                        add_bf16x2_to_f32x2(l2, pw[e]);
                    } else {
                        pw[e] = pack_half2(a, d);
                        add_f16x2_to_f32x2(l2, pw[e]);
                    }
                }
                tmem_st16(ts + 16 * c, pw);
            }
            tmem_wait_st();
            if (rescale) {
                // O moves to the new reference once the product before has landed
                const int pu = u - NQT;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&pv_done[pu % 2], (pu / 2) & 1, limit));
                if (!ok) break;
                tc_fence_after();
                const float2 kk = make_float2(keep, keep);
                const uint32_t to = tbase + lane_off + C::O_COL + (NQT == 2 ? q * HD : 0);
                constexpr int W = HD == 256 ? 4 : 2;             // 32-column chunks in flight
#pragma unroll 1
                for (int c = 0; c < HD / 32; c += W) {
                    uint32_t o[W][32];
#pragma unroll
                    for (int w = 0; w < W; ++w) tmem_ld32(to + 32 * (c + w), o[w]);
                    tmem_wait_ld();
#pragma unroll
                    for (int w = 0; w < W; ++w) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 x = mul_f32x2(
                                make_float2(__uint_as_float(o[w][e]), __uint_as_float(o[w][e + 1])), kk);
                            o[w][e] = __float_as_uint(x.x);
                            o[w][e + 1] = __float_as_uint(x.y);
                        }
                        tmem_st32(to + 32 * (c + w), o[w]);
                    }
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        // the row tile's last product, and the other's: nothing reads Q, K or V any more
        if (ok && n > 0) {
            for (int u = max(0, n * NQT - 2); u < n * NQT; ++u)
                ok = ok && mbar_wait_bounded(&pv_done[u % 2], (u / 2) & 1, limit);
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok && lane == 0) atomicOr(p.status, 4u);
        tc_fence_after();
        const float sum = l2.x + l2.y;
        const uint32_t to = tbase + lane_off + C::O_COL + (NQT == 2 ? q * HD : 0);
        uint32_t sent = 0;
        const int b = sequence(), g = kv_head(), parts = partitions();
        if (parts > 1) {
            // CTA k of the cluster owns the rows [k total / parts, (k + 1) total / parts).  Every partition
            // writes its rows into their owners' shared memory (reading them there instead waits a round trip
            // for each), once all CTAs are through their products.
            __syncwarp();
            cluster_sync_all();
            const int total = min(rows - row0, NQT * 128), rank = (int)cluster_ctarank();
            const int mr = q * 128 + r, most = (total + parts - 1) / parts;
            if (mr < total) {
                int owner = mr * parts / total;
                while ((owner + 1) * total / parts <= mr) ++owner;
                const int slot = rank * most + mr - owner * total / parts;      // < parts * most
                const uint32_t there = dsmem_map(smem_u32(smem), owner);
                dsmem_st_f2(there + C::ML_OFF + slot * 8, m, sum);
                sent = there + slot * HD * 4;
            }
            // 32 channels at a time through the warp's corner of shared memory, so that eight lanes write 128
            // bytes of a row: a row a lane, in 16-byte stores, took 10 k clocks at hd 256
            uint8_t *const corner = smem + C::SEND_OFF + (warp - 4) * 4096;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                uint32_t o[32] = {};
                if (n > 0) {
                    tmem_ld32(to + 32 * c, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    *reinterpret_cast<uint4 *>(corner + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                        make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int rr = 4 * j + lane / 8;
                    const uint32_t row_there = __shfl_sync(0xffffffffu, sent, rr);
                    const uint4 x = *reinterpret_cast<const uint4 *>(corner + rr * 128 + (((lane ^ rr) & 7) << 4));
                    if (row_there) dsmem_st_u4(row_there + (32 * c + 4 * (lane & 7)) * 4, x.x, x.y, x.z, x.w);
                }
                __syncwarp();
            }
        } else if (ok) {
            const bool any = see.hi > see.lo || min(p.sinks, see.lo) > 0;
            const float inv = any ? 1.0f / sum : 0.f;
            // rows in 16 bits through shared memory, each warp its own 32 (Q's place, or the K ring's at hd
            // 256), so that a warp writes whole rows
            uint8_t *stage = smem + q * (128 * HD * 2);
            float2 odd = make_float2(0.f, 0.f);                  // 0, or NaN once a value is not finite
#pragma unroll 1
            for (int c = 0; c < HD / 32; c += 2) {
                uint32_t o[2][32] = {};
                if (n > 0) {
                    tmem_ld32(to + 32 * c, o[0]);
                    tmem_ld32(to + 32 * c + 32, o[1]);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = mul_f32x2(
                            make_float2(__uint_as_float(o[x][2 * e]), __uint_as_float(o[x][2 * e + 1])), make_float2(inv, inv));
                        odd = fma_f32x2(y, make_float2(0.f, 0.f), odd);
                        w[e] = !any ? 0 : p.bf16 ? pack_bf162(y.x, y.y) : pack_half2(y.x, y.y);
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint4 *>(stage + swizzled(r, 4 * (c + x) + v, 128 * 128)) =
                            make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                }
            }
            const bool bad = any && (!(sum > 0.f) || !(odd.x + odd.y == 0.f));
            __syncwarp();
            const unsigned long long at = mine ? reinterpret_cast<unsigned long long>(out_row()) : 0;
#pragma unroll 4
            for (int j = 0; j < 32; j += RPI) {
                const int rr = j + lane / LPR, unit = lane % LPR;
                char *dst = reinterpret_cast<char *>(__shfl_sync(0xffffffffu, at, rr));
                const uint4 x = *reinterpret_cast<const uint4 *>(stage + swizzled(quarter * 32 + rr, unit, 128 * 128));
                if (dst) *reinterpret_cast<uint4 *>(dst + 16 * unit) = x;
            }
            __syncwarp();
            const unsigned empty = Q4 ? __ballot_sync(0xffffffffu, sum == 0.f) : 0;
            for (unsigned again = __ballot_sync(0xffffffffu, bad && mine); again; again &= again - 1) {
                const int at = __ffs(again) - 1, orow = row0 + q * 128 + quarter * 32 + at;
                if constexpr (Q4) mend_row_kv4<HD>(p, b, g, orow, nq, nk, row0, row0 + NQT * 128 - 1, empty >> at & 1);
                else attend_row<HD, Q4>(p, b, orow / p.G, g * p.G + orow % p.G, nq, nk);
            }
        }
        if (parts > 1) {
            // every owner has its rows' partitions, and merges them in their order
            __syncwarp();
            cluster_sync_all();
            constexpr int NT = 128 * NQT, V4 = HD / 4;
            const int tid = threadIdx.x - 128;
            const int total = min(rows - row0, NQT * 128), rank = (int)cluster_ctarank();
            const int most = (total + parts - 1) / parts, r0 = rank * total / parts;
            const int nr = (rank + 1) * total / parts - r0;
            const float2 *ml = reinterpret_cast<const float2 *>(smem + C::ML_OFF);
            float *wgt = reinterpret_cast<float *>(smem + C::WGT_OFF);
            int *mend = reinterpret_cast<int *>(wgt + 8 * C::SLOTS);
            char **dst = reinterpret_cast<char **>(mend + C::SLOTS);
            if (tid < nr) {
                const int orow = row0 + r0 + tid, ot = orow / p.G, oh = g * p.G + orow % p.G;
                float mm[8], top = -INFINITY, total_l = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    mm[k] = k < parts ? ml[k * most + tid].x : -INFINITY;
                    top = fmaxf(top, mm[k]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < parts) {
                        const float l = ml[k * most + tid].y;
                        mm[k] = mm[k] == -INFINITY ? (l == l ? 0.f : l) : ex2_approx(mm[k] - top);
                        total_l = fmaf(mm[k], l, total_l);
                    }
                const Visible v = visible_keys(p, nq, nk, ot);
                const bool any = v.hi > v.lo || min(p.sinks, v.lo) > 0;
                const float inv = any ? 1.0f / total_l : 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < parts) wgt[tid * 8 + k] = any ? mm[k] * inv : 0.f;
                mend[tid] = Q4 && any && total_l == 0.f ? 2 : 0;       // scores of -inf alone
                dst[tid] = static_cast<char *>(p.out.data) + 2 * (b * p.out.batch + ot * p.out.token + oh * p.out.head);
            }
            named_barrier_sync(1, NT);
            // 4 channels of a row an item, four items of a thread at once
            constexpr int U = 4, STEP = NT / V4;                 // rows between a thread's items
            const int ch = 4 * (tid % V4);
            for (int i0 = tid / V4; i0 < nr; i0 += U * STEP) {
                float4 x[U] = {};
                for (int k = 0; k < parts; ++k) {
                    const uint8_t *src = smem + ((k * most + i0) * HD + ch) * 4;
#pragma unroll
                    for (int v = 0; v < U; ++v) {
                        const int i = i0 + v * STEP;
                        if (i < nr) {
                            const float4 y = *reinterpret_cast<const float4 *>(src + v * STEP * HD * 4);
                            const float f = wgt[i * 8 + k];
                            x[v].x = fmaf(f, y.x, x[v].x); x[v].y = fmaf(f, y.y, x[v].y);
                            x[v].z = fmaf(f, y.z, x[v].z); x[v].w = fmaf(f, y.w, x[v].w);
                        }
                    }
                }
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    const int i = i0 + v * STEP;
                    if (i >= nr) continue;
                    if (!(fabsf(x[v].x) + fabsf(x[v].y) + fabsf(x[v].z) + fabsf(x[v].w) <= 3.402823466e38f) &&
                        (!Q4 || !mend[i]))
                        mend[i] = 1;
                    *reinterpret_cast<uint2 *>(dst[i] + 2 * ch) =
                        p.bf16 ? make_uint2(pack_bf162(x[v].x, x[v].y), pack_bf162(x[v].z, x[v].w))
                               : make_uint2(pack_half2(x[v].x, x[v].y), pack_half2(x[v].z, x[v].w));
                }
            }
            named_barrier_sync(1, NT);
            for (int i = warp - 4; i < nr; i += 4 * NQT)
                if (mend[i]) {
                    const int orow = row0 + r0 + i;
                    if constexpr (Q4) mend_row_kv4<HD>(p, b, g, orow, nq, nk, row0, row0 + NQT * 128 - 1, mend[i] == 2);
                    else attend_row<HD, Q4>(p, b, orow / p.G, g * p.G + orow % p.G, nq, nk);
                }
        }
    } else if constexpr (Q4) {
        // ---------------------------------------------------------------- 4-bit tiles into f16 ones
        // One warpgroup turns the K tiles, one the V tiles.  Codes and scales come through a ring of DEPTH
        // tiles in shared memory that each thread fills (cp.async) and reads for itself.
        if constexpr (C::CONV_REGS < C::REGS) set_max_registers_down<C::CONV_REGS>();
        const bool isv = warp >= C::CONV + 4;
        const int w = threadIdx.x & 127;
        constexpr int CPR = HD / 32, STEP = 128 / CPR;           // 16-byte pieces of a row, rows between a thread's
        constexpr int PER = C::PIECES, ST = KST;
        static_assert(KST == VST || !Q4, "one count of stages");
        const int ch = w % CPR, r0 = w / CPR;
        const long long base = ((long long)sequence() * p.nkv + kv_head()) * p.S + r0;
        const unsigned char *codes = (isv ? p.kv4.v : p.kv4.k) + base * (HD / 2) + 16 * ch;
        const unsigned char *scales = (isv ? p.kv4.v_scale : p.kv4.k_scale) + base * (HD / 16) + ((2 * ch) & ~3);
        uint64_t *full = isv ? v_full : k_full, *empty = isv ? v_empty : k_empty;
        uint8_t *const ring = smem + C::F_OFF + (isv ? C::DEPTH * C::FETCH : 0);
        const uint32_t ring32 = smem_u32(ring) + 16 * w, sring32 = smem_u32(ring) + PER * 2048 + 4 * w;
        auto fetch = [&](int i, int slot) {
            if (i < n) {
                const int k0 = tile_start(i), end = tile_end(i) - r0;
#pragma unroll
                for (int c = 0; c < PER; ++c) {
                    const int j = k0 + c * STEP;
                    const int live = j < end ? 16 : 0;
                    const long long at = live ? j : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     ring32 + slot * C::FETCH + c * 2048),
                                 "l"(codes + at * (HD / 2)), "r"(live) : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                     sring32 + slot * C::FETCH + c * 512),
                                 "l"(scales + at * (HD / 16)), "r"(live >> 2) : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // the 4 units of a piece, in an order by which eight lanes of a store hit eight different units
        const int turn = HD == 256 ? ch >> 1 : HD == 128 ? 2 * (ch >> 1) : 0;
        uint32_t unit_at[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) unit_at[v] = swizzled(r0, 4 * ch + (v ^ turn), C::PANEL_BYTES);
        bool ok = true;
        // V once Q has left its ring, which leaves Q and the first K tiles the bandwidth
        if (isv && n > 0)
            for (int q = 0; q < NQT; ++q) ok = ok && mbar_wait_bounded(&q_ready[q], 0, limit);
        for (int i = 0; i < C::DEPTH - 1; ++i) fetch(i, i);
        int slot = 0, st = 0, phase = 1;
        for (int i = 0; ok && i < n; ++i) {
            fetch(i + C::DEPTH - 1, slot == 0 ? C::DEPTH - 1 : slot - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(C::DEPTH - 1) : "memory");
            if (i >= ST && !mbar_wait_bounded(&empty[st], phase, limit)) {
                ok = false;
                break;
            }
            uint8_t *dst = smem + (isv ? C::V_OFF : C::K_OFF) + st * C::STAGE;
            uint4 code[PER];
            uint32_t word[PER];
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                code[c] = *reinterpret_cast<const uint4 *>(ring + slot * C::FETCH + c * 2048 + 16 * w);
                word[c] = *reinterpret_cast<const uint32_t *>(ring + slot * C::FETCH + PER * 2048 + c * 512 + 4 * w);
            }
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                const uint32_t scale = ch & 1 ? word[c] >> 16 : word[c];
                uint32_t sp[2];
                asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
                    : "=r"(sp[0]) : "r"(__byte_perm(scale, 0, 0x0000)));
                asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
                    : "=r"(sp[1]) : "r"(__byte_perm(scale, 0, 0x0011)));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int at = v ^ turn;
                    const uint32_t even = at & 2 ? code[c].z : code[c].x, odd = at & 2 ? code[c].w : code[c].y;
                    *reinterpret_cast<uint4 *>(dst + unit_at[v] + c * STEP * 128) =
                        widen_unit(at & 1 ? odd : even, at & 2 ? sp[1] : sp[0]);
                }
            }
            fence_async_shared();
            mbar_arrive(&full[st]);
            if (++slot == C::DEPTH) slot = 0;
            if (++st == ST) { st = 0; phase ^= 1; }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (!ok && (w & 31) == 0) atomicOr(p.status, 1u);
    }

    if (partitions() > 1 && (warp < 4 || warp >= 4 + 4 * NQT)) {
        // the softmax warps merge in between (they have the registers)
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM);
    }
}

template <int HD, int KIND> cudaError_t prepare_tiles()
{
    for (auto kernel : {window_tiles_kernel<HD, KIND, false>, window_tiles_kernel<HD, KIND, true>}) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<HD, KIND>::SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Clusters of n CTAs that the GPU holds at once (0: the kernel takes none of that size).
template <int HD, int KIND> cudaError_t count_clusters(int slots[kMaxParts + 1])
{
    using C = TileCfg<HD, KIND>;
    for (int n = 1; n <= kMaxParts; ++n) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = n;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        slots[n] = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&slots[n], window_tiles_kernel<HD, KIND, true>, &cfg);
        if (e != cudaSuccess) return e;
    }
    return slots[1] > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int HD, int KIND> cudaError_t launch_tiles(const WindowParams &p, const WindowMaps &maps, cudaStream_t s)
{
    using C = TileCfg<HD, KIND>;
    const long long rows = (long long)p.T * p.G;
    cudaLaunchConfig_t cfg = {};
    const unsigned blocks = (unsigned)((rows + C::NQT * 128 - 1) / (C::NQT * 128));
    // dealt: a cluster for each row tile that there can be
    cfg.gridDim = p.dealt ? dim3(blocks * p.batch * p.nkv * p.chunks) : dim3(blocks, p.batch * p.nkv, p.chunks);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.dealt ? p.chunks : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = p.dealt ? 1 : p.chunks;
    cfg.attrs = attr;
    cfg.numAttrs = p.chunks > 1 ? 1 : 0;
    return p.dealt ? cudaLaunchKernelEx(&cfg, window_tiles_kernel<HD, KIND, true>, maps, p)
                   : cudaLaunchKernelEx(&cfg, window_tiles_kernel<HD, KIND, false>, maps, p);
}

}  // namespace
}  // namespace dg
