// serving.cuh -- declarations shared by the serving operators' translation units: rotary positions
// and per-head norms on [batch, T, heads, hd] rows (rope_rows.cu), the 4-bit cache (kv4_append.cu),
// attention with a sliding window and sink tokens (window_*.cu), and their C entries
// (serving_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace dg {

// Element types, the DG_DTYPE_* values.
enum RowType : int { kRowF32 = 0, kRowF16 = 1, kRowBf16 = 2 };

// [batch, T, heads, hd] with strides in elements; the hd elements of a head are dense.
struct Rows {
    void *data;
    long long batch, token, head;
};

constexpr int kMaxRotPairs = 128;      // rot_dim <= hd <= 256

struct RopeRowsParams {
    Rows in[3], out[3];                // q, k, v (heads[i] == 0: absent)
    int heads[3];
    const void *positions;             // [batch, T], dense
    const float *w[2];                 // q and k norm weights [hd] or null
    int batch, T, H;                   // H: heads of all three together
    int in_type, out_type, pos64;
    int rot, interleaved, norm;        // norm: RMS norm of q, k (weighted) and v
    int tokens_per_block;
    float eps, magnitude;
    // frequency of pair i in turns per position, as a fraction of 2^64: position * turn[i] mod 2^64
    // is the angle's fraction of a turn for any 64-bit position
    unsigned long long turn[kMaxRotPairs];
};
cudaError_t launch_rope_rows(RopeRowsParams &p, int hd, cudaStream_t s);

// The 4-bit cache: e2m1 codes, two to a byte (element 2i in the low half), [batch, nkv, cap, hd/2],
// and one e4m3 scale for 16 elements, [batch, nkv, cap, hd/16].
struct Kv4 {
    unsigned char *k, *k_scale, *v, *v_scale;
};

struct Kv4AppendParams {
    Rows in[2], out[2];                // K, V; out.data null: values not returned
    unsigned char *codes[2], *scales[2];
    const int *start, *length;         // [batch]; length may be null (T)
    int batch, T, nkv, cap, type;
};
cudaError_t launch_kv4_append(const Kv4AppendParams &p, int hd, cudaStream_t s);

// Attention: query i of sequence b stands at position p = kv_len - q_len + i and sees key j iff
// j < kv_len, j <= p + right (right >= 0), and j >= p - left (left >= 0) or j < sinks.
struct WindowParams {
    Rows q, k, v, out;                 // k, v: 16-bit rows (kv4: unused)
    Kv4 kv4;
    const int *q_len, *kv_len;         // [batch] or null (T, S)
    int batch, T, S, nh, nkv, G;
    int left, right, sinks;
    int bf16;                          // q, out (and k, v) are bf16, else f16
    float scale;
    uint32_t *status;
    unsigned long long wait_limit_ns;
    // tiles: key partitions of a row tile.  Few rows: CTAs; their unfinished pairs' results until the last
    // CTA of a pair merges them, O [2 chunks, rows_cap, hd] and (m, l) [2 chunks, rows_cap], and how many
    // have arrived of each pair [batch * nkv] (0 between calls)
    int chunks, rows_cap;
    // tiles of a padded batch of up to 32 sequences, in clusters that the kernel deals to the row tiles
    // (TilePlan); else 0
    int dealt, cluster_slots;
    float tile_clocks, merge_clocks;
    float *part_o;
    float2 *part_ml;
    unsigned int *arrived;
};

// Limits that keep positions and window ends in 32 bits: S and T at most kMaxLength, left and right
// held to kMaxReach (beyond any key) by the caller.
constexpr int kMaxLength = 1 << 28, kMaxReach = 1 << 29;

// What query row i of a sequence of nq queries and nk keys sees: [lo, hi) and [0, min(sinks, hi)).
struct Visible {
    int lo, hi;
};
__host__ __device__ inline Visible visible_keys(const WindowParams &p, int nq, int nk, int i)
{
    const int pos = nk - nq + i;
    const int hi = p.right < 0 ? nk : pos + p.right + 1 < nk ? (pos + p.right + 1 > 0 ? pos + p.right + 1 : 0) : nk;
    const int lo = p.left < 0 || pos <= p.left ? 0 : pos - p.left;
    return {lo < hi ? lo : hi, hi};
}

cudaError_t launch_window_rows(const WindowParams &p, int hd, cudaStream_t s);

// Rows of a kv head (T * G) that launch_window_few takes: up to where the tile kernel is as fast.  us, few
// against tiles, 8 sequences of 8192 keys, 4 kv heads (and one of 2048), bf16 (f16: the same within 3):
//   16-bit  hd 64:   8 rows 30 31 (13 13), 16 rows 34 30 (15 13)
//           hd 128:  2 rows 42 47 (15 15), 8 rows 44 46 (17 15), 16 rows 50 47 (22 15)
//           hd 256:  2 rows 67 66 (16 18), 8 rows 73 67 (22 17)
//   4-bit   hd 64:   8 rows 22 42 (13 16), 16 rows 28 42 (15 15)
//           hd 128:  8 rows 30 45 (15 20), 16 rows 37 45 (20 19)
//           hd 256:  2 rows 37 45 (15 22), 8 rows 42 45 (20 22)
inline int few_rows_max(int hd, bool kv4) { return kv4 ? (hd == 256 ? 8 : 16) : hd == 256 ? 4 : 8; }
// The keys a row can see at most.
inline long long window_keys(int T, int S, int left, int right, int sinks)
{
    const long long span = left < 0 || right < 0 ? S : (long long)left + right + T + sinks;
    return span < S ? span : S;
}
// CTAs of a call: kFewCtasPerSm an SM at most, or one a (sequence, kv head) pair beyond kFewSequences.
constexpr int kFewCtasPerSm = 4, kFewSequences = 512;
// CTAs an SM holds at once (after prepare_window_few; 0: the kernel cannot run); two: more than 8 rows (4-bit).
int few_ctas_per_sm(int hd, bool two, bool kv4);
cudaError_t launch_window_few(const WindowParams &p, int hd, bool kv4, cudaStream_t s);
cudaError_t prepare_window_few();

// Many rows: tiles on the tensor cores; p.chunks is the number of key partitions of a row tile.
int tile_rows(int hd, bool kv4);       // rows of a CTA
// Clusters of n CTAs that the GPU holds at once, n = 1 .. kMaxParts (after prepare_window_tiles).
constexpr int kMaxParts = 8;
cudaError_t tile_clusters(int hd, bool kv4, int slots[kMaxParts + 1]);
cudaError_t tile_clusters_kv4(int hd, int slots[kMaxParts + 1]);
// Key partitions of a row tile, and whether the kernel deals them.
struct TilePlan {
    int parts, dealt;
    float tile_clocks, merge_clocks;
};
TilePlan tile_plan(long long pairs, long long rows, int hd, bool kv4, int keys, const int slots[kMaxParts + 1],
                   bool ragged, bool few_sequences);
cudaError_t launch_window_tiles(const WindowParams &p, int hd, bool kv4, cudaStream_t s);
cudaError_t prepare_window_tiles();
cudaError_t launch_window_tiles_kv4(const WindowParams &p, int hd, cudaStream_t s);
cudaError_t prepare_window_tiles_kv4();

}  // namespace dg
