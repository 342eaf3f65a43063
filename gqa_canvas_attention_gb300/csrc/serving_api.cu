// serving_api.cu -- the C entries of the serving operators (declared in include/dg_attn.h): argument
// checks, the rotary frequencies, and the attention plan with its scratch.
#include "../../include/dg_attn.h"
#include "serving.cuh"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

namespace {

thread_local char g_error[512] = "";

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return status;
}

int cuda_fail(cudaError_t e, const char *what)
{
    return fail(DG_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int type_size(int type) { return type == DG_DTYPE_F32 ? 4 : 2; }

// One tensor of a call: its rows, sizes and element size.  Strides of dimensions of size 1 count
// for nothing.
struct Tensor {
    const char *name;
    const dg_attn_rows *r;
    long long n[3];                  // batch, token, head
    int hd, size;

    long long stride(int d) const { return d == 0 ? r->batch : d == 1 ? r->token : r->head; }
    const char *first() const
    {
        long long at = 0;
        for (int d = 0; d < 3; ++d)
            if (n[d] > 1 && stride(d) < 0) at += stride(d) * (n[d] - 1);
        return static_cast<const char *>(r->data) + at * size;
    }
    const char *end() const
    {
        long long at = hd;
        for (int d = 0; d < 3; ++d)
            if (n[d] > 1 && stride(d) > 0) at += stride(d) * (n[d] - 1);
        return static_cast<const char *>(r->data) + at * size;
    }
};

// Elements that a dimension reaches over at most, so that byte offsets of three of them stay in 64 bits.
constexpr long long kMaxExtent = 1LL << 57;

int check_layout(const Tensor &t)
{
    if (!t.r->data) return fail(DG_ERR_ARG, "%s is NULL", t.name);
    if (!aligned16(t.r->data)) return fail(DG_ERR_ALIGN, "%s is not 16-byte aligned", t.name);
    for (int d = 0; d < 3; ++d) {
        if (t.n[d] <= 1) continue;
        if (t.stride(d) > kMaxExtent / t.n[d] || t.stride(d) < -kMaxExtent / t.n[d])
            return fail(DG_ERR_ARG, "%s: a stride of %lld elements leaves the address space", t.name, t.stride(d));
        if ((t.stride(d) * t.size) % 16)
            return fail(DG_ERR_ALIGN, "%s: a stride of %lld elements is not a multiple of 16 bytes", t.name,
                        t.stride(d));
    }
    return DG_OK;
}

// An output's rows share no element: in the order of their strides, each steps past the ones below.
int check_distinct(const Tensor &t)
{
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return std::llabs(t.stride(a)) < std::llabs(t.stride(b)); });
    long long extent = t.hd;
    for (int d : order) {
        if (t.n[d] == 1) continue;
        if (std::llabs(t.stride(d)) < extent) return fail(DG_ERR_ARG, "rows of %s overlap", t.name);
        extent += std::llabs(t.stride(d)) * (t.n[d] - 1);
    }
    return DG_OK;
}

// One term of the distance between a row of one tensor and a row of another: step * x, x in [lo, hi].
struct Term {
    long long step, lo, hi;
};

// Whether distance + sum step_i x_i can lie in (-before, after); terms in falling order of their steps, all
// positive.  Each term leaves few x, since the smaller ones reach less far than one step of it in any usual
// layout; where that is not so and `budget` runs out, the answer is yes.
bool can_meet(const Term *t, int n, long long distance, long long before, long long after, int &budget)
{
    if (n == 0) return -before < distance && distance < after;
    long long low = distance, high = distance;       // with the smaller terms at their ends
    for (int i = 1; i < n; ++i) {
        low += t[i].step * t[i].lo;
        high += t[i].step * t[i].hi;
    }
    auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0); };
    const long long from = std::max(t->lo, floor_div(-before - high, t->step) + 1);
    const long long to = std::min(t->hi, -(floor_div(low - after, t->step) + 1));
    for (long long x = from; x <= to; ++x) {
        if (--budget < 0) return true;
        if (can_meet(t + 1, n - 1, distance + t->step * x, before, after, budget)) return true;
    }
    return false;
}

// Whether two tensors share bytes, as slices of one buffer do not although their ranges meet.
bool may_overlap(const Tensor &a, const Tensor &b)
{
    if (a.end() <= b.first() || b.end() <= a.first()) return false;
    Term t[6];
    int n = 0;
    for (int side = 0; side < 2; ++side) {
        const Tensor &x = side ? b : a;
        for (int d = 0; d < 3; ++d) {
            const long long step = x.stride(d) * x.size * (side ? 1 : -1), last = x.n[d] - 1;
            if (step == 0 || last == 0) continue;
            const Term one = {std::llabs(step), step > 0 ? 0 : -last, step > 0 ? last : 0};
            int i = 0;
            while (i < n && t[i].step != one.step) ++i;
            if (i == n) t[n++] = {one.step, 0, 0};
            t[i].lo += one.lo;
            t[i].hi += one.hi;
        }
    }
    std::sort(t, t + n, [](const Term &x, const Term &y) { return x.step > y.step; });
    int budget = 2000;
    return can_meet(t, n, static_cast<const char *>(b.r->data) - static_cast<const char *>(a.r->data),
                    (long long)b.hd * b.size, (long long)a.hd * a.size, budget);
}

bool same_rows(const Tensor &a, const Tensor &b)
{
    if (a.r->data != b.r->data || a.size != b.size) return false;
    for (int d = 0; d < 3; ++d)
        if (a.n[d] > 1 && a.stride(d) != b.stride(d)) return false;
    return true;
}

dg::Rows rows(const dg_attn_rows &r, const long long n[3])
{
    // a dimension of size 1 is never stepped along
    return {r.data, n[0] > 1 ? r.batch : 0, n[1] > 1 ? r.token : 0, n[2] > 1 ? r.head : 0};
}

bool known_type(int t) { return t == DG_DTYPE_F32 || t == DG_DTYPE_F16 || t == DG_DTYPE_BF16; }

}  // namespace

struct dg_attn_rope {
    int hd, rot, layout;
    double magnitude;
    double f[dg::kMaxRotPairs];
    unsigned long long turn[dg::kMaxRotPairs];
};

struct dg_attn_window_plan {
    int nh, nkv, hd, batch, T, S, device, sms;
    uint32_t *status;
    unsigned long long wait_limit_ns;
    // few query rows of a kv head: the results of its runs of keys until they are merged
    unsigned int *arrived;           // [batch * nkv]
    float *part_o;                   // [slots, rows, hd]
    float2 *part_ml;                 // [slots, rows]
    int few_rows;                    // rows they hold
    int few_ctas[2][2];              // CTAs an SM holds, by more than 8 rows and 4-bit keys
    int clusters[2][dg::kMaxParts + 1];     // many rows: clusters of n CTAs that the GPU holds, by 4-bit keys
};

namespace {

int rope_rows(const dg_attn_rope *rope, const dg_attn_rope_args *a, bool norm, cudaStream_t stream)
{
    if (!rope || !a) return fail(DG_ERR_ARG, "NULL rope or arguments");
    if (a->batch < 0 || a->T < 0 || a->nh < 1 || a->nkv < 0 || (long long)a->nh + 2LL * a->nkv > (1 << 18) ||
        (long long)a->batch * a->T > (1 << 30))
        return fail(DG_ERR_ARG, "batch %d, T %d, nh %d, nkv %d: batch * T <= 2^30", a->batch, a->T, a->nh, a->nkv);
    if (!known_type(a->in_type) || !known_type(a->out_type)) return fail(DG_ERR_ARG, "unknown element type");
    if (a->pos_int64 != 0 && a->pos_int64 != 1) return fail(DG_ERR_ARG, "pos_int64 is 0 or 1");
    if (norm && !(a->eps >= 0.f && std::isfinite(a->eps))) return fail(DG_ERR_ARG, "eps must be finite, not negative");
    if (a->batch == 0 || a->T == 0) return DG_OK;
    const bool has_k = a->nkv > 0, has_v = norm && a->nkv > 0 && a->v.data;
    if (!a->positions) return fail(DG_ERR_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(a->positions) % (a->pos_int64 ? 8 : 4))
        return fail(DG_ERR_ALIGN, "positions is not aligned to its type");
    if (norm && (!aligned16(a->q_norm_w) || !aligned16(a->k_norm_w)))
        return fail(DG_ERR_ALIGN, "a norm weight is not 16-byte aligned");
    const dg_attn_rows *in[3] = {&a->q, &a->k, &a->v}, *out[3] = {&a->q_out, &a->k_out, &a->v_out};
    const char *in_name[3] = {"q", "k", "v"}, *out_name[3] = {"q_out", "k_out", "v_out"};
    const bool has[3] = {true, has_k, has_v};
    Tensor ti[3], to[3];
    dg::RopeRowsParams p = {};
    for (int i = 0; i < 3; ++i) {
        const long long heads = i ? a->nkv : a->nh;
        ti[i] = {in_name[i], in[i], {a->batch, a->T, heads}, rope->hd, type_size(a->in_type)};
        to[i] = {out_name[i], out[i], {a->batch, a->T, heads}, rope->hd, type_size(a->out_type)};
        if (!has[i]) continue;
        for (int rc : {check_layout(ti[i]), check_layout(to[i])})
            if (rc) return rc;
        if (int rc = check_distinct(to[i])) return rc;
        p.heads[i] = (int)heads;
        p.in[i] = rows(*in[i], ti[i].n);
        p.out[i] = rows(*out[i], to[i].n);
        p.H += (int)heads;
    }
    for (int i = 0; i < 3; ++i) {
        if (!has[i]) continue;
        for (int j = 0; j < 3; ++j) {
            if (!has[j]) continue;
            const bool in_place = i == j && a->in_type == a->out_type && same_rows(to[i], ti[j]);
            if (!in_place && may_overlap(to[i], ti[j]))
                return fail(DG_ERR_ARG, "%s overlaps %s", to[i].name, ti[j].name);
            if (i < j && may_overlap(to[i], to[j]))
                return fail(DG_ERR_ARG, "%s overlaps %s", to[i].name, to[j].name);
        }
    }
    p.positions = a->positions;
    p.w[0] = norm ? a->q_norm_w : nullptr;
    p.w[1] = norm ? a->k_norm_w : nullptr;
    p.batch = a->batch;
    p.T = a->T;
    p.in_type = a->in_type;
    p.out_type = a->out_type;
    p.pos64 = a->pos_int64;
    p.rot = rope->rot;
    p.interleaved = rope->layout == DG_ROPE_INTERLEAVED;
    p.norm = norm;
    p.eps = a->eps;
    p.magnitude = (float)rope->magnitude;
    memcpy(p.turn, rope->turn, sizeof(p.turn));
    const cudaError_t e = dg::launch_rope_rows(p, rope->hd, stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, "rotary positions");
}

int check_cache(const dg_attn_kv4 *c)
{
    if (!c) return fail(DG_ERR_ARG, "NULL cache");
    if (c->batch < 1 || c->nkv < 1 || c->cap < 1 || (c->hd != 64 && c->hd != 128 && c->hd != 256) ||
        (long long)c->batch * c->nkv > (1LL << 48) / c->cap)
        return fail(DG_ERR_ARG, "cache of batch %d, nkv %d, cap %d, hd %d", c->batch, c->nkv, c->cap, c->hd);
    if (!c->k || !c->k_scale || !c->v || !c->v_scale) return fail(DG_ERR_ARG, "a cache buffer is NULL");
    if (!aligned16(c->k) || !aligned16(c->k_scale) || !aligned16(c->v) || !aligned16(c->v_scale))
        return fail(DG_ERR_ALIGN, "a cache buffer is not 16-byte aligned");
    return DG_OK;
}

// The four buffers of a cache as tensors of bytes.
void cache_tensors(const dg_attn_kv4 *c, dg_attn_rows r[4], Tensor t[4])
{
    unsigned char *p[4] = {c->k, c->k_scale, c->v, c->v_scale};
    for (int i = 0; i < 4; ++i) {
        const long long n = (long long)c->batch * c->nkv * c->cap;
        const int bytes = c->hd / (i % 2 ? 16 : 2);
        r[i] = {p[i], bytes, 0, 0};
        t[i] = {"the cache", &r[i], {n, 1, 1}, bytes, 1};
    }
}

int attend(dg_attn_window_plan *plan, const dg_attn_window_args *a, const dg_attn_kv4 *cache, bool kv4,
           cudaStream_t stream)
{
    if (!plan || !a) return fail(DG_ERR_ARG, "NULL plan or arguments");
    if (a->batch < 0 || a->batch > plan->batch || a->T < 0 || a->T > plan->T || a->S < 0 || a->S > plan->S)
        return fail(DG_ERR_ARG, "batch %d, T %d, S %d: the plan holds %d, %d, %d", a->batch, a->T, a->S, plan->batch,
                    plan->T, plan->S);
    if (a->type != DG_DTYPE_F16 && a->type != DG_DTYPE_BF16) return fail(DG_ERR_ARG, "q and out are f16 or bf16");
    if (a->left < -1 || a->right < -1 || a->sinks < 0) return fail(DG_ERR_ARG, "left and right >= -1, sinks >= 0");
    if (!std::isfinite(a->scale)) return fail(DG_ERR_ARG, "scale must be finite");
    if (kv4) {
        if (int rc = check_cache(cache)) return rc;
        if (cache->batch != a->batch || cache->nkv != plan->nkv || cache->hd != plan->hd || cache->cap != a->S)
            return fail(DG_ERR_ARG, "the cache's batch, nkv, cap or hd is not the call's");
    }
    if (a->batch == 0 || a->T == 0) return DG_OK;
    int device = -1;
    if (cudaError_t e = cudaGetDevice(&device)) return cuda_fail(e, "attention");
    if (device != plan->device)
        return fail(DG_ERR_ARG, "the plan belongs to device %d, device %d is current", plan->device, device);
    for (const int *l : {a->q_len, a->kv_len})
        if (reinterpret_cast<uintptr_t>(l) % 4) return fail(DG_ERR_ALIGN, "lengths are not 4-byte aligned");
    const Tensor q = {"q", &a->q, {a->batch, a->T, plan->nh}, plan->hd, 2};
    const Tensor out = {"out", &a->out, {a->batch, a->T, plan->nh}, plan->hd, 2};
    const Tensor k = {"k", &a->k, {a->batch, a->S, plan->nkv}, plan->hd, 2};
    const Tensor v = {"v", &a->v, {a->batch, a->S, plan->nkv}, plan->hd, 2};
    for (int rc : {check_layout(q), check_layout(out)})
        if (rc) return rc;
    if (int rc = check_distinct(out)) return rc;
    if (may_overlap(out, q)) return fail(DG_ERR_ARG, "out overlaps q");
    dg::WindowParams p = {};
    if (kv4) {
        dg_attn_rows r[4];
        Tensor t[4];
        cache_tensors(cache, r, t);
        for (const Tensor &x : t)
            if (may_overlap(out, x)) return fail(DG_ERR_ARG, "out overlaps the cache");
        p.kv4 = {cache->k, cache->k_scale, cache->v, cache->v_scale};
    } else if (a->S > 0) {
        for (int rc : {check_layout(k), check_layout(v)})
            if (rc) return rc;
        if (may_overlap(out, k) || may_overlap(out, v)) return fail(DG_ERR_ARG, "out overlaps k or v");
        p.k = rows(a->k, k.n);
        p.v = rows(a->v, v.n);
    }
    p.q = rows(a->q, q.n);
    p.out = rows(a->out, out.n);
    p.q_len = a->q_len;
    p.kv_len = a->kv_len;
    p.batch = a->batch;
    p.T = a->T;
    p.S = a->S;
    p.nh = plan->nh;
    p.nkv = plan->nkv;
    p.G = plan->nh / plan->nkv;
    p.left = std::min(a->left, dg::kMaxReach);
    p.right = std::min(a->right, dg::kMaxReach);
    p.sinks = a->sinks;
    p.bf16 = a->type == DG_DTYPE_BF16;
    p.scale = a->scale;
    p.status = plan->status;
    p.wait_limit_ns = plan->wait_limit_ns;
    const long long rows = (long long)p.T * p.G;
    cudaError_t e;
    if (rows <= std::min(plan->few_rows, dg::few_rows_max(plan->hd, kv4))) {
        p.chunks = p.batch > dg::kFewSequences ? p.batch * p.nkv : plan->few_ctas[rows > 8][kv4] * plan->sms;
        p.rows_cap = (int)rows;
        p.part_o = plan->part_o;
        p.part_ml = plan->part_ml;
        p.arrived = plan->arrived;
        e = dg::launch_window_few(p, plan->hd, kv4, stream);
    } else {
        // a block's rows span block / G + 1 tokens at most
        const int block = dg::tile_rows(plan->hd, kv4);
        const long long keys = dg::window_keys(std::min(p.T, block / p.G + 2), p.S, p.left, p.right, p.sinks);
        const int *slots = plan->clusters[kv4];
        const dg::TilePlan t = dg::tile_plan((long long)p.batch * p.nkv, rows, plan->hd, kv4, (int)keys, slots,
                                             p.q_len || p.kv_len, p.batch > 1 && p.batch <= 32);
        p.chunks = t.parts;
        p.dealt = t.dealt;
        p.cluster_slots = slots[t.parts];
        p.tile_clocks = t.tile_clocks;
        p.merge_clocks = t.merge_clocks;
        e = dg::launch_window_tiles(p, plan->hd, kv4, stream);
    }
    return e == cudaSuccess ? DG_OK : cuda_fail(e, "attention");
}

}  // namespace

extern "C" {

dg_attn_rope *dg_attn_rope_create(int hd, int rot_dim, int layout, double theta, int scaling, double factor,
                                  double original)
{
    if (hd != 32 && hd != 64 && hd != 128 && hd != 256) {
        fail(DG_ERR_ARG, "hd %d: 32, 64, 128 or 256", hd);
        return nullptr;
    }
    if (rot_dim < 8 || rot_dim > hd || rot_dim % 8) {
        fail(DG_ERR_ARG, "rot_dim %d: a multiple of 8 up to hd", rot_dim);
        return nullptr;
    }
    if ((layout != DG_ROPE_HALF && layout != DG_ROPE_INTERLEAVED) || scaling < DG_ROPE_SCALE_NONE ||
        scaling > DG_ROPE_SCALE_YARN) {
        fail(DG_ERR_ARG, "unknown layout or scaling");
        return nullptr;
    }
    if (!(theta > 1.0 && std::isfinite(theta)) ||
        (scaling != DG_ROPE_SCALE_NONE && !(factor >= 1.0 && std::isfinite(factor))) ||
        (scaling == DG_ROPE_SCALE_YARN && !(original >= 1.0 && std::isfinite(original)))) {
        fail(DG_ERR_ARG, "theta > 1, factor >= 1 and original >= 1 are wanted, all finite");
        return nullptr;
    }
    dg_attn_rope *r = new (std::nothrow) dg_attn_rope();
    if (!r) {
        fail(DG_ERR_ARG, "out of host memory");
        return nullptr;
    }
    r->hd = hd;
    r->rot = rot_dim;
    r->layout = layout;
    r->magnitude = 1.0;
    const double two_pi = 6.283185307179586476925;
    const double inv_two_pi = 0.15915494309189535, inv_two_pi_rest = -9.839338337591243e-18;    // their sum: to 2^-110
    if (scaling == DG_ROPE_SCALE_NTK) theta *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    double lo = 0, hi = 0;
    if (scaling == DG_ROPE_SCALE_YARN) {
        // the pair that makes n turns over the original positions: i = rot ln(original / 2 pi n) / 2 ln theta
        auto pair = [&](double n) { return rot_dim * std::log(original / (n * two_pi)) / (2 * std::log(theta)); };
        lo = std::max(std::floor(pair(32)), 0.0);
        hi = std::min(std::ceil(pair(1)), rot_dim - 1.0);
        r->magnitude = 0.1 * std::log(factor) + 1.0;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == DG_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == DG_ROPE_SCALE_YARN) {
            const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1 - ramp) + f / factor * ramp;
        }
        r->f[i] = f;
        // f / 2 pi to 2^-64 of a turn, in two parts (a double alone ends at 2^-56); f <= 1, so it is below 1/6
        const double turn = f * inv_two_pi, rest = std::fma(f, inv_two_pi, -turn) + f * inv_two_pi_rest;
        r->turn[i] = (unsigned long long)std::llround(std::ldexp(turn, 64)) +
                     (unsigned long long)std::llround(std::ldexp(rest, 64));
    }
    return r;
}

void dg_attn_rope_destroy(dg_attn_rope *rope) { delete rope; }

int dg_attn_rope_frequencies(const dg_attn_rope *rope, double *f, double *magnitude)
{
    if (!rope || !f || !magnitude) return fail(DG_ERR_ARG, "NULL argument");
    for (int i = 0; i < rope->rot / 2; ++i) f[i] = rope->f[i];
    *magnitude = rope->magnitude;
    return DG_OK;
}

int dg_attn_rope_apply(const dg_attn_rope *rope, const dg_attn_rope_args *args, cudaStream_t stream)
{
    return rope_rows(rope, args, false, stream);
}

int dg_attn_qk_norm_rope(const dg_attn_rope *rope, const dg_attn_rope_args *args, cudaStream_t stream)
{
    return rope_rows(rope, args, true, stream);
}

int dg_attn_kv4_append(const dg_attn_kv4 *cache, const dg_attn_kv4_args *a, cudaStream_t stream)
{
    if (int rc = check_cache(cache)) return rc;
    if (!a) return fail(DG_ERR_ARG, "NULL arguments");
    if (a->T < 0) return fail(DG_ERR_ARG, "T %d", a->T);
    if (!known_type(a->type)) return fail(DG_ERR_ARG, "unknown element type");
    if (!a->k_out.data != !a->v_out.data) return fail(DG_ERR_ARG, "k_out and v_out go together");
    if (a->T == 0) return DG_OK;
    if (!a->start) return fail(DG_ERR_ARG, "start is NULL");
    for (const int *l : {a->start, a->length})
        if (reinterpret_cast<uintptr_t>(l) % 4) return fail(DG_ERR_ALIGN, "start or length is not 4-byte aligned");
    if (cache->batch > 65535 || (long long)a->T * cache->nkv > (1LL << 30) / (cache->hd / 16))
        return fail(DG_ERR_ARG, "batch %d, T * nkv * hd %lld: at most 65535 and 2^34", cache->batch,
                    (long long)a->T * cache->nkv * cache->hd);
    const bool values = a->k_out.data != nullptr;
    const dg_attn_rows *in[2] = {&a->k, &a->v}, *out[2] = {&a->k_out, &a->v_out};
    const char *in_name[2] = {"k", "v"}, *out_name[2] = {"k_out", "v_out"};
    dg_attn_rows r[4];
    Tensor ti[2], to[2], tc[4];
    cache_tensors(cache, r, tc);
    dg::Kv4AppendParams p = {};
    for (int i = 0; i < 2; ++i) {
        ti[i] = {in_name[i], in[i], {cache->batch, a->T, cache->nkv}, cache->hd, type_size(a->type)};
        to[i] = {out_name[i], out[i], {cache->batch, a->T, cache->nkv}, cache->hd, type_size(a->type)};
        if (int rc = check_layout(ti[i])) return rc;
        p.in[i] = rows(*in[i], ti[i].n);
        if (values) {
            if (int rc = check_layout(to[i])) return rc;
            if (int rc = check_distinct(to[i])) return rc;
            p.out[i] = rows(*out[i], to[i].n);
        }
    }
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 4; ++j) {
            if (may_overlap(tc[j], ti[i]) || (values && may_overlap(tc[j], to[i])))
                return fail(DG_ERR_ARG, "the cache overlaps k, v, k_out or v_out");
        }
        for (int j = 0; values && j < 2; ++j)
            if (may_overlap(to[i], ti[j])) return fail(DG_ERR_ARG, "%s overlaps %s", to[i].name, ti[j].name);
    }
    if (values && may_overlap(to[0], to[1])) return fail(DG_ERR_ARG, "k_out overlaps v_out");
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (may_overlap(tc[i], tc[j])) return fail(DG_ERR_ARG, "two cache buffers overlap");
    p.codes[0] = cache->k;
    p.codes[1] = cache->v;
    p.scales[0] = cache->k_scale;
    p.scales[1] = cache->v_scale;
    p.start = a->start;
    p.length = a->length;
    p.batch = cache->batch;
    p.T = a->T;
    p.nkv = cache->nkv;
    p.cap = cache->cap;
    p.type = a->type;
    const cudaError_t e = dg::launch_kv4_append(p, cache->hd, stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, "storing rows");
}

dg_attn_window_plan *dg_attn_window_plan_create(int nh, int nkv, int hd, int batch, int T, int S)
{
    if (nkv < 1 || nh < 1 || nh % nkv || (hd != 64 && hd != 128 && hd != 256)) {
        fail(DG_ERR_ARG, "nh %d, nkv %d, hd %d: nh a multiple of nkv, hd 64, 128 or 256", nh, nkv, hd);
        return nullptr;
    }
    // rows of a kv group (T * G) and their count over the batch are numbered in 32 bits
    if (batch < 1 || T < 1 || S < 0 || (long long)batch * nkv > 65535 || (long long)T * nh > (1LL << 30) ||
        (long long)batch * T * nh > (1LL << 31) - 1 || S > dg::kMaxLength || T > dg::kMaxLength) {
        fail(DG_ERR_ARG, "batch %d, T %d, S %d: batch * nkv <= 65535, batch * T * nh < 2^31, T, S <= 2^28", batch, T, S);
        return nullptr;
    }
    dg_attn_window_plan *p = new (std::nothrow) dg_attn_window_plan();
    if (!p) {
        fail(DG_ERR_ARG, "out of host memory");
        return nullptr;
    }
    *p = {};
    p->nh = nh;
    p->nkv = nkv;
    p->hd = hd;
    p->batch = batch;
    p->T = T;
    p->S = S;
    p->wait_limit_ns = 2000ull * 1000000ull;
    // calls of up to few_rows rows a kv head (any T they come from): two unfinished pairs a CTA
    const int G = nh / nkv;
    p->few_rows = (int)std::min<long long>((long long)T * G, dg::few_rows_max(hd, true));
    const size_t arrived = sizeof(unsigned int) * batch * nkv;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device);
    if (e == cudaSuccess) e = cudaMalloc(&p->status, 256);
    if (e == cudaSuccess) e = cudaMemset(p->status, 0, 256);
    if (e == cudaSuccess) e = cudaMalloc(&p->arrived, arrived);
    if (e == cudaSuccess) e = cudaMemset(p->arrived, 0, arrived);
    const size_t slots = 2 * dg::kFewCtasPerSm * p->sms;
    if (e == cudaSuccess) e = cudaMalloc(&p->part_o, sizeof(float) * slots * p->few_rows * hd);
    if (e == cudaSuccess) e = cudaMalloc(&p->part_ml, sizeof(float2) * slots * p->few_rows);
    if (e == cudaSuccess) e = dg::prepare_window_few();
    for (int two = 0; e == cudaSuccess && two <= (p->few_rows > 8); ++two)
        for (int kv4 = two; kv4 < 2; ++kv4)
            if (!(p->few_ctas[two][kv4] = dg::few_ctas_per_sm(hd, two, kv4))) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) e = dg::prepare_window_tiles();
    for (int kv4 = 0; e == cudaSuccess && kv4 < 2; ++kv4) e = dg::tile_clusters(hd, kv4, p->clusters[kv4]);
    // a stream of a later call need not wait for the default one, which clears the scratch
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    if (e != cudaSuccess) {
        cuda_fail(e, "attention plan");
        dg_attn_window_plan_destroy(p);
        return nullptr;
    }
    return p;
}

void dg_attn_window_plan_destroy(dg_attn_window_plan *plan)
{
    if (!plan) return;
    cudaFree(plan->status);
    cudaFree(plan->arrived);
    cudaFree(plan->part_o);
    cudaFree(plan->part_ml);
    delete plan;
}

int dg_attn_window_attend(dg_attn_window_plan *plan, const dg_attn_window_args *args, cudaStream_t stream)
{
    return attend(plan, args, nullptr, false, stream);
}

int dg_attn_window_attend_kv4(dg_attn_window_plan *plan, const dg_attn_window_args *args, const dg_attn_kv4 *cache,
                              cudaStream_t stream)
{
    return attend(plan, args, cache, true, stream);
}

int dg_attn_window_sync_status(dg_attn_window_plan *plan, cudaStream_t stream)
{
    if (!plan) return fail(DG_ERR_ARG, "NULL plan");
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, plan->status, sizeof(v), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemsetAsync(plan->status, 0, sizeof(v), stream);
    if (e != cudaSuccess) return cuda_fail(e, "status");
    if (v) return fail(DG_ERR_TIMEOUT, "a device wait ran out (status %u)", v);
    return DG_OK;
}

const char *dg_attn_serving_last_error(void) { return g_error; }

}  // extern "C"
