// rope_api.cu -- the rotation and cache entry points of include/rmsnorm.h:
// host-side argument checks, kernel choice and launches. No allocation, no
// synchronisation, no host copies; everything is enqueued on the caller's
// stream.
#include "heads_host.h"

using namespace rmsk;

namespace {

constexpr int kPathRope = 13, kPathRopeAppend = 14, kPathKv4Read = 15;
constexpr int kBwdCtasPerSm = 4;          // the backward's grid, at most

const RopeSet &rope_set(int dtype)
{
    return dtype == RMSNORM_BF16 ? rope_bf16 : (dtype == RMSNORM_F16 ? rope_f16 : rope_f32);
}

int check_rope(const rmsnorm_rotation *r, int64_t T, int64_t D, float eps, int dtype)
{
    if (!dtype_ok(dtype))
        return RMSNORM_ERR_BAD_DTYPE;
    if (T < 0 || D < 1)
        return RMSNORM_ERR_BAD_SHAPE;
    if (T > INT32_MAX || D > RMSNORM_ROPE_MAX_D)
        return RMSNORM_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return RMSNORM_ERR_BAD_EPS;
    if (r == nullptr)
        return RMSNORM_OK;
    if (r->rot < 0 || r->rot > D || r->rot % 2)
        return RMSNORM_ERR_BAD_SHAPE;
    if (r->adjacent & ~1)
        return RMSNORM_ERR_BAD_FLAGS;
    if (r->rot == 0)
        return RMSNORM_OK;
    if (!index_bits_ok(r->position_bits))
        return RMSNORM_ERR_BAD_DTYPE;
    if (!std::isfinite(r->amplitude))
        return RMSNORM_ERR_BAD_EPS;
    if (T > 0 && (r->positions == nullptr || r->freq == nullptr))
        return RMSNORM_ERR_NULLPTR;
    if (!aligned(r->positions, r->position_bits / 8) || !aligned(r->freq, 8))
        return RMSNORM_ERR_MISALIGNED;
    return RMSNORM_OK;
}

RopeTurn turn_of(const rmsnorm_rotation *r)
{
    RopeTurn t = {};
    if (r != nullptr && r->rot > 0)
        t = {r->positions, r->freq, (int)r->rot, r->position_bits == 64 ? 1 : 0, r->adjacent, r->amplitude};
    return t;
}

struct Strided {
    const void *p;
    int64_t a, b, c;               // strides, elements
};

// The widest packs that the rows' places allow: an index into set.k.
int pick_packs(const RopeSet &set, int64_t D, const RopeTurn &t, size_t es, const Strided *rows, int n,
               const void *wq, const void *wk)
{
    for (int i = 0; i + 1 < set.n; ++i) {
        const int E = set.k[i].E;
        const int64_t bytes = E * (int64_t)es;
        if (D % E || (!t.adjacent && t.rot % (2 * E)) || !aligned(wq, bytes) || !aligned(wk, bytes))
            continue;
        bool ok = true;
        for (int j = 0; j < n && ok; ++j)
            ok = aligned(rows[j].p, bytes) &&
                 strides_multiple(bytes, es, {rows[j].a, rows[j].b, rows[j].c});
        if (ok)
            return i;
    }
    return set.n - 1;
}

// log2 of the lanes a row takes: a lane two packs, or one of 32 lanes eight
// elements.
int lane_shift(int E, int64_t D)
{
    if (E == 1)
        return 5;
    const int64_t pairs = (D / E + 1) / 2;
    int s = 0;
    while ((1 << s) < pairs)
        ++s;
    return s;
}

// Heads a piece: the sines and the map are made once for a piece, at the cost of
// some 1.2 heads; the groups of lanes take the pieces in rounds, the last of which
// may leave most of them idle. So the length of the least rounds x (heads + 1.2),
// of up to eight heads, the longer of two equals. Few tokens come to single heads,
// and many to eight (32768 x 40 x 128 forward, 16384 x 40 x 128 backward, append of
// 8192 tokens: eight 107, 95 and 41 us, four 123, 97 and 44, sixteen 112, 140 and
// 53). Between them the rounds decide: at 4096 x 20 heads with the norm the longest
// that fills the lanes once takes 13.2 us forward and 26.7 backward for heads of
// 128, 14.8 and 33.2 for heads of 80; this rule 10.8, 19.6, 13.5 and 23.1.
int piece(int64_t T, std::initializer_list<int64_t> heads, int64_t groups)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int hc = 8; hc >= 1; hc /= 2) {
        int64_t n = 0;
        for (int64_t h : heads)
            n += (h + hc - 1) / hc;
        const int64_t cost = (T * n + groups - 1) / groups * (5 * hc + 6);
        if (cost < least) {
            least = cost;
            best = hc;
        }
    }
    return best;
}

int check_rows(const rmsnorm_heads *r, int64_t T, int64_t D, size_t es, bool has_y)
{
    if (r->heads < 0)
        return RMSNORM_ERR_BAD_SHAPE;
    if (r->heads > INT32_MAX / 2)
        return RMSNORM_ERR_UNSUPPORTED;
    if (r->heads == 0)
        return RMSNORM_OK;                      // whatever its strides
    if (!rows_within({T, r->heads, 1}, {r->x_token, r->x_head, 0}, D) ||
        (has_y && !rows_apart({T, r->heads, 1}, {r->y_token, r->y_head, 0}, D)))
        return RMSNORM_ERR_BAD_STRIDE;
    if (T == 0)
        return RMSNORM_OK;
    if (!r->x || !r->y)
        return RMSNORM_ERR_NULLPTR;
    if (!aligned(r->x, es) || !aligned(r->y, es) || !aligned(r->w, es))
        return RMSNORM_ERR_MISALIGNED;
    return RMSNORM_OK;
}

RopeRows rows_of(const rmsnorm_heads *r)
{
    RopeRows o = {};
    if (r != nullptr && r->heads > 0)
        o = {r->x, r->x_token, r->x_head, r->w, r->y, r->y_token, r->y_head, (int)r->heads, 0};
    return o;
}

Span index_span(const void *p, int64_t n, int bits) { return flat(p, (size_t)n * bits / 8); }

// What no output of a call may touch: the inputs beside the rows.
bool touches_inputs(Span o, const rmsnorm_rotation *r, int64_t T, int64_t D, size_t es, const void *wq,
                    const void *wk)
{
    if (overlap(o, flat(wq, (size_t)D * es)) || overlap(o, flat(wk, (size_t)D * es)))
        return true;
    return r != nullptr && r->rot > 0 &&
           (overlap(o, index_span(r->positions, T, r->position_bits)) ||
            overlap(o, flat(r->freq, (size_t)r->rot / 2 * 8)));
}

// form: 0 the forward, 1 the append of rows, 2 the append in 4 bits.
int launch_rows(RopeParams &p, const RopeKernel &k, int form, cudaStream_t stream)
{
    int dev, sms, bps, st;
    const void *fn = k.fwd[form][p.turn.adjacent];
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)) ||
        (st = blocks_per_sm(fn, kRopeThreads, dev, &bps, k.fwd_smem[form])))
        return st;
    p.shift = lane_shift(k.E, p.D);
    const int64_t per = kRopeThreads >> p.shift;
    p.HC = piece(p.T, {p.part[0].heads, p.part[1].heads, p.part[2].heads}, (int64_t)sms * bps * per);
    int64_t n = 0;
    for (RopeRows &r : p.part)
        n += r.chunks = (r.heads + p.HC - 1) / p.HC;
    const int64_t ctas = std::min<int64_t>((p.T * n + per - 1) / per, (int64_t)sms * bps);
    void *args[1] = {&p};
    const cudaError_t e = launch_pdl(fn, dim3((unsigned)ctas), kRopeThreads, (size_t)k.fwd_smem[form], stream,
                                     args);
    if (e != cudaSuccess)
        return cuda_fail(e);
    t_last_path = form ? kPathRopeAppend : kPathRope;
    return RMSNORM_OK;
}

struct CacheArgs {
    bool bits4;
    int64_t pages, page_size, k_page, v_page;
    const float *k_scale, *v_scale;
};

// Both forms of the append. q, k and v with the cache's strides in y.
int append_impl(const rmsnorm_heads *q, const rmsnorm_heads *k, const rmsnorm_heads *v,
                const rmsnorm_rotation *rot, const void *slots, int slot_bits, const CacheArgs &c, int64_t T,
                int64_t D, float eps, int dtype, cudaStream_t stream)
{
    int st = check_rope(rot, T, D, eps, dtype);
    if (st)
        return st;
    if (!k || !v)
        return RMSNORM_ERR_NULLPTR;
    if (!index_bits_ok(slot_bits))
        return RMSNORM_ERR_BAD_DTYPE;
    if (k->heads < 1 || k->heads != v->heads || c.pages < 0 || c.page_size < 1)
        return RMSNORM_ERR_BAD_SHAPE;
    if (c.pages > (INT64_MAX >> 8) / c.page_size || c.page_size > INT32_MAX ||
        (c.bits4 && (c.page_size % kKv4Tile || (D != 64 && D != 128))))
        return RMSNORM_ERR_UNSUPPORTED;
    const size_t es = elem_size(dtype);
    if ((q && (st = check_rows(q, T, D, es, true))) || (st = check_rows(k, T, D, es, false)) ||
        (st = check_rows(v, T, D, es, false)))
        return st;
    if (v->w)
        return RMSNORM_ERR_UNSUPPORTED;
    if (!c.bits4 && (!rows_apart({c.pages, c.page_size, k->heads}, {c.k_page, k->y_token, k->y_head}, D) ||
                     !rows_apart({c.pages, c.page_size, v->heads}, {c.v_page, v->y_token, v->y_head}, D)))
        return RMSNORM_ERR_BAD_STRIDE;
    if (T == 0)
        return RMSNORM_OK;
    if (!slots)
        return RMSNORM_ERR_NULLPTR;
    if (!aligned(slots, slot_bits / 8) || (c.bits4 && !aligned(k->y, 16)) || !aligned(c.k_scale, 4) ||
        !aligned(c.v_scale, 4))
        return RMSNORM_ERR_MISALIGNED;

    const void *wq = q ? q->w : nullptr;
    const int64_t Hq = q ? q->heads : 0, Hk = k->heads;
    const Span sx[3] = {q ? heads_span(q->x, T, Hq, D, q->x_token, q->x_head, es) : Span{nullptr, 0, 0, 0},
                        heads_span(k->x, T, Hk, D, k->x_token, k->x_head, es),
                        heads_span(v->x, T, Hk, D, v->x_token, v->x_head, es)};
    const Span sy = q ? heads_span(q->y, T, Hq, D, q->y_token, q->y_head, es) : Span{nullptr, 0, 0, 0};
    Span cache[2];
    if (c.bits4) {
        cache[0] = flat(k->y, (size_t)(c.pages * c.page_size * Hk * (D * 9 / 8)));
        cache[1] = {nullptr, 0, 0, 0};
    } else {
        const int64_t last[2] = {c.k_page, c.v_page};
        for (int i = 0; i < 2; ++i) {
            const rmsnorm_heads *r = i ? v : k;
            cache[i] = c.pages ? flat(r->y, (size_t)((c.pages - 1) * last[i] + (c.page_size - 1) * r->y_token +
                                                     (Hk - 1) * r->y_head + D) * es)
                               : Span{nullptr, 0, 0, 0};
        }
        if (k->y == v->y)
            return RMSNORM_ERR_ALIAS;
    }
    if ((q && !heads_same_or_disjoint(sy, q->y_token, q->y_head, sx[0], q->x_token, q->x_head, T, Hq)) ||
        overlap(sy, sx[1]) || overlap(sy, sx[2]) || overlap(sy, cache[0]) || overlap(sy, cache[1]))
        return RMSNORM_ERR_ALIAS;
    for (Span o : {sy, cache[0], cache[1]})
        if (overlap(o, index_span(slots, T, slot_bits)) || touches_inputs(o, rot, T, D, es, wq, k->w) ||
            overlap(o, flat(c.k_scale, (size_t)Hk * 4)) || overlap(o, flat(c.v_scale, (size_t)Hk * 4)))
            return RMSNORM_ERR_ALIAS;
    for (Span o : cache)
        for (Span i : sx)
            if (overlap(o, i))
                return RMSNORM_ERR_ALIAS;

    RopeParams p = {};
    p.part[0] = rows_of(q);
    p.part[1] = rows_of(k);
    p.part[2] = rows_of(v);
    p.turn = turn_of(rot);
    p.T = T;
    p.D = (int)D;
    p.eps = eps;
    p.inv_d = 1.f / (float)D;
    p.cache = {slots, slot_bits == 64 ? 1 : 0, c.page_size, c.pages * c.page_size,
               c.bits4 ? Hk * (c.page_size / kKv4Tile) * 18 * D : c.k_page, c.v_page, c.k_scale, c.v_scale};
    Strided rows[6];
    int n = 0;
    for (const RopeRows &r : p.part) {
        if (r.heads == 0)
            continue;
        rows[n++] = {r.x, T > 1 ? r.xt : 0, r.heads > 1 ? r.xh : 0, 0};
        const bool to_cache = &r != &p.part[0];
        if (to_cache && c.bits4)
            continue;
        rows[n++] = {r.y, r.yt, r.heads > 1 ? r.yh : 0,
                     to_cache ? (&r == &p.part[1] ? c.k_page : c.v_page) : 0};
    }
    const RopeSet &set = rope_set(dtype);
    const RopeKernel &kern = set.k[pick_packs(set, D, p.turn, es, rows, n, wq, k->w)];
    return launch_rows(p, kern, c.bits4 ? 2 : 1, stream);
}

} // namespace

extern "C" {

int rmsnorm_rope_fwd(const rmsnorm_heads *q, const rmsnorm_heads *k, const rmsnorm_rotation *rot, float *rstd,
                     int64_t T, int64_t D, float eps, int dtype, void *stream)
{
    int st = check_rope(rot, T, D, eps, dtype);
    if (st)
        return st;
    if (!q)
        return RMSNORM_ERR_NULLPTR;
    if (q->heads < 1)
        return RMSNORM_ERR_BAD_SHAPE;
    const size_t es = elem_size(dtype);
    if ((st = check_rows(q, T, D, es, true)) || (k && (st = check_rows(k, T, D, es, true))))
        return st;
    if (T == 0)
        return RMSNORM_OK;
    if (!aligned(rstd, 4))
        return RMSNORM_ERR_MISALIGNED;
    const int64_t Hk = k ? k->heads : 0;
    const void *wk = k ? k->w : nullptr;
    const Span none = {nullptr, 0, 0, 0};
    const Span xq = heads_span(q->x, T, q->heads, D, q->x_token, q->x_head, es),
               yq = heads_span(q->y, T, q->heads, D, q->y_token, q->y_head, es),
               xk = Hk ? heads_span(k->x, T, Hk, D, k->x_token, k->x_head, es) : none,
               yk = Hk ? heads_span(k->y, T, Hk, D, k->y_token, k->y_head, es) : none,
               sr = flat(rstd, (size_t)(T * (q->heads + Hk)) * 4);
    if (!heads_same_or_disjoint(yq, q->y_token, q->y_head, xq, q->x_token, q->x_head, T, q->heads) ||
        (Hk && !heads_same_or_disjoint(yk, k->y_token, k->y_head, xk, k->x_token, k->x_head, T, Hk)) ||
        overlap(yq, yk) || overlap(yq, xk) || overlap(yk, xq))
        return RMSNORM_ERR_ALIAS;
    for (Span o : {yq, yk, sr})
        if (touches_inputs(o, rot, T, D, es, q->w, wk))
            return RMSNORM_ERR_ALIAS;
    for (Span i : {xq, xk, yq, yk})
        if (overlap(sr, i))
            return RMSNORM_ERR_ALIAS;

    RopeParams p = {};
    p.part[0] = rows_of(q);
    p.part[1] = rows_of(k);
    p.turn = turn_of(rot);
    p.rstd = rstd;
    p.T = T;
    p.D = (int)D;
    p.eps = eps;
    p.inv_d = 1.f / (float)D;
    Strided rows[4];
    int n = 0;
    for (const RopeRows &r : {p.part[0], p.part[1]})
        if (r.heads) {
            rows[n++] = {r.x, T > 1 ? r.xt : 0, r.heads > 1 ? r.xh : 0, 0};
            rows[n++] = {r.y, T > 1 ? r.yt : 0, r.heads > 1 ? r.yh : 0, 0};
        }
    const RopeSet &set = rope_set(dtype);
    const RopeKernel &kern = set.k[pick_packs(set, D, p.turn, es, rows, n, q->w, wk)];
    return launch_rows(p, kern, 0, static_cast<cudaStream_t>(stream));
}

size_t rmsnorm_rope_bwd_workspace_bytes(int64_t D)
{
    int dev, sms;
    if (D < 1 || D > RMSNORM_ROPE_MAX_D || current_device(&dev) || sm_count(dev, &sms))
        return 0;
    return (size_t)sms * kBwdCtasPerSm * (size_t)D * 4;
}

int rmsnorm_rope_bwd(const rmsnorm_heads_grad *q, const rmsnorm_heads_grad *k, const rmsnorm_rotation *rot,
                     const float *rstd, void *workspace, size_t workspace_bytes, int64_t T, int64_t D, float eps,
                     int dtype, void *stream)
{
    int st = check_rope(rot, T, D, eps, dtype);
    if (st)
        return st;
    if (!q)
        return RMSNORM_ERR_NULLPTR;
    const rmsnorm_heads_grad *parts[2] = {q, k};    // (k without heads: its dw is zero)
    const size_t es = elem_size(dtype);
    if (q->heads < 1 || (k && k->heads < 0))
        return RMSNORM_ERR_BAD_SHAPE;
    const Span none = {nullptr, 0, 0, 0};
    Span sy[2] = {none, none}, sx[2] = {none, none}, sd[2] = {none, none}, sw[2] = {none, none};
    bool any_norm = false;
    for (int i = 0; i < 2; ++i) {
        const rmsnorm_heads_grad *r = parts[i];
        if (r == nullptr)
            continue;
        if (r->heads > INT32_MAX / 2)
            return RMSNORM_ERR_UNSUPPORTED;
        const bool norm = r->w != nullptr;
        any_norm |= norm;
        if (r->heads > 0 && (!rows_within({T, r->heads, 1}, {r->dy_token, r->dy_head, 0}, D) ||
                             (norm && !rows_within({T, r->heads, 1}, {r->x_token, r->x_head, 0}, D)) ||
                             !rows_apart({T, r->heads, 1}, {r->dx_token, r->dx_head, 0}, D)))
            return RMSNORM_ERR_BAD_STRIDE;
        if (norm && !r->dw)
            return RMSNORM_ERR_NULLPTR;
        if (!aligned(r->dw, 4))
            return RMSNORM_ERR_MISALIGNED;
        if (norm)
            sw[i] = flat(r->dw, (size_t)D * 4);
        if (T == 0 || r->heads == 0)
            continue;
        if (!r->dy || !r->dx || (norm && !r->x))
            return RMSNORM_ERR_NULLPTR;
        if (!aligned(r->dy, es) || !aligned(r->dx, es) || !aligned(r->x, es) || !aligned(r->w, es))
            return RMSNORM_ERR_MISALIGNED;
        sy[i] = heads_span(r->dy, T, r->heads, D, r->dy_token, r->dy_head, es);
        if (norm)
            sx[i] = heads_span(r->x, T, r->heads, D, r->x_token, r->x_head, es);
        sd[i] = heads_span(r->dx, T, r->heads, D, r->dx_token, r->dx_head, es);
    }
    if (T == 0 && !any_norm)
        return RMSNORM_OK;
    if (!aligned(rstd, 4) || !aligned(workspace, 16))
        return RMSNORM_ERR_MISALIGNED;
    int dev, sms;
    const int64_t Hk = parts[1] ? parts[1]->heads : 0, H = q->heads + Hk;
    const Span ss = flat(rstd, (size_t)(T * H) * 4);
    const Span wsp = any_norm ? flat(workspace, workspace_bytes) : none;
    const void *w0 = q->w, *w1 = parts[1] ? parts[1]->w : nullptr;
    for (int i = 0; i < 2; ++i) {
        const int j = 1 - i;
        const rmsnorm_heads_grad *r = parts[i];
        if ((r && (!heads_same_or_disjoint(sd[i], r->dx_token, r->dx_head, sy[i], r->dy_token, r->dy_head, T,
                                           r->heads) ||
                   !heads_same_or_disjoint(sd[i], r->dx_token, r->dx_head, sx[i], r->x_token, r->x_head, T,
                                           r->heads))) ||
            overlap(sd[i], sy[j]) || overlap(sd[i], sx[j]) || overlap(sd[i], ss) ||
            touches_inputs(sd[i], rot, T, D, es, w0, w1))
            return RMSNORM_ERR_ALIAS;
        for (Span o : {sd[0], sd[1], sy[0], sy[1], sx[0], sx[1], ss})
            if (overlap(sw[i], o) || overlap(wsp, o))
                return RMSNORM_ERR_ALIAS;
        if (overlap(sw[i], wsp) || touches_inputs(sw[i], rot, T, D, es, w0, w1))
            return RMSNORM_ERR_ALIAS;
    }
    if (overlap(sd[0], sd[1]) || overlap(sw[0], sw[1]) || touches_inputs(wsp, rot, T, D, es, w0, w1))
        return RMSNORM_ERR_ALIAS;
    if (any_norm && (workspace == nullptr || workspace_bytes < rmsnorm_rope_bwd_workspace_bytes(D)))
        return RMSNORM_ERR_WORKSPACE;

    RopeGradParams p = {};
    Strided rows[6];
    int n = 0;
    for (int i = 0; i < 2; ++i) {
        const rmsnorm_heads_grad *r = parts[i];
        if (r == nullptr)
            continue;
        p.part[i] = {r->dy, r->dy_token, r->dy_head, r->x, r->x_token, r->x_head, r->w,
                     r->dx, r->dx_token, r->dx_head, r->dw, (int)r->heads, 0};
        if (r->heads == 0)
            continue;
        const int64_t t = T > 1, h = r->heads > 1;
        rows[n++] = {r->dy, t * r->dy_token, h * r->dy_head, 0};
        rows[n++] = {r->dx, t * r->dx_token, h * r->dx_head, 0};
        if (r->w)
            rows[n++] = {r->x, t * r->x_token, h * r->x_head, 0};
    }
    p.turn = turn_of(rot);
    p.rstd = rstd;
    p.partial = static_cast<float *>(workspace);
    p.T = T;
    p.D = (int)D;
    p.eps = eps;
    p.inv_d = 1.f / (float)D;
    const RopeSet &set = rope_set(dtype);
    const RopeKernel &kern = set.k[pick_packs(set, D, p.turn, es, rows, n, w0, w1)];
    const void *fn = kern.bwd[p.turn.adjacent];
    int bps;
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)) ||
        (st = blocks_per_sm(fn, kRopeThreads, dev, &bps, kern.bwd_smem)))
        return st;
    p.shift = lane_shift(kern.E, D);
    const int64_t per = kRopeThreads >> p.shift;
    const int64_t most = (int64_t)sms * std::min(bps, kBwdCtasPerSm);
    p.HC = piece(T, {q->heads, Hk}, most * per);
    int64_t need[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        p.part[i].chunks = (p.part[i].heads + p.HC - 1) / p.HC;
        need[i] = (T * p.part[i].chunks + per - 1) / per;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t cq = need[0], ck = need[1];
    if (cq + ck > most) {
        // shares by heads, at least one CTA each
        cq = std::max<int64_t>(1, std::min<int64_t>(most * q->heads / H, most - (Hk ? 1 : 0)));
        ck = Hk ? most - cq : 0;
    }
    p.ctas_q = (int)cq;
    const int ctas = (int)(cq + ck);
    if (ctas > 0) {
        void *args[1] = {&p};
        const cudaError_t e = launch_pdl(fn, dim3((unsigned)ctas), kRopeThreads, (size_t)kern.bwd_smem, s, args);
        if (e != cudaSuccess)
            return cuda_fail(e);
    }
    if (any_norm) {
        const float *part = p.partial;
        int c0 = p.ctas_q, c1 = ctas, d = (int)D;
        float *dw0 = q->w ? q->dw : nullptr, *dw1 = w1 ? parts[1]->dw : nullptr;
        void *args[6] = {&part, &c0, &c1, &d, &dw0, &dw1};
        const cudaError_t e = launch_pdl(rope_dw_kernel, dim3((unsigned)((D + 31) / 32), 2), 1024, 0, s, args);
        if (e != cudaSuccess)
            return cuda_fail(e);
    }
    t_last_path = kPathRope;
    return RMSNORM_OK;
}

int rmsnorm_rope_append(const rmsnorm_heads *q, const rmsnorm_heads *k, const rmsnorm_heads *v,
                        const rmsnorm_rotation *rot, const void *slots, int slot_bits, int64_t pages,
                        int64_t page_size, int64_t k_page, int64_t v_page, int64_t T, int64_t D, float eps,
                        int dtype, void *stream)
{
    const CacheArgs c = {false, pages, page_size, k_page, v_page, nullptr, nullptr};
    return append_impl(q, k, v, rot, slots, slot_bits, c, T, D, eps, dtype, static_cast<cudaStream_t>(stream));
}

int rmsnorm_rope_append_kv4(const rmsnorm_heads *q, const rmsnorm_heads *k, const rmsnorm_heads *v,
                            const rmsnorm_rotation *rot, const void *slots, int slot_bits, void *cache,
                            int64_t pages, int64_t page_size, const float *k_scale, const float *v_scale,
                            int64_t T, int64_t D, float eps, int dtype, void *stream)
{
    if (!k || !v)
        return RMSNORM_ERR_NULLPTR;
    rmsnorm_heads kk = *k, vv = *v;
    kk.y = vv.y = cache;
    const CacheArgs c = {true, pages, page_size, 0, 0, k_scale, v_scale};
    return append_impl(q, &kk, &vv, rot, slots, slot_bits, c, T, D, eps, dtype, static_cast<cudaStream_t>(stream));
}

int rmsnorm_kv4_read(const void *cache, int64_t pages, int64_t page_size, int64_t heads, int64_t D,
                     const void *slots, int slot_bits, int64_t n, void *k, void *k_scale, void *v, void *v_scale,
                     void *stream)
{
    if (!index_bits_ok(slot_bits))
        return RMSNORM_ERR_BAD_DTYPE;
    if (pages < 0 || page_size < 1 || heads < 1 || n < 0)
        return RMSNORM_ERR_BAD_SHAPE;
    if ((D != 64 && D != 128) || page_size % kKv4Tile || page_size > INT32_MAX || heads > INT32_MAX / 64 ||
        pages > (INT64_MAX >> 10) / page_size / heads || n > INT32_MAX)
        return RMSNORM_ERR_UNSUPPORTED;
    if (n == 0)
        return RMSNORM_OK;
    if ((!cache && pages) || !slots || !k || !k_scale || !v || !v_scale)
        return RMSNORM_ERR_NULLPTR;
    if (!aligned(cache, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, slot_bits / 8))
        return RMSNORM_ERR_MISALIGNED;
    const size_t rows = (size_t)(n * heads * D);
    const Span out[4] = {flat(k, rows), flat(k_scale, rows / 16), flat(v, rows), flat(v_scale, rows / 16)};
    const Span in[2] = {flat(cache, (size_t)(pages * page_size * heads * (D * 9 / 8))),
                        flat(slots, (size_t)n * slot_bits / 8)};
    for (int i = 0; i < 4; ++i) {
        if (overlap(out[i], in[0]) || overlap(out[i], in[1]))
            return RMSNORM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return RMSNORM_ERR_ALIAS;
    }
    Kv4ReadParams p = {static_cast<const uint8_t *>(cache), slots, slot_bits == 64 ? 1 : 0, (int)heads, (int)D,
                       page_size, pages * page_size, n, static_cast<uint8_t *>(k), static_cast<uint8_t *>(k_scale),
                       static_cast<uint8_t *>(v), static_cast<uint8_t *>(v_scale)};
    int dev, sms, st;
    if ((st = current_device(&dev)) || (st = sm_count(dev, &sms)))
        return st;
    const int64_t ctas = std::min<int64_t>((n * heads * (D / 8) + 255) / 256, (int64_t)sms * 8);
    void *args[1] = {&p};
    const cudaError_t e = launch_pdl(kv4_read_kernel, dim3((unsigned)ctas), 256, 0,
                                     static_cast<cudaStream_t>(stream), args);
    if (e != cudaSuccess)
        return cuda_fail(e);
    t_last_path = kPathKv4Read;
    return RMSNORM_OK;
}

} // extern "C"
