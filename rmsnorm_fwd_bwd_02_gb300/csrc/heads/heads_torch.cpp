// heads_torch.cpp -- the Python binding of the entry points on attention heads
// (module _heads_torch): checks torch tensors, allocates the outputs that the
// caller did not pass, and calls the C ABI on the current stream. In C++ for
// its time on the host, as the 8-bit calls': these calls take a few
// microseconds on the GPU in a decode step.
//
// The module does not link the library: rmsnorm.py hands it the functions'
// addresses and the Python function that raises a status.
#include "../torch/binding.h"

#include <algorithm>
#include <cmath>

namespace {

decltype(&rmsnorm_rope_fwd) g_fwd = nullptr;
decltype(&rmsnorm_rope_bwd) g_bwd = nullptr;
decltype(&rmsnorm_rope_bwd_workspace_bytes) g_bwd_bytes = nullptr;
decltype(&rmsnorm_rope_append) g_append = nullptr;
decltype(&rmsnorm_rope_append_kv4) g_append4 = nullptr;
decltype(&rmsnorm_kv4_read) g_read = nullptr;
decltype(&rmsnorm_kv4_attention) g_attend = nullptr;
decltype(&rmsnorm_kv4_attention_workspace_bytes) g_attend_bytes = nullptr;

void on_cuda(const Tensor &t, const char *name)
{
    if (!t.is_cuda())
        refuse(c10::str(name, " must be a CUDA tensor, got ", t.device()));
}

// The strides of heads [T, H, D] with unit feature stride.
void heads(const Tensor &t, const char *name, int64_t T, int64_t H, int64_t D, ScalarType dtype, at::Device dev,
           int64_t &token, int64_t &head)
{
    on_device(t, name, dev);
    if (t.scalar_type() != dtype)
        refuse(c10::str(name, " must be ", dtype, ", got ", t.scalar_type()));
    if (t.dim() != 3 || t.size(0) != T || (H >= 0 && t.size(1) != H) || t.size(2) != D)
        refuse(c10::str(name, " must be of shape [", T, ", ", H < 0 ? std::string("heads") : std::to_string(H),
                        ", ", D, "], got ", t.sizes()));
    if (t.stride(2) != 1 && D > 1)
        refuse(c10::str(name, " must have unit stride over a head's features"));
    head = t.size(1) > 1 ? t.stride(1) : D;
    token = T > 1 ? t.stride(0) : t.size(1) * D;
}

const void *weight(const Tensor *w, const char *name, int64_t D, ScalarType dtype, at::Device dev)
{
    if (w == nullptr)
        return nullptr;
    on_device(*w, name, dev);
    if (w->scalar_type() != dtype || w->numel() != D || !w->is_contiguous())
        refuse(c10::str(name, " must be a contiguous ", dtype, " tensor of ", D, " elements, got ",
                        w->scalar_type(), " ", w->sizes()));
    return w->data_ptr();
}

// int32 or int64 of one dimension
int index_bits(const Tensor &t, const char *name, int64_t n, at::Device dev)
{
    on_device(t, name, dev);
    if ((t.scalar_type() != at::kInt && t.scalar_type() != at::kLong) || t.dim() != 1 || t.size(0) != n ||
        !t.is_contiguous())
        refuse(c10::str(name, " must be a contiguous int32 or int64 tensor of shape [", n, "], got ",
                        t.scalar_type(), " ", t.sizes()));
    return t.scalar_type() == at::kLong ? 64 : 32;
}

rmsnorm_rotation rotation(PyObject *positions, PyObject *freq, PyObject *interleaved, PyObject *amplitude,
                          int64_t T, at::Device dev)
{
    rmsnorm_rotation r = {};
    const Tensor *p = optional(positions, "positions"), *f = optional(freq, "freq");
    if ((p == nullptr) != (f == nullptr))
        refuse("positions and freq come together, or both are None (no rotation)");
    r.position_bits = 32;
    r.amplitude = 1.f;
    if (p == nullptr)
        return r;
    r.position_bits = index_bits(*p, "positions", T, dev);
    r.positions = p->data_ptr();
    on_device(*f, "freq", dev);
    if (f->scalar_type() != at::kDouble || f->dim() != 1 || !f->is_contiguous())
        refuse(c10::str("freq must be a contiguous float64 tensor of one dimension, got ", f->scalar_type(), " ",
                        f->sizes()));
    r.freq = static_cast<const double *>(f->data_ptr());
    r.rot = 2 * f->size(0);
    const int adjacent = PyObject_IsTrue(interleaved);
    const double amp = PyFloat_AsDouble(amplitude);
    if (adjacent < 0 || (amp == -1.0 && PyErr_Occurred()))
        throw python_error();
    r.adjacent = adjacent;
    r.amplitude = (float)amp;
    return r;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

// Heads in and out; the output is made where none was passed.
struct Part {
    rmsnorm_heads h = {};
    Tensor out;                    // what was made
};

void part_in(Part &p, const Tensor &x, const char *name, const Tensor *w, const char *wname, int64_t T, int64_t D,
             ScalarType dtype, at::Device dev)
{
    heads(x, name, T, -1, D, dtype, dev, p.h.x_token, p.h.x_head);
    p.h.x = x.data_ptr();
    p.h.heads = x.size(1);
    p.h.w = weight(w, wname, D, dtype, dev);
}

void part_out(Part &p, const Tensor *y, const char *name, Outputs &made, int64_t T, int64_t D, ScalarType dtype,
              at::Device dev)
{
    const int64_t H = p.h.heads;
    if (y == nullptr)
        p.out = made.dense({T, H, D}, dtype);
    const Tensor &t = y ? *y : p.out;
    heads(t, name, T, H, D, dtype, dev, p.h.y_token, p.h.y_head);
    p.h.y = t.data_ptr();
}

size_t bytes_of(int64_t n, ScalarType t) { return Outputs::bytes(1, n, t); }

PyObject *given(PyObject *in, const Tensor &made)
{
    return in != Py_None ? Py_NewRef(in) : THPVariable_Wrap(made);
}

void *stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

void three_d(const Tensor &t, const char *name)
{
    if (t.dim() != 3)
        refuse(c10::str(name, " must be 3-D [tokens, heads, features], got ", t.sizes()));
    on_cuda(t, name);
}

// rope_fwd(q, positions, freq, k, wq, wk, yq, yk, eps, interleaved, amplitude, want_rstd)
PyObject *rope_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 12))
        return nullptr;
    const Tensor &q = tensor(a[0], "q");
    const Tensor *k = optional(a[3], "k"), *wq = optional(a[4], "wq"), *wk = optional(a[5], "wk"),
                 *yq = optional(a[6], "yq"), *yk = optional(a[7], "yk");
    const double eps = number(a[8]);
    const int want = PyObject_IsTrue(a[11]);
    if (want < 0)
        return nullptr;
    three_d(q, "q");
    if (k == nullptr && (wk || yk))
        refuse("wk and yk belong to k: pass k too");
    const int64_t T = q.size(0), D = q.size(2);
    const ScalarType dtype = q.scalar_type();
    const int code = row_code(dtype);
    const at::Device dev = q.device();
    const rmsnorm_rotation r = rotation(a[1], a[2], a[9], a[10], T, dev);
    Part pq, pk;
    part_in(pq, q, "q", wq, "wq", T, D, dtype, dev);
    if (k)
        part_in(pk, *k, "k", wk, "wk", T, D, dtype, dev);
    const bool new_rstd = want && (wq || wk);
    const int64_t H = pq.h.heads + pk.h.heads;

    const c10::cuda::CUDAGuard guard(dev);
    // rstd has an allocation of its own: torch.save refuses tensors of two types in one storage
    Outputs made((yq ? 0 : bytes_of(q.numel(), dtype)) + (k && !yk ? bytes_of(k->numel(), dtype) : 0));
    part_out(pq, yq, "yq", made, T, D, dtype, dev);
    if (k)
        part_out(pk, yk, "yk", made, T, D, dtype, dev);
    const Tensor rstd = new_rstd ? Outputs().dense({T, H}, at::kFloat) : Tensor();
    const int st = g_fwd(&pq.h, k ? &pk.h : nullptr, &r,
                         new_rstd ? static_cast<float *>(rstd.data_ptr()) : nullptr, T, D, (float)eps, code,
                         stream_of(dev));
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_rope_fwd");
    PyObject *out = PyTuple_New(3);
    if (out == nullptr)
        return nullptr;
    PyTuple_SET_ITEM(out, 0, given(a[6], pq.out));
    PyTuple_SET_ITEM(out, 1, given(a[7], pk.out));
    PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(rstd));
    return out;
    END_HANDLE_TH_ERRORS
}

// rope_bwd(dyq, q, positions, freq, dyk, k, wq, wk, rstd, dq, dk, eps, interleaved, amplitude)
PyObject *rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 14))
        return nullptr;
    const Tensor &dyq = tensor(a[0], "dyq");
    const Tensor *q = optional(a[1], "q"), *dyk = optional(a[4], "dyk"), *k = optional(a[5], "k"),
                 *wq = optional(a[6], "wq"), *wk = optional(a[7], "wk"), *rstd = optional(a[8], "rstd"),
                 *dq = optional(a[9], "dq"), *dk = optional(a[10], "dk");
    const double eps = number(a[11]);
    three_d(dyq, "dyq");
    if (dyk == nullptr && (wk || dk || k))
        refuse("k, wk and dk belong to dyk: pass dyk too");
    const int64_t T = dyq.size(0), D = dyq.size(2);
    const ScalarType dtype = dyq.scalar_type();
    const int code = row_code(dtype);
    const at::Device dev = dyq.device();
    const rmsnorm_rotation r = rotation(a[2], a[3], a[12], a[13], T, dev);
    rmsnorm_heads_grad g[2] = {};
    const Tensor *dy[2] = {&dyq, dyk}, *x[2] = {q, k}, *w[2] = {wq, wk}, *dx[2] = {dq, dk};
    static const char *const kDy[2] = {"dyq", "dyk"}, *const kX[2] = {"q", "k"}, *const kW[2] = {"wq", "wk"},
                                   *const kDx[2] = {"dq", "dk"};
    size_t total = 0, small = 0;
    for (int i = 0; i < 2; ++i) {
        if (dy[i] == nullptr)
            continue;
        heads(*dy[i], kDy[i], T, -1, D, dtype, dev, g[i].dy_token, g[i].dy_head);
        g[i].dy = dy[i]->data_ptr();
        g[i].heads = dy[i]->size(1);
        g[i].w = weight(w[i], kW[i], D, dtype, dev);
        if (g[i].w && x[i] == nullptr)
            refuse(c10::str(kX[i], " is needed for the gradient of its norm"));
        if (x[i]) {
            heads(*x[i], kX[i], T, g[i].heads, D, dtype, dev, g[i].x_token, g[i].x_head);
            g[i].x = x[i]->data_ptr();
        }
        total += dx[i] ? 0 : bytes_of(dy[i]->numel(), dtype);
        small += w[i] ? bytes_of(D, at::kFloat) : 0;
    }
    const int64_t H = g[0].heads + g[1].heads;
    if (rstd)
        fp32(*rstd, "rstd", {T, H}, dev);

    const c10::cuda::CUDAGuard guard(dev);
    Outputs made(total), sums(small);       // the weights' gradients share an allocation
    Tensor out_dx[2], out_dw[2];
    for (int i = 0; i < 2; ++i) {
        if (dy[i] == nullptr)
            continue;
        if (dx[i] == nullptr)
            out_dx[i] = made.dense({T, g[i].heads, D}, dtype);
        const Tensor &t = dx[i] ? *dx[i] : out_dx[i];
        heads(t, kDx[i], T, g[i].heads, D, dtype, dev, g[i].dx_token, g[i].dx_head);
        g[i].dx = t.data_ptr();
        if (w[i]) {
            out_dw[i] = sums.dense({D}, at::kFloat);
            g[i].dw = static_cast<float *>(out_dw[i].data_ptr());
        }
    }
    // the workspace is the call's own: memory of this stream, free again for
    // what runs behind it
    const size_t need = wq || wk ? g_bwd_bytes(D) : 0;
    const Tensor ws = need ? Outputs().dense({(int64_t)need}, at::kByte) : Tensor();
    const int st = g_bwd(&g[0], dyk ? &g[1] : nullptr, &r,
                         rstd ? static_cast<const float *>(rstd->data_ptr()) : nullptr,
                         need ? ws.data_ptr() : nullptr, need, T, D, (float)eps, code, stream_of(dev));
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_rope_bwd");
    PyObject *out = PyTuple_New(4);
    if (out == nullptr)
        return nullptr;
    for (int i = 0; i < 2; ++i) {
        PyTuple_SET_ITEM(out, i, given(a[9 + i], out_dx[i]));
        PyTuple_SET_ITEM(out, 2 + i, THPVariable_Wrap(out_dw[i]));
    }
    return out;
    END_HANDLE_TH_ERRORS
}

// The sizes of a 4-bit cache [pages, heads, page_size / 16, 18 D].
struct Cache4 {
    int64_t pages, page_size, D;
};

Cache4 cache4(const Tensor &c, const char *name, int64_t H, at::Device dev)
{
    on_device(c, name, dev);
    if (c.scalar_type() != at::kByte || c.dim() != 4 || !c.is_contiguous() || (H >= 0 && c.size(1) != H) ||
        c.size(3) % 18)
        refuse(c10::str(name, " must be a contiguous uint8 tensor of shape [pages, ",
                        H < 0 ? std::string("heads") : std::to_string(H),
                        ", page_size / 16, 18 * head_dim], got ", c.scalar_type(), " ", c.sizes()));
    return {c.size(0), c.size(2) * 16, c.size(3) / 18};
}

const float *head_scale(const Tensor *t, const char *name, int64_t H, at::Device dev)
{
    return t ? fp32(*t, name, {H}, dev) : nullptr;
}

// append(k, v, positions, freq, slots, cache_k, cache_v, q, wq, wk, yq, eps, interleaved, amplitude, k_scale,
// v_scale, bits4): with bits4 cache_k is the 4-bit cache and cache_v None
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 17))
        return nullptr;
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[4], "slots");
    const Tensor *q = optional(a[7], "q"), *wq = optional(a[8], "wq"), *wk = optional(a[9], "wk"),
                 *yq = optional(a[10], "yq"), *ks = optional(a[14], "k_scale"), *vs = optional(a[15], "v_scale");
    const double eps = number(a[11]);
    const bool bits4 = a[16] == Py_True;
    three_d(k, "k");
    if (q == nullptr && (wq || yq))
        refuse("wq and yq belong to q: pass q too");
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2);
    const ScalarType dtype = k.scalar_type();
    const int code = row_code(dtype);
    const at::Device dev = k.device();
    const rmsnorm_rotation r = rotation(a[2], a[3], a[12], a[13], T, dev);
    Part pq, pk, pv;
    part_in(pk, k, "k", wk, "wk", T, D, dtype, dev);
    part_in(pv, v, "v", nullptr, "", T, D, dtype, dev);
    if (pv.h.heads != H)
        refuse(c10::str("v must be of shape ", k.sizes(), ", got ", v.sizes()));
    if (q)
        part_in(pq, *q, "q", wq, "wq", T, D, dtype, dev);
    const int slot_bits = index_bits(slots, "slots", T, dev);
    int64_t pages = 0, page_size = 0, page[2] = {0, 0};
    void *cache = nullptr;
    if (bits4) {
        const Tensor &c = tensor(a[5], "cache");
        const Cache4 s = cache4(c, "cache", H, dev);
        if (s.D != D)
            refuse(c10::str("cache has heads of ", s.D, " features, k of ", D));
        pages = s.pages;
        page_size = s.page_size;
        cache = c.data_ptr();
    } else {
        const Tensor *c[2] = {&tensor(a[5], "cache_k"), &tensor(a[6], "cache_v")};
        static const char *const kName[2] = {"cache_k", "cache_v"};
        for (int i = 0; i < 2; ++i) {
            const Tensor &t = *c[i];
            on_device(t, kName[i], dev);
            if (t.scalar_type() != dtype || t.dim() != 4 || t.size(2) != H || t.size(3) != D ||
                (t.stride(3) != 1 && D > 1) || t.sizes() != c[0]->sizes())
                refuse(c10::str(kName[i], " must be a ", dtype, " tensor of shape [pages, page_size, ", H, ", ", D,
                                "] with unit stride over a head's features, got ", t.scalar_type(), " ",
                                t.sizes()));
            rmsnorm_heads &h = i ? pv.h : pk.h;
            h.y = t.data_ptr();
            h.y_head = H > 1 ? t.stride(2) : D;
            h.y_token = t.size(1) > 1 ? t.stride(1) : H * D;
            page[i] = t.size(0) > 1 ? t.stride(0) : t.size(1) * H * D;
        }
        pages = c[0]->size(0);
        page_size = c[0]->size(1);
    }
    const float *ksp = head_scale(ks, "k_scale", H, dev), *vsp = head_scale(vs, "v_scale", H, dev);

    const c10::cuda::CUDAGuard guard(dev);
    Outputs made;
    if (q)
        part_out(pq, yq, "yq", made, T, D, dtype, dev);
    const rmsnorm_heads *hq = q ? &pq.h : nullptr;
    const int st = bits4 ? g_append4(hq, &pk.h, &pv.h, &r, slots.data_ptr(), slot_bits, cache, pages, page_size,
                                     ksp, vsp, T, D, (float)eps, code, stream_of(dev))
                         : g_append(hq, &pk.h, &pv.h, &r, slots.data_ptr(), slot_bits, pages, page_size, page[0],
                                    page[1], T, D, (float)eps, code, stream_of(dev));
    if (st != RMSNORM_OK)
        return raised(st, bits4 ? "rmsnorm_rope_append_kv4" : "rmsnorm_rope_append");
    return given(a[10], pq.out);
    END_HANDLE_TH_ERRORS
}

// kv4_read(cache, slots)
PyObject *kv4_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 2))
        return nullptr;
    const Tensor &c = tensor(a[0], "cache"), &slots = tensor(a[1], "slots");
    on_cuda(c, "cache");
    const at::Device dev = c.device();
    const Cache4 s = cache4(c, "cache", -1, dev);
    const int64_t N = slots.dim() == 1 ? slots.size(0) : -1, H = c.size(1), D = s.D;
    const int bits = index_bits(slots, "slots", N, dev);
    const c10::cuda::CUDAGuard guard(dev);
    Outputs made(2 * (bytes_of(N * H * D, at::kByte) + bytes_of(N * H * D / 16, at::kByte)));
    Tensor out[4];
    for (int i = 0; i < 4; ++i)
        out[i] = made.dense({N, H, i % 2 ? D / 16 : D}, at::kFloat8_e4m3fn);
    const int st = g_read(c.data_ptr(), s.pages, s.page_size, H, D, slots.data_ptr(), bits, N, out[0].data_ptr(),
                          out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), stream_of(dev));
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_kv4_read");
    PyObject *r = PyTuple_New(4);
    if (r == nullptr)
        return nullptr;
    for (int i = 0; i < 4; ++i)
        PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
    return r;
    END_HANDLE_TH_ERRORS
}

// A contiguous int32 tensor of one dimension.
const int *int32s(const Tensor &t, const char *name, int64_t n, at::Device dev)
{
    on_device(t, name, dev);
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(c10::str(name, " must be a contiguous int32 tensor of shape [", n, "], got ", t.scalar_type(), " ",
                        t.sizes()));
    return static_cast<const int *>(t.data_ptr());
}

// kv4_attention(q, cache, block_table, seq_lens, q_starts, k_scale, v_scale, scale, out, lse, want_lse, workspace)
PyObject *kv4_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 12))
        return nullptr;
    const Tensor &q = tensor(a[0], "q"), &c = tensor(a[1], "cache"), &table = tensor(a[2], "block_table"),
                 &lens = tensor(a[3], "seq_lens");
    const Tensor *starts = optional(a[4], "q_starts"), *ks = optional(a[5], "k_scale"),
                 *vs = optional(a[6], "v_scale"), *out_in = optional(a[8], "out"), *lse_in = optional(a[9], "lse"),
                 *ws_in = optional(a[11], "workspace");
    const int want = PyObject_IsTrue(a[10]);
    if (want < 0)
        return nullptr;
    three_d(q, "q");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const ScalarType dtype = q.scalar_type();
    const int code = row_code(dtype);
    const at::Device dev = q.device();
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)std::max<int64_t>(D, 1)) : number(a[7]);
    int64_t qt, qh;
    heads(q, "q", T, H, D, dtype, dev, qt, qh);
    const Cache4 s = cache4(c, "cache", -1, dev);
    const int64_t Hk = c.size(1);
    if (s.D != D)
        refuse(c10::str("cache has heads of ", s.D, " features, q of ", D));
    on_device(table, "block_table", dev);
    if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
        refuse(c10::str("block_table must be an int32 tensor of shape [sequences, blocks] with unit stride over "
                        "its blocks, got ", table.scalar_type(), " ", table.sizes()));
    const int64_t B = table.size(0), blocks = table.size(1), ld = B > 1 ? table.stride(0) : blocks;
    const int *lensp = int32s(lens, "seq_lens", B, dev);
    const int *startsp = starts ? int32s(*starts, "q_starts", B + 1, dev) : nullptr;
    if (!starts && T != B)
        refuse(c10::str("q has ", T, " tokens for ", B, " sequences: pass q_starts"));
    const float *ksp = head_scale(ks, "k_scale", Hk, dev), *vsp = head_scale(vs, "v_scale", Hk, dev);
    int64_t ot = H * D, oh = D;
    if (out_in)
        heads(*out_in, "out", T, H, D, dtype, dev, ot, oh);
    if (lse_in)
        fp32(*lse_in, "lse", {T, H}, dev);
    if (ws_in) {
        on_device(*ws_in, "workspace", dev);
        if (!ws_in->is_contiguous())
            refuse("workspace must be contiguous");
    }

    const c10::cuda::CUDAGuard guard(dev);
    const bool new_lse = want && !lse_in;
    const Tensor out = out_in ? *out_in : Outputs().dense({T, H, D}, dtype);
    const Tensor lse = lse_in ? *lse_in : new_lse ? Outputs().dense({T, H}, at::kFloat) : Tensor();
    // the call's own memory of this stream, free again for what runs behind it
    const Tensor ws = ws_in ? *ws_in : Outputs().dense({(int64_t)g_attend_bytes(D)}, at::kByte);
    const int st = g_attend(q.data_ptr(), qt, qh, out.data_ptr(), ot, oh,
                            lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr, c.data_ptr(), s.pages,
                            s.page_size, Hk, ksp, vsp, static_cast<const int *>(table.data_ptr()), ld, blocks,
                            lensp, startsp, B, T, H, D, (float)scale, ws.data_ptr(), ws.nbytes(), code,
                            stream_of(dev));
    if (st != RMSNORM_OK)
        return raised(st, "rmsnorm_kv4_attention");
    PyObject *r = PyTuple_New(2);
    if (r == nullptr)
        return nullptr;
    PyTuple_SET_ITEM(r, 0, given(a[8], out));
    PyTuple_SET_ITEM(r, 1, given(a[9], lse));
    return r;
    END_HANDLE_TH_ERRORS
}

// init(addresses of rope_fwd, rope_bwd, rope_bwd_workspace_bytes, rope_append, rope_append_kv4, kv4_read,
// kv4_attention, kv4_attention_workspace_bytes, check)
PyObject *init(PyObject *, PyObject *args)
{
    unsigned long long f[8];
    PyObject *check;
    if (!PyArg_ParseTuple(args, "KKKKKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7],
                          &check))
        return nullptr;
    g_fwd = reinterpret_cast<decltype(g_fwd)>((uintptr_t)f[0]);
    g_bwd = reinterpret_cast<decltype(g_bwd)>((uintptr_t)f[1]);
    g_bwd_bytes = reinterpret_cast<decltype(g_bwd_bytes)>((uintptr_t)f[2]);
    g_append = reinterpret_cast<decltype(g_append)>((uintptr_t)f[3]);
    g_append4 = reinterpret_cast<decltype(g_append4)>((uintptr_t)f[4]);
    g_read = reinterpret_cast<decltype(g_read)>((uintptr_t)f[5]);
    g_attend = reinterpret_cast<decltype(g_attend)>((uintptr_t)f[6]);
    g_attend_bytes = reinterpret_cast<decltype(g_attend_bytes)>((uintptr_t)f[7]);
    Py_INCREF(check);
    Py_XSETREF(g_check, check);
    Py_RETURN_NONE;
}

template <typename F> PyCFunction as_function(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"rope_fwd", as_function(rope_fwd), METH_FASTCALL, nullptr},
                         {"rope_bwd", as_function(rope_bwd), METH_FASTCALL, nullptr},
                         {"append", as_function(append), METH_FASTCALL, nullptr},
                         {"kv4_read", as_function(kv4_read), METH_FASTCALL, nullptr},
                         {"kv4_attention", as_function(kv4_attention), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_heads_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__heads_torch() { return PyModule_Create(&module); }
