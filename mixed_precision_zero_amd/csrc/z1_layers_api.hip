// z1_layers_api.hip -- host side of the layers declared in
// include/z1_layers.h: argument validation, the shapes of the products and of
// their workspaces, and the launches.
#include <algorithm>
#include <initializer_list>

#include "z1_host.h"
#include "z1_layers.h"
#include "z1_layers_internal.h"
#include "z1_linear_tile.h"

using namespace z1::host;
using z1::ops::Copy;
using z1::ops::Drop;
using z1::ops::Epilogue;
using z1::ops::Form;
using z1::ops::Operand;
using z1::ops::pad_to;
using z1::ops::Product;

namespace {

bool drop_ok(const z1_drop &d) { return d.p >= 0.0 && d.p <= 1.0; }

Drop drop_of(const z1_drop &d)
{
    const uint32_t threshold = (uint32_t)rint(d.p * 65536.0);
    if (!d.rng || d.p == 0.0)
        return Drop{nullptr, 0, 0, 1.f};
    return Drop{d.rng, d.offset, threshold, threshold == 65536 ? 0.f : (float)(65536.0 / (65536.0 - threshold))};
}

z1_status status_of(hipError_t e) { return e == hipSuccess ? Z1_OK : Z1_EHIP; }
hipStream_t hip(z1_stream s) { return reinterpret_cast<hipStream_t>(s); }

// A matrix of a call: null (where it may be), or rows that do not overlap.
bool rows_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, bool needed)
{
    if (!p)
        return !needed || rows == 0;
    return ld >= cols;
}

// Whether one of the others is this buffer.
bool among(const void *p, std::initializer_list<const void *> others)
{
    return p && std::find(others.begin(), others.end(), p) != others.end();
}

const void *read_rng(const z1_drop &d) { return d.p > 0.0 ? d.rng : nullptr; }

// A workspace of which no byte is needed is no buffer of the call.
const void *used(const void *workspace, int64_t need) { return need > 0 ? workspace : nullptr; }

// --------------------------------------------------------------------------
// Products
// --------------------------------------------------------------------------

constexpr int64_t kMostRows = INT64_C(1) << 30, kMostSide = INT64_C(1) << 20, kMostLd = INT64_C(1) << 21;

struct Matrix {
    const void *p;
    int64_t rows, cols, ld;
};

// Copied rows are padded to whole groups of eight elements.
constexpr int64_t kPackCols = 8;

// Whether a product reads the matrix where it lies: 16-byte chunks throughout.
bool in_place(const Matrix &m, int32_t dtype)
{
    const int64_t size = (int64_t)type_size(dtype);
    return aligned(m.p, 16) && (m.rows == 1 || m.ld * size % 16 == 0) && m.cols * size % 16 == 0;
}

// One product and what it takes of the workspace.
struct Plan {
    Product g{};
    bool pack_p = false, pack_q = false;
    bool fits = true;   // a launch
    int64_t at_p = 0, at_q = 0, at_parts = 0, bytes = 0;
};

Plan plan_product(Form form, int32_t dtype, const Matrix &p, const Matrix &q)
{
    Plan w;
    Product &g = w.g;
    const bool p_deep = form == z1::ops::kForward, q_deep = form != z1::ops::kWeight;
    const int64_t size = (int64_t)type_size(dtype);
    if (form == z1::ops::kForward && q.rows <= z1::ops::kRowsMost) {
        g.p = Operand{p.p, (p.rows == 1 ? p.cols : p.ld) * size, (int32_t)p.rows, (int32_t)p.cols};
        g.q = Operand{q.p, (q.rows == 1 ? q.cols : q.ld) * size, (int32_t)q.rows, (int32_t)q.cols};
        g.P = (int32_t)p.rows;
        g.Q = (int32_t)q.rows;
        return w;
    }
    const auto operand = [&](const Matrix &m, bool deep, bool &pack, int64_t &at) {
        pack = !in_place(m, dtype);
        int64_t cols = m.cols, ld = m.ld;
        if (pack) {
            cols = ld = pad_to(cols, kPackCols);
            at = w.bytes;
            w.bytes += pad_to(m.rows * cols * size, 16);
        } else if (m.rows == 1) {
            ld = cols;
        }
        return Operand{m.p, ld * size, (int32_t)(deep ? m.rows : cols), (int32_t)(deep ? cols : m.rows)};
    };
    g.q = operand(q, q_deep, w.pack_q, w.at_q);   // first: see run_product
    g.p = operand(p, p_deep, w.pack_p, w.at_p);
    g.P = (int32_t)(p_deep ? p.rows : p.cols);
    g.Q = (int32_t)(q_deep ? q.rows : q.cols);
    const int64_t bytes = std::max(g.p.depth, g.q.depth) * size;   // of depth
    const z1::ops::TileChoice c = z1::ops::pick_product(g.P, g.Q, bytes, dtype == Z1_F32);
    if (c.tile == 0) {
        w.fits = false;
        return w;
    }
    g.tile = c.tile;
    g.splits = c.splits;
    g.piece = c.piece;
    g.tiles_p = (g.P + g.tile - 1) / g.tile;
    g.tiles_q = (g.Q + g.tile - 1) / g.tile;
    if (g.splits > 1) {
        w.at_parts = w.bytes;
        w.bytes += (int64_t)g.splits * g.tiles_p * g.tiles_q * g.tile * g.tile * 4;
    }
    return w;
}

// has_q: Q's copy lies at the workspace's start from a product before this one, where any
// product puts it, whichever way it reads Q.
z1_status run_product(Form form, int32_t dtype, int32_t out_dtype, Plan &w, const Matrix &p, const Matrix &q,
                      void *workspace, hipStream_t s, bool has_q = false)
{
    Product &g = w.g;
    char *base = static_cast<char *>(workspace);
    if (g.tile == 0)
        return status_of(z1::ops::launch_rows(dtype, g, s));
    const auto copy = [&](bool pack, const Matrix &m, int64_t at, Operand &o) {
        if (!pack)
            return Copy{};
        o.base = base + at;
        return Copy{m.p, base + at, m.ld, m.rows, m.cols, pad_to(m.cols, kPackCols)};
    };
    Copy of_q = copy(w.pack_q, q, w.at_q, g.q);
    const Copy of_p = copy(w.pack_p, p, w.at_p, g.p);
    if (has_q)
        of_q = Copy{};
    hipError_t e = z1::ops::launch_pack(dtype, of_p, of_q, s);
    g.parts = reinterpret_cast<float *>(base + w.at_parts);
    if (e == hipSuccess)
        e = z1::ops::launch_product(form, dtype, out_dtype, g, s);
    return status_of(e);
}

// Sizes, types, and the operands themselves.
z1_status product_sizes(int64_t rows, int64_t in, int64_t out, int32_t dtype)
{
    return rows >= 0 && rows <= kMostRows && in >= 1 && in <= kMostSide && out >= 1 && out <= kMostSide &&
                   dtype_ok(dtype)
               ? Z1_OK
               : Z1_EINVAL;
}

bool operand_ok(const Matrix &m) { return rows_ok(m.p, m.rows, m.cols, m.ld, true) && m.ld < kMostLd; }

z1_status linear_plan(const z1_linear_args *a, Matrix &x, Matrix &weight, Plan &w)
{
    if (!a || product_sizes(a->rows, a->in, a->out, a->dtype) != Z1_OK)
        return Z1_EINVAL;
    x = Matrix{a->x, a->rows, a->in, a->ld_x};
    weight = Matrix{a->weight, a->out, a->in, a->ld_weight};
    if (!operand_ok(x) || !operand_ok(weight))
        return Z1_EINVAL;
    w = plan_product(z1::ops::kForward, a->dtype, weight, x);
    return w.fits ? Z1_OK : Z1_EINVAL;
}

struct GradPlan {
    Matrix dz, x, weight;
    Plan dx, dw;
    int64_t bytes;
};

// The two products run one after the other in the same workspace.
z1_status linear_grad_plan(const z1_linear_grad_args *a, GradPlan &w)
{
    if (!a || product_sizes(a->rows, a->in, a->out, a->dtype) != Z1_OK || (!a->dx && !a->dweight && a->rows > 0))
        return Z1_EINVAL;
    w.dz = Matrix{a->dz, a->rows, a->out, a->ld_dz};
    w.x = Matrix{a->x, a->rows, a->in, a->ld_x};
    w.weight = Matrix{a->weight, a->out, a->in, a->ld_weight};
    w.bytes = 0;
    if (!operand_ok(w.dz) || (a->dx && !operand_ok(w.weight)) || (a->dweight && !operand_ok(w.x)))
        return Z1_EINVAL;
    if (a->dx) {
        w.dx = plan_product(z1::ops::kInput, a->dtype, w.weight, w.dz);
        w.bytes = w.dx.bytes;
    }
    if (a->dweight) {
        w.dw = plan_product(z1::ops::kWeight, a->dtype, w.x, w.dz);
        w.bytes = std::max(w.bytes, w.dw.bytes);
    }
    return w.dx.fits && w.dw.fits ? Z1_OK : Z1_EINVAL;
}

z1_status workspace_ok(const void *workspace, int64_t have, int64_t need)
{
    if (have < need || (need > 0 && !workspace))
        return Z1_EINVAL;
    return need > 0 && !aligned(workspace, 16) ? Z1_EALIGN : Z1_OK;
}

bool act_ok(int32_t act) { return act >= Z1_ACT_NONE && act <= Z1_ACT_RELU2; }

bool heads_ok(const z1_heads &k, int64_t tokens, bool grad)
{
    if (k.heads < 0 || k.heads > (1 << 16))
        return false;
    if (k.heads == 0 || tokens == 0)
        return true;
    // out may be the input (or in the gradient dout) with the same strides
    const auto apart = [&](const void *p, int64_t token, int64_t head) {
        return p != k.out || ((tokens == 1 || token == k.out_token) && (k.heads == 1 || head == k.out_head));
    };
    return k.out && (!grad || k.dout) && (k.x || (grad && !k.weight)) && apart(k.x, k.x_token, k.x_head) &&
           (!grad || apart(k.dout, k.dout_token, k.dout_head));
}

// Whether an output of the call is another buffer of it that it may not be.  work: the
// workspace, where one is used.
bool qk_overlap(const z1_qk_args *a, bool grad, const void *work)
{
    const z1_heads &q = a->q, &k = a->k;
    const bool has_q = a->tokens > 0 && q.heads > 0, has_k = a->tokens > 0 && k.heads > 0;
    const auto of = [](bool there, const void *p) { return there ? p : nullptr; };
    const void *q_out = of(has_q, q.out), *k_out = of(has_k, k.out), *q_dw = of(grad, q.dweight), *k_dw = of(grad, k.dweight);
    const void *q_x = of(has_q, q.x), *k_x = of(has_k, k.x), *q_w = of(has_q, q.weight), *k_w = of(has_k, k.weight);
    const void *q_dout = of(has_q && grad, q.dout), *k_dout = of(has_k && grad, k.dout);
    const void *at = of(has_q || has_k, a->positions), *freq = of(has_q || has_k, a->inv_freq);
    return among(q_out, {k_out, k_x, k_dout, q_w, k_w, q_dw, k_dw, at, freq}) || among(k_out, {q_x, q_dout, q_w, k_w, q_dw, k_dw, at, freq}) ||
           among(q_dw, {k_dw, q_x, k_x, q_dout, k_dout, q_w, k_w, at, freq}) || among(k_dw, {q_x, k_x, q_dout, k_dout, q_w, k_w, at, freq}) ||
           among(work, {q_out, k_out, q_dw, k_dw, q_x, k_x, q_dout, k_dout, q_w, k_w, at, freq});
}

z1_status qk_check(const z1_qk_args *a, bool grad, const void *work = nullptr)
{
    if (!a || a->tokens < 0 || a->tokens > INT32_MAX || a->dim < 1 || a->dim > 512 || a->n_freq < 0 ||
        a->n_freq > a->dim / 2 || !dtype_ok(a->dtype) || !itype_ok(a->position_type) || !(a->eps >= 0.0) ||
        !is_finite(a->eps) || (a->interleaved != 0 && a->interleaved != 1) || (a->accumulate != 0 && a->accumulate != 1) ||
        !heads_ok(a->q, a->tokens, grad) || !heads_ok(a->k, a->tokens, grad))
        return Z1_EINVAL;
    if ((a->tokens > 0 && !a->positions) || (a->n_freq > 0 && !a->inv_freq))
        return Z1_EINVAL;
    if (grad && ((a->q.dweight && !a->q.weight) || (a->k.dweight && !a->k.weight)))
        return Z1_EINVAL;
    if (qk_overlap(a, grad, work))
        return Z1_EINVAL;
    const size_t size = type_size(a->dtype);
    for (const z1_heads *k : {&a->q, &a->k})
        if (!aligned(k->x, size) || !aligned(k->out, size) || !aligned(k->dout, size) || !aligned(k->weight, size) ||
            !aligned(k->dweight, 4))
            return Z1_EALIGN;
    return aligned(a->positions, itype_size(a->position_type)) && aligned(a->inv_freq, 8) ? Z1_OK : Z1_EALIGN;
}

}  // namespace

extern "C" {

int32_t z1_layers_abi_version(void) { return Z1_LAYERS_ABI_VERSION; }

z1_status z1_dropout(const z1_dropout_args *a, z1_stream stream)
{
    if (!a || a->rows < 0 || a->rows > INT32_MAX || a->cols < 1 || a->cols > (1 << 24) || !dtype_ok(a->dtype) ||
        a->reserved != 0 || !drop_ok(a->drop) || !rows_ok(a->x, a->rows, a->cols, a->ld_x, true) ||
        !rows_ok(a->y, a->rows, a->cols, a->ld_y, true) || !rows_ok(a->residual, a->rows, a->cols, a->ld_residual, false))
        return Z1_EINVAL;
    if (a->rows > 1 && ((a->y == a->x && a->ld_y != a->ld_x) || (a->y == a->residual && a->ld_y != a->ld_residual)))
        return Z1_EINVAL;
    if (a->rows > 0 && among(a->y, {read_rng(a->drop)}))
        return Z1_EINVAL;
    const size_t size = type_size(a->dtype);
    if (!aligned(a->x, size) || !aligned(a->y, size) || !aligned(a->residual, size) || !aligned(a->drop.rng, 8))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return status_of(z1::ops::launch_dropout(*a, drop_of(a->drop), hip(stream)));
}

z1_status z1_linear_workspace(const z1_linear_args *args, int64_t *bytes)
{
    Matrix x, weight;
    Plan w;
    if (!bytes || linear_plan(args, x, weight, w) != Z1_OK)
        return Z1_EINVAL;
    *bytes = w.bytes;
    return Z1_OK;
}

z1_status z1_linear(const z1_linear_args *a, void *workspace, int64_t workspace_bytes, z1_stream stream)
{
    Matrix x, weight;
    Plan w;
    if (linear_plan(a, x, weight, w) != Z1_OK || !act_ok(a->act) || !drop_ok(a->drop) ||
        !rows_ok(a->y, a->rows, a->out, a->ld_y, true) || !rows_ok(a->pre, a->rows, a->out, a->ld_pre, false) ||
        !rows_ok(a->mul, a->rows, a->out, a->ld_mul, false) || !rows_ok(a->residual, a->rows, a->out, a->ld_residual, false))
        return Z1_EINVAL;
    if (a->rows > 1 && ((a->y == a->residual && a->ld_y != a->ld_residual) || (a->y == a->mul && a->ld_y != a->ld_mul)))
        return Z1_EINVAL;
    const void *rng = read_rng(a->drop);
    if (a->rows > 0 &&
        (among(a->y, {a->x, a->weight, a->bias, a->pre, rng}) || among(a->pre, {a->x, a->weight, a->bias, a->mul, a->residual, rng}) ||
         among(used(workspace, w.bytes), {a->x, a->weight, a->bias, a->mul, a->residual, a->pre, a->y, rng})))
        return Z1_EINVAL;
    const z1_status ws = workspace_ok(workspace, workspace_bytes, w.bytes);
    if (ws == Z1_EINVAL)
        return ws;
    const size_t size = type_size(a->dtype);
    for (const void *p : {a->x, a->weight, a->bias, a->mul, a->residual, (const void *)a->pre, (const void *)a->y})
        if (!aligned(p, size))
            return Z1_EALIGN;
    if (ws != Z1_OK || !aligned(a->drop.rng, 8))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    if (a->rows == 0)
        return Z1_OK;
    w.g.e = Epilogue{a->y, a->pre, a->residual, a->mul, a->bias, a->ld_y, a->ld_pre, a->ld_residual, a->ld_mul,
                     drop_of(a->drop), a->act};
    return run_product(z1::ops::kForward, a->dtype, a->dtype, w, weight, x, workspace, hip(stream));
}

z1_status z1_linear_dz_workspace(int64_t rows, int64_t out, int64_t *bytes)
{
    if (!bytes || rows < 0 || rows > kMostRows || out < 1 || out > kMostSide)
        return Z1_EINVAL;
    const int64_t piece = z1::ops::dz_piece(rows, out);
    *bytes = (rows + piece - 1) / piece * out * 4;
    return Z1_OK;
}

z1_status z1_linear_dz(const z1_linear_dz_args *a, void *workspace, int64_t workspace_bytes, z1_stream stream)
{
    int64_t need = 0;
    if (!a || z1_linear_dz_workspace(a->rows, a->out, &need) != Z1_OK || !dtype_ok(a->dtype) || !act_ok(a->act) ||
        a->reserved != 0 || (a->accumulate != 0 && a->accumulate != 1) || !drop_ok(a->drop) ||
        (!a->dz && !a->dmul && !a->dbias))
        return Z1_EINVAL;
    if (!a->dbias)
        need = 0;
    if (!rows_ok(a->dy, a->rows, a->out, a->ld_dy, true) ||
        !rows_ok(a->pre, a->rows, a->out, a->ld_pre, a->act != Z1_ACT_NONE || a->dmul) ||
        !rows_ok(a->mul, a->rows, a->out, a->ld_mul, false) || !rows_ok(a->dz, a->rows, a->out, a->ld_dz, false) ||
        !rows_ok(a->dmul, a->rows, a->out, a->ld_dmul, false))
        return Z1_EINVAL;
    if (a->rows > 1 && a->dz &&
        ((a->dz == a->dy && a->ld_dz != a->ld_dy) || (a->dz == a->pre && a->ld_dz != a->ld_pre) ||
         (a->dz == a->mul && a->ld_dz != a->ld_mul)))
        return Z1_EINVAL;
    const void *rng = read_rng(a->drop);
    if (a->rows > 0 &&
        (among(a->dmul, {a->dz, a->dy, rng}) || among(a->dz, {rng}) || among(a->dbias, {a->dy, a->pre, a->mul, a->dz, a->dmul, rng}) ||
         among(used(workspace, need), {a->dy, a->pre, a->mul, a->dz, a->dmul, a->dbias, rng})))
        return Z1_EINVAL;
    if (a->rows > 1 && a->dmul &&
        ((a->dmul == a->pre && a->ld_dmul != a->ld_pre) || (a->dmul == a->mul && a->ld_dmul != a->ld_mul)))
        return Z1_EINVAL;
    const z1_status ws = workspace_ok(workspace, workspace_bytes, need);
    if (ws == Z1_EINVAL)
        return ws;
    const size_t size = type_size(a->dtype);
    for (const void *p : {a->dy, a->pre, a->mul, (const void *)a->dz, (const void *)a->dmul})
        if (!aligned(p, size))
            return Z1_EALIGN;
    if (ws != Z1_OK || !aligned(a->dbias, 4) || !aligned(a->drop.rng, 8))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return status_of(z1::ops::launch_linear_dz(*a, drop_of(a->drop), static_cast<float *>(workspace), hip(stream)));
}

z1_status z1_linear_grad_workspace(const z1_linear_grad_args *args, int64_t *bytes)
{
    GradPlan w;
    if (!bytes || linear_grad_plan(args, w) != Z1_OK)
        return Z1_EINVAL;
    *bytes = w.bytes;
    return Z1_OK;
}

z1_status z1_linear_grad(const z1_linear_grad_args *a, void *workspace, int64_t workspace_bytes, z1_stream stream)
{
    GradPlan w;
    if (linear_grad_plan(a, w) != Z1_OK || (a->dweight_dtype != Z1_F32 && a->dweight_dtype != a->dtype) ||
        a->reserved != 0 || (a->accumulate != 0 && a->accumulate != 1) || (a->accumulate && a->dweight_dtype != Z1_F32) ||
        !rows_ok(a->dx, a->rows, a->in, a->ld_dx, false) || !rows_ok(a->add, a->rows, a->in, a->ld_add, false) ||
        (a->dweight && a->ld_dweight < a->in))
        return Z1_EINVAL;
    if (a->rows > 1 && a->dx && a->dx == a->add && a->ld_dx != a->ld_add)
        return Z1_EINVAL;
    // dx is written before dweight is computed; without dweight x is not read
    if (a->rows > 0 && (among(a->dx, {a->dz, a->weight, a->dweight, a->dweight ? a->x : nullptr}) ||
                        among(a->dweight, {a->dz, a->x, a->dx ? a->weight : nullptr, a->dx ? a->add : nullptr}) ||
                        among(used(workspace, w.bytes), {a->dz, a->dweight ? a->x : nullptr, a->dx ? a->weight : nullptr,
                                                         a->dx ? a->add : nullptr, a->dx, a->dweight})))
        return Z1_EINVAL;
    const z1_status ws = workspace_ok(workspace, workspace_bytes, w.bytes);
    if (ws == Z1_EINVAL)
        return ws;
    const size_t size = type_size(a->dtype);
    for (const void *p : {a->dz, a->x, a->weight, a->add, (const void *)a->dx})
        if (!aligned(p, size))
            return Z1_EALIGN;
    if (ws != Z1_OK || !aligned(a->dweight, type_size(a->dweight_dtype)))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    const Drop none{nullptr, 0, 0, 1.f};
    if (a->dx && a->rows > 0) {
        w.dx.g.e = Epilogue{a->dx, nullptr, a->add, nullptr, nullptr, a->ld_dx, 0, a->ld_add, 0, none, Z1_ACT_NONE};
        const z1_status st = run_product(z1::ops::kInput, a->dtype, a->dtype, w.dx, w.weight, w.dz, workspace, hip(stream));
        if (st != Z1_OK)
            return st;
    }
    // of no rows, dweight is a sum of nothing
    if (a->dweight && (a->rows > 0 || !a->accumulate)) {
        w.dw.g.e = Epilogue{a->dweight, nullptr, a->accumulate ? a->dweight : nullptr, nullptr, nullptr,
                            a->ld_dweight, 0, a->ld_dweight, 0, none, Z1_ACT_NONE};
        return run_product(z1::ops::kWeight, a->dtype, a->dweight_dtype, w.dw, w.x, w.dz, workspace, hip(stream),
                           a->dx && a->rows > 0);
    }
    return Z1_OK;
}

z1_status z1_qk_norm_rope(const z1_qk_args *args, z1_stream stream)
{
    const z1_status st = qk_check(args, false);
    if (st != Z1_OK)
        return st;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return status_of(z1::ops::launch_qk(*args, hip(stream)));
}

z1_status z1_qk_norm_rope_grad_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads, int32_t dim, int64_t *bytes)
{
    if (!bytes || tokens < 0 || tokens > INT32_MAX || q_heads < 0 || q_heads > (1 << 16) || k_heads < 0 ||
        k_heads > (1 << 16) || dim < 1 || dim > 512)
        return Z1_EINVAL;
    *bytes = (z1::ops::qk_grad_groups(tokens, q_heads, k_heads, 0) + z1::ops::qk_grad_groups(tokens, q_heads, k_heads, 1)) * dim * 4;
    return Z1_OK;
}

z1_status z1_qk_norm_rope_grad(const z1_qk_args *a, void *workspace, int64_t workspace_bytes, z1_stream stream)
{
    int64_t need = 0;
    const bool sums = a && (a->q.dweight || a->k.dweight);
    if (sums && z1_qk_norm_rope_grad_workspace(a->tokens, a->q.heads, a->k.heads, a->dim, &need) != Z1_OK)
        return Z1_EINVAL;
    const z1_status st = qk_check(a, true, used(workspace, need));
    if (st == Z1_EINVAL)
        return st;
    const z1_status ws = workspace_ok(workspace, workspace_bytes, need);
    if (ws == Z1_EINVAL)
        return ws;
    if (st != Z1_OK || ws != Z1_OK)
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return status_of(z1::ops::launch_qk_grad(*a, sums ? static_cast<float *>(workspace) : nullptr, hip(stream)));
}

}  // extern "C"
