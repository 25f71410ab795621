// z1_ops_api.hip -- host side of the operators declared in include/z1_ops.h:
// argument validation, the Muon handle's tables and workspace, and the
// launches.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <vector>

#include "z1_host.h"
#include "z1_ops.h"
#include "z1_ops_internal.h"

using namespace z1::host;
using z1::ops::MuonChunk;
using z1::ops::MuonMat;
using z1::ops::MuonTables;
using z1::ops::MuonTile;
using z1::ops::MuonUpdate;
using z1::ops::pad_to;
using z1::ops::pick_tile;

struct z1_muon {
    int device = -1;
    bool can_step = false, can_ortho = false;
    int32_t ns_steps = 0;
    MuonTables t{};
    void *block = nullptr;   // one allocation: tables, partials, matrices
};

namespace {

// Host allocations are the only operations of a body that can throw; they
// become Z1_ENOMEM and never cross the C interface.
template <typename F>
z1_status no_throw(F &&body)
{
    try {
        return body();
    } catch (...) {
        return Z1_ENOMEM;
    }
}

// --------------------------------------------------------------------------
// Muon
// --------------------------------------------------------------------------

// Largest |p| on [0, top] for p(x) = a x + b x^3 + c x^5: the ends and the
// roots of p' = a + 3 b s + 5 c s^2, s = x^2.
double largest_p(double a, double b, double c, double top)
{
    const auto p = [&](double x) { return fabs(x * (a + x * x * (b + x * x * c))); };
    double best = p(top);
    const double qa = 5.0 * c, qb = 3.0 * b;
    double roots[2];
    int n = 0;
    if (qa == 0.0) {
        if (qb != 0.0)
            roots[n++] = -a / qb;
    } else {
        const double d = qb * qb - 4.0 * qa * a;
        if (d >= 0.0) {
            roots[n++] = (-qb + sqrt(d)) / (2.0 * qa);
            roots[n++] = (-qb - sqrt(d)) / (2.0 * qa);
        }
    }
    for (int i = 0; i < n; ++i)
        if (roots[i] > 0.0 && roots[i] < top * top)
            best = std::max(best, p(sqrt(roots[i])));
    return best;
}

// The fp16 operands hold |x| < 65504 / 2^14 = 3.998; rounding adds a little
// to the exact iteration's range.
constexpr double kRange = 3.9;

bool coefficients_ok(const z1_muon_bind *b)
{
    if (!is_finite(b->a) || !is_finite(b->b) || !is_finite(b->c))
        return false;
    double top = 1.0;   // |X| <= |X|_F = 1
    for (int k = 0; k < b->ns_steps; ++k) {
        const double s = top * top;
        if (top > kRange || s > kRange)
            return false;
        double q = fabs(s * (b->b + b->c * s));       // |b s + c s^2| on [0, top^2]
        const double v = b->c != 0.0 ? -b->b / (2.0 * b->c) : -1.0;
        if (v > 0.0 && v < s)
            q = std::max(q, fabs(v * (b->b + b->c * v)));
        if (!(q <= kRange))
            return false;
        top = largest_p(b->a, b->b, b->c, top);
        if (!is_finite(top))
            return false;
    }
    return true;
}

// Spreads a list of tiles over the 8 XCDs: workgroup p runs on XCD p mod 8,
// so entry p takes the next tile of XCD p mod 8's contiguous eighth, and
// tiles that share operand panels share an L2.
void spread(std::vector<MuonTile> &t)
{
    const size_t n = t.size(), per = n / 8, more = n % 8;
    std::vector<MuonTile> out(n);
    size_t at = 0;
    for (size_t x = 0; x < 8; ++x) {
        const size_t len = per + (x < more ? 1 : 0);
        for (size_t q = 0; q < len; ++q)
            out[q * 8 + x] = t[at++];
    }
    t.swap(out);
}

// The tiles of one matrix's product in blocks of kGroup tile rows, column by
// column inside a block: the tiles of a few dozen consecutive entries then
// share few panels.
void add_tiles(std::vector<MuonTile> &t, int32_t mat, int nt_i, int nt_j, bool lower)
{
    constexpr int kGroup = 8;
    for (int g = 0; g < nt_i; g += kGroup)
        for (int j = 0; j < nt_j; ++j)
            for (int i = g; i < std::min(nt_i, g + kGroup); ++i)
                if (!lower || i >= j)
                    t.push_back(MuonTile{mat, i, j, (int32_t)t.size()});
}

struct MuonDeleter {
    void operator()(z1_muon *m) const
    {
        if (m->block) {
            (void)hipDeviceSynchronize();   // an upload may still be in flight
            (void)hipFree(m->block);
        }
        delete m;
    }
};

template <typename T>
size_t reserve(size_t &at, size_t count)
{
    const size_t here = at;
    at = (at + count * sizeof(T) + 255) / 256 * 256;
    return here;
}

z1_status muon_create(z1_muon **out, const z1_muon_bind *b, bool wide, z1_stream stream)
{
    const int32_t n = b->n;
    const int dev = current_device();
    if (!runs_on(dev, stream))
        return Z1_EINVAL;
    std::unique_ptr<z1_muon, MuonDeleter> m(new z1_muon);
    m->device = dev;
    m->can_step = b->master != nullptr;
    m->can_ortho = b->ortho != nullptr;
    m->ns_steps = b->ns_steps;
    MuonTables &t = m->t;
    t.grad_bf16 = b->grad_dtype == Z1_BF16;
    t.wide = wide;
    t.a = (float)b->a;
    t.b = (float)b->b;
    t.c = (float)b->c;
    t.eps = b->eps;
    // the matrices of the tiled path first, then the small ones
    std::vector<int32_t> order, few;
    std::vector<int64_t> rows, cols;
    for (int32_t i = 0; i < n; ++i) {
        if (!wide && z1::ops::muon_small(pad_to(std::min(b->rows[i], b->cols[i]), 32),
                                pad_to(std::max(b->rows[i], b->cols[i]), 32))) {
            few.push_back(i);
        } else {
            order.push_back(i);
            rows.push_back(b->rows[i]);
            cols.push_back(b->cols[i]);
        }
    }
    t.n = (int32_t)order.size();
    t.n_small = (int32_t)few.size();
    order.insert(order.end(), few.begin(), few.end());
    int32_t whole = 64;   // sides are padded to whole tiles of every product
    for (int p = 0; p < 3; ++p) {
        t.tile[p] = pick_tile(p, t.n, rows.data(), cols.data(), wide ? 3 : 1);
        whole = std::max(whole, t.tile[p]);
    }

    // more workgroups than one launch takes: refused before the tables are built
    constexpr double kMostTiles = INT32_MAX / 512;
    double n_cast = 0.0, n_chunk = 0.0;
    for (int32_t i = 0; i < t.n; ++i) {
        const int64_t c = z1::ops::kCastTile;
        n_cast += (double)(pad_to(rows[i], whole) / c) * (double)(pad_to(cols[i], whole) / c);
        n_chunk += ceil((double)rows[i] * (double)cols[i] / z1::ops::kMuonChunk);
    }
    if (n_cast > kMostTiles || n_chunk > kMostTiles)
        return Z1_EINVAL;

    std::vector<MuonMat> mats((size_t)n);
    std::vector<MuonChunk> chunks;
    std::vector<MuonTile> cast, tiles[3];
    for (int32_t at = 0; at < n; ++at) {
        const int32_t i = order[(size_t)at];
        const int32_t side = at < t.n ? whole : 32;
        MuonMat &q = mats[(size_t)at];
        q = MuonMat{};
        q.grad = b->grad[i];
        q.rows = (int32_t)b->rows[i];
        q.cols = (int32_t)b->cols[i];
        q.flip = q.rows > q.cols;
        q.m = q.flip ? q.cols : q.rows;
        q.n = q.flip ? q.rows : q.cols;
        q.mp = (int32_t)pad_to(q.m, side);
        q.np = (int32_t)pad_to(q.n, side);
        q.vec = aligned(q.grad, 16);
        if (m->can_step) {
            q.mom = b->momentum[i];
            q.master = b->master[i];
            q.weight = static_cast<uint16_t *>(b->weights[i]);
            q.vec = q.vec && aligned(q.mom, 16);
        }
        if (m->can_ortho)
            q.ortho = static_cast<uint16_t *>(b->ortho[i]);
        q.vec4 = q.cols % 4 == 0 && aligned(q.master, 16) && aligned(q.weight, 8) && aligned(q.ortho, 8);
        q.lr_scale = b->lr_scale ? b->lr_scale[i] : 1.0;
        q.wd_scale = b->wd_scale ? b->wd_scale[i] : 1.0;
        if (at >= t.n)
            continue;
        const int64_t numel = (int64_t)q.rows * q.cols;
        q.part0 = (int64_t)chunks.size();
        for (int64_t s = 0; s < numel; s += z1::ops::kMuonChunk)
            chunks.push_back(MuonChunk{s, at, (int32_t)std::min<int64_t>(z1::ops::kMuonChunk, numel - s)});
        q.n_part = (int64_t)chunks.size() - q.part0;
        t.n_part_most = std::max(t.n_part_most, q.n_part);
        add_tiles(cast, at, q.mp / z1::ops::kCastTile, q.np / z1::ops::kCastTile, false);
        for (int p = 0; p < 3; ++p)
            add_tiles(tiles[p], at, q.mp / t.tile[p], (p == 2 ? q.np : q.mp) / t.tile[p], p < 2);
    }
    std::vector<MuonTile> pieces;
    int64_t panels = INT64_MAX;
    for (int32_t at = 0; at < t.n; ++at)
        panels = std::min<int64_t>(panels, mats[(size_t)at].np / 32);
    t.splits = z1::ops::gram_splits(t.tile[0], (int64_t)tiles[0].size(), panels);
    if (t.splits > 1)
        for (const MuonTile &q : tiles[0])
            for (int32_t s = 0; s < t.splits; ++s)
                pieces.push_back(MuonTile{q.mat, q.ti, q.tj, q.part * t.splits + s});
    for (auto &list : tiles)
        spread(list);
    spread(pieces);
    t.n_chunks = (int64_t)chunks.size();
    t.n_cast = (int64_t)cast.size();
    for (int p = 0; p < 3; ++p)
        t.n_tiles[p] = (int64_t)tiles[p].size();
    if (n == 0) {
        *out = m.release();
        return Z1_OK;
    }
    size_t bytes = 0;
    const size_t o_mats = reserve<MuonMat>(bytes, mats.size());
    const size_t o_chunks = reserve<MuonChunk>(bytes, chunks.size());
    const size_t o_cast = reserve<MuonTile>(bytes, cast.size());
    size_t o_tiles[3];
    for (int p = 0; p < 3; ++p)
        o_tiles[p] = reserve<MuonTile>(bytes, tiles[p].size());
    const size_t o_pieces = reserve<MuonTile>(bytes, pieces.size());
    const size_t tables = bytes;
    const size_t o_sums = reserve<float>(bytes, pieces.size() * 64 * 64);
    const size_t o_part = reserve<double>(bytes, chunks.size());
    const size_t o_inv = reserve<double>(bytes, mats.size());
    // each matrix's operands: X, Y, Y, A, B, then L, or the five's remainders
    // and F
    const size_t n_bufs = wide ? 11 : 6;
    std::vector<size_t> offs;
    for (int32_t at = 0; at < t.n; ++at) {
        const MuonMat &q = mats[(size_t)at];
        const size_t mn = (size_t)q.mp * (size_t)q.np, mm = (size_t)q.mp * (size_t)q.mp;
        for (size_t k = 0; k < n_bufs; ++k)
            offs.push_back(reserve<_Float16>(bytes, k == 10 ? 2 * mn : k % 5 < 3 ? mn : mm));
    }
    if (hipMalloc(&m->block, bytes) != hipSuccess) {
        (void)hipGetLastError();
        m->block = nullptr;
        return Z1_ENOMEM;
    }
    char *base = static_cast<char *>(m->block);
    for (size_t i = 0; i < (size_t)t.n; ++i) {
        MuonMat &q = mats[i];
        const auto buf = [&](size_t k) { return reinterpret_cast<_Float16 *>(base + offs[n_bufs * i + k]); };
        q.X = buf(0);
        q.Y[0] = buf(1);
        q.Y[1] = buf(2);
        q.A = buf(3);
        q.B = buf(4);
        if (wide) {
            q.Xl = buf(5);
            q.Yl[0] = buf(6);
            q.Yl[1] = buf(7);
            q.Al = buf(8);
            q.Bl = buf(9);
            q.F = reinterpret_cast<float *>(buf(10));
        } else {
            q.L = buf(5);
        }
    }
    t.mats = reinterpret_cast<MuonMat *>(base + o_mats);
    t.chunks = reinterpret_cast<MuonChunk *>(base + o_chunks);
    t.cast = reinterpret_cast<MuonTile *>(base + o_cast);
    for (int p = 0; p < 3; ++p)
        t.tiles[p] = reinterpret_cast<MuonTile *>(base + o_tiles[p]);
    t.pieces = reinterpret_cast<MuonTile *>(base + o_pieces);
    t.parts = reinterpret_cast<float *>(base + o_sums);
    t.partials = reinterpret_cast<double *>(base + o_part);
    t.inv = reinterpret_cast<double *>(base + o_inv);
    std::vector<char> host(tables);
    memcpy(&host[o_mats], mats.data(), mats.size() * sizeof(MuonMat));
    if (t.n > 0) {
        memcpy(&host[o_chunks], chunks.data(), chunks.size() * sizeof(MuonChunk));
        memcpy(&host[o_cast], cast.data(), cast.size() * sizeof(MuonTile));
        for (int p = 0; p < 3; ++p)
            memcpy(&host[o_tiles[p]], tiles[p].data(), tiles[p].size() * sizeof(MuonTile));
        if (!pieces.empty())
            memcpy(&host[o_pieces], pieces.data(), pieces.size() * sizeof(MuonTile));
    }
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    // a create call may wait: the staging buffer is this function's own
    if (hipMemcpyAsync(base, host.data(), tables, hipMemcpyHostToDevice, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess) {
        (void)hipGetLastError();
        return Z1_EHIP;
    }
    *out = m.release();
    return Z1_OK;
}

z1_status muon_checked(z1_muon **out, const z1_muon_bind *b, bool wide, z1_stream stream)
{
    if (out)
        *out = nullptr;
    if (!out || !b || b->n < 0 || b->reserved != 0)
        return Z1_EINVAL;
    if (b->grad_dtype != Z1_F32 && b->grad_dtype != Z1_BF16)
        return Z1_EINVAL;
    if (b->ns_steps < 1 || b->ns_steps > 32 || !(b->eps >= 0.0) || !is_finite(b->eps) || !coefficients_ok(b))
        return Z1_EINVAL;
    const bool step = b->momentum || b->master || b->weights;
    if (step && !(b->momentum && b->master && b->weights))
        return Z1_EINVAL;
    if (!step && !b->ortho)
        return Z1_EINVAL;
    if (b->n > 0 && (!b->rows || !b->cols || !b->grad))
        return Z1_EINVAL;
    for (int pass = 0; pass < 2; ++pass) {     // every null before any alignment
        for (int32_t i = 0; i < b->n; ++i) {
            if (b->rows[i] < 1 || b->rows[i] > (1 << 20) || b->cols[i] < 1 || b->cols[i] > (1 << 20))
                return Z1_EINVAL;
            if ((b->lr_scale && !is_finite(b->lr_scale[i])) || (b->wd_scale && !is_finite(b->wd_scale[i])))
                return Z1_EINVAL;
            const struct {
                const void *p;
                uintptr_t a;
                bool used;
            } all[5] = {{b->grad[i], (uintptr_t)type_size(b->grad_dtype), true},
                        {step ? b->momentum[i] : nullptr, 4, step},
                        {step ? b->master[i] : nullptr, 4, step},
                        {step ? b->weights[i] : nullptr, 2, step},
                        {b->ortho ? b->ortho[i] : nullptr, 2, b->ortho != nullptr}};
            for (const auto &q : all) {
                if (q.used && pass == 0 && !q.p)
                    return Z1_EINVAL;
                if (q.used && pass == 1 && !aligned(q.p, q.a))
                    return Z1_EALIGN;
            }
        }
    }
    return no_throw([&] { return muon_create(out, b, wide, stream); });
}

}  // namespace

extern "C" {

int32_t z1_ops_abi_version(void) { return Z1_OPS_ABI_VERSION; }

z1_status z1_muon_create(z1_muon **out, const z1_muon_bind *b, z1_stream stream)
{
    return muon_checked(out, b, false, stream);
}

z1_status z1_muon_create_wide(z1_muon **out, const z1_muon_bind *b, z1_stream stream)
{
    return muon_checked(out, b, true, stream);
}

z1_status z1_muon_destroy(z1_muon *m)
{
    if (!m)
        return Z1_OK;
    const int prev = current_device();
    const bool move = prev >= 0 && prev != m->device && hipSetDevice(m->device) == hipSuccess;
    hipError_t e = hipSuccess;
    if (m->block)
        e = hipFree(m->block);   // waits for work that uses it
    if (move)
        (void)hipSetDevice(prev);
    delete m;
    return e == hipSuccess ? Z1_OK : Z1_EHIP;
}

z1_status z1_muon_step(z1_muon *m, const z1_muon_hp *hp, const double *d_S, z1_stream stream)
{
    if (!m || !hp || hp->reserved != 0 || (hp->nesterov != 0 && hp->nesterov != 1))
        return Z1_EINVAL;
    if (!is_finite(hp->lr) || !(hp->momentum >= 0.0 && hp->momentum < 1.0) ||
        !(hp->weight_decay >= 0.0) || !is_finite(hp->weight_decay) || isnan(hp->clip))
        return Z1_EINVAL;
    if (hp->clip > 0.0 && !d_S)
        return Z1_EINVAL;
    if (!runs_on(m->device, stream))
        return Z1_EINVAL;
    if (d_S && !aligned(d_S, 8))
        return Z1_EALIGN;
    if (!m->can_step)
        return Z1_ESTATE;
    MuonUpdate u{};
    u.lr = hp->lr;
    u.wd = hp->weight_decay;
    u.mu = (float)hp->momentum;
    u.nesterov = hp->nesterov;
    u.clip = hp->clip;
    u.d_S = d_S;
    u.step = 1;
    return z1::ops::launch_muon(m->t, u, m->ns_steps, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

z1_status z1_muon_orthogonalize(z1_muon *m, z1_stream stream)
{
    if (!m)
        return Z1_EINVAL;
    if (!runs_on(m->device, stream))
        return Z1_EINVAL;
    if (!m->can_ortho)
        return Z1_ESTATE;
    MuonUpdate u{};
    return z1::ops::launch_muon(m->t, u, m->ns_steps, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

// --------------------------------------------------------------------------
// Embedding
// --------------------------------------------------------------------------

static bool embed_sizes_ok(int64_t n_ids, int64_t vocab, int64_t dim)
{
    return n_ids >= 0 && n_ids <= (INT64_C(1) << 30) && vocab >= 1 && vocab <= (1 << 24) &&
           dim >= 1 && dim <= (1 << 20);
}

static z1_status embed_shape(const z1_embed_args *a, z1::ops::EmbedShape *e)
{
    if (!a || !embed_sizes_ok(a->n_ids, a->vocab, a->dim) || !itype_ok(a->id_type) ||
        !dtype_ok(a->dtype) || !is_finite(a->scale) || (a->n_ids > 0 && !a->ids))
        return Z1_EINVAL;
    if (a->n_ids > 0 && !aligned(a->ids, itype_size(a->id_type)))
        return Z1_EALIGN;
    e->n = a->n_ids;
    e->vocab = a->vocab;
    e->dim = a->dim;
    e->ids = a->ids;
    e->id32 = a->id_type == Z1_I32;
    e->scale = (float)a->scale;
    return Z1_OK;
}

z1_status z1_embed_lookup(const z1_embed_args *args, const void *weight, int64_t ld_weight,
                          void *out, int64_t ld_out, z1_stream stream)
{
    z1::ops::EmbedShape e{};
    const z1_status st = embed_shape(args, &e);
    if (st == Z1_EINVAL)
        return st;
    if (!weight || (e.n > 0 && !out) || ld_weight < e.dim || ld_out < e.dim)
        return Z1_EINVAL;
    if (st != Z1_OK || !aligned(weight, type_size(args->dtype)) || !aligned(out, type_size(args->dtype)))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return z1::ops::launch_lookup(args->dtype, e, weight, ld_weight, out, ld_out,
                                  reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

z1_status z1_embed_grad_workspace(int64_t n_ids, int64_t vocab, int64_t dim, int64_t *bytes)
{
    if (!bytes || !embed_sizes_ok(n_ids, vocab, dim))
        return Z1_EINVAL;
    *bytes = z1::ops::embed_work(n_ids, vocab, dim).bytes;
    return Z1_OK;
}

z1_status z1_embed_grad(const z1_embed_args *args, const void *dout, int64_t ld_dout,
                        float *dweight, int32_t accumulate, void *workspace,
                        int64_t workspace_bytes, z1_stream stream)
{
    z1::ops::EmbedShape e{};
    const z1_status st = embed_shape(args, &e);
    if (st == Z1_EINVAL)
        return st;
    if (!dweight || (e.n > 0 && (!dout || !workspace)) || ld_dout < e.dim ||
        (accumulate != 0 && accumulate != 1) ||
        workspace_bytes < z1::ops::embed_work(e.n, e.vocab, e.dim).bytes)
        return Z1_EINVAL;
    if (st != Z1_OK || !aligned(dout, type_size(args->dtype)) || !aligned(dweight, 4) ||
        !aligned(workspace, 16))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return z1::ops::launch_embed_grad(args->dtype, e, dout, ld_dout, dweight, accumulate != 0,
                                      workspace, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

// --------------------------------------------------------------------------
// Losses
// --------------------------------------------------------------------------

static z1_status logits_rows(const z1_logits *x, void *d, int64_t ld_d, z1::ops::Rows *r)
{
    if (!x || x->n_rows < 0 || x->n_rows > INT32_MAX || x->vocab < 1 || x->vocab > (1 << 30) ||
        !dtype_ok(x->dtype) || !itype_ok(x->target_type) || x->ld < x->vocab ||
        (d && ld_d < x->vocab) || (x->n_rows > 0 && (!x->logits || !x->targets)))
        return Z1_EINVAL;
    const size_t es = type_size(x->dtype);
    if (!aligned(x->logits, es) || !aligned(d, es) || !aligned(x->targets, itype_size(x->target_type)))
        return Z1_EALIGN;
    r->n = x->n_rows;
    r->vocab = x->vocab;
    r->ld = x->ld;
    r->ld_d = ld_d;
    r->x = x->logits;
    r->y = x->targets;
    r->d = d;
    r->y32 = x->target_type == Z1_I32;
    const uintptr_t gap = reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(x->logits);
    r->d_vec = gap % 16 == 0 && (x->n_rows == 1 || ((x->ld - ld_d) * (int64_t)es) % 16 == 0);
    return Z1_OK;
}

z1_status z1_token_logprob(const z1_logits *x, float *logp, float *lse, z1_stream stream)
{
    z1::ops::Rows r{};
    const z1_status st = logits_rows(x, nullptr, 0, &r);
    if (st == Z1_EINVAL || (r.n > 0 && !logp))
        return Z1_EINVAL;
    if (st != Z1_OK || !aligned(logp, 4) || !aligned(lse, 4))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return z1::ops::launch_logprob(x->dtype, r, logp, lse, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

z1_status z1_logprob_grad(const z1_logits *x, const float *lse, const float *dlogp, void *dlogits,
                          int64_t ld_d, z1_stream stream)
{
    z1::ops::Rows r{};
    const z1_status st = logits_rows(x, dlogits, ld_d, &r);
    if (st == Z1_EINVAL || (r.n > 0 && (!lse || !dlogp || !dlogits)))
        return Z1_EINVAL;
    if (dlogits && dlogits == x->logits && ld_d != x->ld && x->n_rows > 1)
        return Z1_EINVAL;
    if (st != Z1_OK || !aligned(lse, 4) || !aligned(dlogp, 4))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return z1::ops::launch_logprob_grad(x->dtype, r, lse, dlogp, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

z1_status z1_policy_loss(const z1_logits *x, const z1_policy_args *a, z1_stream stream)
{
    if (!a || !a->loss)
        return Z1_EINVAL;
    z1::ops::Rows r{};
    const z1_status st = logits_rows(x, a->dlogits, a->ld_dlogits, &r);
    if (st == Z1_EINVAL || (r.n > 0 && (!a->old_logp || !a->advantages || !a->token_loss)))
        return Z1_EINVAL;
    if (a->dlogits && a->dlogits == x->logits && a->ld_dlogits != x->ld && x->n_rows > 1)
        return Z1_EINVAL;
    if (!(a->clip_low >= 0.0 && a->clip_low <= 1.0) || !(a->clip_high >= 0.0) || !is_finite(a->clip_high) ||
        !is_finite(a->kl_coef) || !is_finite(a->scale))
        return Z1_EINVAL;
    if (st != Z1_OK || !aligned(a->old_logp, 4) || !aligned(a->ref_logp, 4) ||
        !aligned(a->advantages, 4) || !aligned(a->weights, 4) || !aligned(a->loss, 4) ||
        !aligned(a->token_loss, 4) || !aligned(a->logp, 4))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    // without a coefficient there is no KL term: 0 times what overflows in it
    // would be NaN
    const float *ref = (float)a->kl_coef != 0.f ? a->ref_logp : nullptr;
    const z1::ops::PolicyPtrs p{a->old_logp, ref, a->advantages, a->weights, a->token_loss, a->logp};
    const z1::ops::PolicyScalars k{(float)(1.0 - a->clip_low), (float)(1.0 + a->clip_high),
                                   (float)a->kl_coef, (float)a->scale};
    return z1::ops::launch_policy(x->dtype, r, p, k, a->loss, a->scale,
                                  reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? Z1_OK
               : Z1_EHIP;
}

z1_status z1_preference_loss(const z1_preference_args *a, z1_stream stream)
{
    if (!a || a->n_rows < 0 || a->n_rows > INT32_MAX || a->n_pairs < 0 || a->n_pairs > (1 << 23) ||
        !itype_ok(a->target_type) || !itype_ok(a->cu_type) || !a->loss || !a->cu_seqlens)
        return Z1_EINVAL;
    if (!is_finite(a->beta) || !is_finite(a->scale) || !(a->label_smoothing >= 0.0 && a->label_smoothing <= 1.0))
        return Z1_EINVAL;
    if ((a->n_rows > 0 && (!a->logp || !a->ref_logp || !a->targets)) || (a->n_pairs > 0 && !a->pair_loss))
        return Z1_EINVAL;
    if (!aligned(a->logp, 4) || !aligned(a->ref_logp, 4) || !aligned(a->targets, itype_size(a->target_type)) ||
        !aligned(a->cu_seqlens, itype_size(a->cu_type)) || !aligned(a->loss, 4) ||
        !aligned(a->pair_loss, 4) || !aligned(a->margins, 4) || !aligned(a->dlogp, 4))
        return Z1_EALIGN;
    if (!runs_on(current_device(), stream))
        return Z1_EINVAL;
    return z1::ops::launch_preference(*a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? Z1_OK : Z1_EHIP;
}

}  // extern "C"
