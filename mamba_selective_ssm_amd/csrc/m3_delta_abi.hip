// C ABI of the gated delta rule and of the record pools: argument validation
// (complete before any HIP call), workspace sizes and launches.
#include "m3scan.h"

#include <math.h>
#include <string.h>

#include "m3_delta.hpp"
#include "m3_pool.hpp"

namespace {

struct Span {
    const char* p;
    int64_t bytes;
};

bool meet(const Span& a, const Span& b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
Span span(const void* p, int64_t bytes) { return Span{static_cast<const char*>(p), bytes}; }
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
m3_status status_of(hipError_t e) { return static_cast<m3_status>(m3::record_hip(e)); }

// HIP launches count a dimension's threads in 32 bits.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;
constexpr int64_t kMaxBlocks256 = kMaxThreads / 256;

// Sizes shared by the three calls.
m3_status check_sizes(int64_t batch, int64_t seqlen, int64_t H, int64_t G, int64_t P, int64_t N, int32_t io, int32_t l2norm,
                      float scale, float eps)
{
    if (batch < 0 || seqlen < 0 || H < 0 || P < 1 || N < 1) return M3_ERR_SHAPE;
    if (io != M3_F32 && io != M3_BF16) return M3_ERR_DTYPE;
    if (!m3::delta_supported(N, P, io)) return M3_ERR_UNSUPPORTED;
    if (G < 0 || (G > 0 && H % G != 0)) return M3_ERR_OPTION;
    if (l2norm != 0 && l2norm != 1) return M3_ERR_OPTION;
    if (l2norm && !(eps >= 0.f && eps < 3.0e38f)) return M3_ERR_OPTION;
    if (!(fabsf(scale) < 3.0e38f)) return M3_ERR_OPTION;
    // offsets inside one chunk are kept in 32 bits: 64 H 128 values
    if (H > ((int64_t)1 << 14) || G > ((int64_t)1 << 14) || batch > ((int64_t)1 << 24)) return M3_ERR_UNSUPPORTED;
    if (batch * H > ((int64_t)1 << 24)) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

struct DeltaPlan {
    int64_t G, nc, chunks;     // q/k groups; chunks of the longest row; (chunk slot, head) entries
    int64_t places;            // DeltaParams::places
    size_t tri_w, tri_o, sc;   // bytes of one array of each kind
    size_t st, rowsP, heads;   // gradient: states, [64][P] rows, per-head dq or dk
    size_t order;              // packed rows in the walks' order
    size_t carry;              // states between a long prefill's parts
    bool parts;                // whether it has them
    size_t fwd, bwd;           // whole workspaces
};

m3_status plan_delta(const m3_delta_args* a, bool train, DeltaPlan* out)
{
    if (a == nullptr) return M3_ERR_NULL;
    const m3_status s = check_sizes(a->batch, a->seqlen, a->nheads, a->ngroups, a->headdim, a->dstate, a->io_dtype,
                                    a->l2norm, a->scale, a->norm_eps);
    if (s != M3_OK) return s;
    const bool packed = a->cu_seqlens != nullptr;
    if (packed && (a->max_seqlen < 0 || a->max_seqlen > a->seqlen)) return M3_ERR_OPTION;
    const int64_t longest = packed ? a->max_seqlen : a->seqlen, H = a->nheads;
    if (longest > ((int64_t)1 << 30) || a->seqlen > ((int64_t)1 << 38)) return M3_ERR_UNSUPPORTED;
    out->G = a->ngroups > 0 ? a->ngroups : H;
    out->nc = (longest + m3::kDC - 1) / m3::kDC;
    const int64_t slots = packed ? a->seqlen / m3::kDC + a->batch + 1 : a->batch * out->nc;
    // long prefills of few rows in parts
    out->parts = m3::delta_in_parts(a->batch * H, out->nc, a->headdim, a->io_dtype);
    const int64_t direct = a->batch * out->nc, most = H > 0 ? kMaxBlocks256 / H : direct;
    out->places = packed && (direct > 2 * slots || direct > most) && (train || !out->parts) ? slots : 0;
    if ((out->places > 0 ? slots : direct) > most) return M3_ERR_UNSUPPORTED;
    // the walks: 16 columns of one row and head to a workgroup, 512 threads
    // (bf16: so few in one workgroup only where there are few, else 32 columns,
    // 448 threads), or twice 320; the other kernels that the gradient adds
    const int64_t slices = (a->batch * H + 7) / 8 * 8 * (a->headdim / 16);
    if (slices > kMaxThreads / (train ? 640 : a->io_dtype == M3_F32 ? 512 : 448)) return M3_ERR_UNSUPPORTED;
    if (train) {
        const int64_t tok = packed ? a->seqlen : a->batch * a->seqlen;   // dense: 64 chunks' worth at most
        if (a->batch >= kMaxBlocks256) return M3_ERR_UNSUPPORTED;
        if (out->G > 0 && tok > 4 * (kMaxThreads - 255) / (out->G * a->dstate)) return M3_ERR_UNSUPPORTED;
    }
    out->chunks = slots * H;
    const size_t n = (size_t)out->chunks;
    out->tri_w = up256(n * m3::kTriValues * 3 * 2);   // three bf16 planes
    out->tri_o = up256(n * m3::kTriValues * 4);       // float32
    out->sc = up256(n * m3::kDScal * 64 * 4);
    out->st = up256(n * (size_t)(a->dstate * a->headdim) * 4);
    out->rowsP = up256(n * (size_t)(64 * a->headdim) * 4);
    const size_t tokens = (size_t)(packed ? 1 : a->batch) * (size_t)a->seqlen;
    out->heads = out->G == H ? 0 : up256(tokens * (size_t)(H * a->dstate) * 4);
    // (places are counted row against row: left out where that would show, and
    // so many rows leave no CU idle for long)
    out->order = packed && a->batch <= 16384 ? up256((size_t)a->batch * 4) : 0;
    // (sized for any max_seqlen)
    out->carry = m3::delta_in_parts(a->batch * H, (a->seqlen + m3::kDC - 1) / m3::kDC, a->headdim, a->io_dtype)
                     ? up256((size_t)(a->batch * H * a->dstate * a->headdim) * 4)
                     : 0;
    out->fwd = n == 0 ? 0 : out->tri_w + out->tri_o + out->sc + out->order + out->carry;
    out->bwd = n == 0 ? 0 : out->tri_w + out->sc + out->order + 2 * out->st + 2 * out->rowsP + 2 * out->heads;
    return M3_OK;
}

// Bytes of the caller's arrays.
struct DeltaBytes {
    int64_t qk, vo, gb, rec, idx;
};
DeltaBytes bytes_of(const m3_delta_args* a, const DeltaPlan& pl)
{
    const int64_t e = a->io_dtype == M3_F32 ? 4 : 2;
    const int64_t tok = (a->cu_seqlens != nullptr ? 1 : a->batch) * a->seqlen;
    DeltaBytes r;
    r.qk = tok * pl.G * a->dstate * e;
    r.vo = tok * a->nheads * a->headdim * e;
    r.gb = tok * a->nheads * 4;
    r.rec = (a->slots != nullptr ? a->nslots : a->batch) * a->nheads * a->dstate * a->headdim * 4;
    r.idx = a->batch * 4;
    return r;
}

m3::DeltaParams params_of(const m3_delta_args* a, const DeltaPlan& pl)
{
    m3::DeltaParams p;
    memset(&p, 0, sizeof(p));
    p.q = a->q; p.k = a->k; p.v = a->v; p.g = a->g; p.beta = a->beta;
    p.h_in = a->h_in; p.o = a->o; p.h_out = a->h_out;
    p.cu = a->cu_seqlens; p.slots = a->slots; p.nslots = a->nslots;
    p.L = a->seqlen;
    p.max_len = a->cu_seqlens != nullptr ? a->max_seqlen : a->seqlen;
    p.rows = (int)a->batch; p.H = (int)a->nheads; p.G = (int)pl.G;
    p.N = (int)a->dstate; p.P = (int)a->headdim;
    p.scale = a->scale; p.eps = a->norm_eps; p.l2norm = a->l2norm;
    p.nc = (int)pl.nc;
    p.places = pl.places;
    return p;
}

int64_t pool_pieces(const m3_pool& p)
{
    int64_t n = 0;
    for (int i = 0; i < p.narrays; ++i) n += (p.row_bytes[i] + m3::kPoolPiece - 1) / m3::kPoolPiece;
    return n;
}

m3_status check_pool(const m3_pool& p)
{
    if (p.narrays < 1 || p.narrays > M3_POOL_MAX_ARRAYS || p.slots < 0) return M3_ERR_SHAPE;
    if (p.slots > ((int64_t)1 << 30)) return M3_ERR_UNSUPPORTED;
    for (int i = 0; i < p.narrays; ++i) {
        if (p.row_bytes[i] < 1) return M3_ERR_SHAPE;
        if (p.row_bytes[i] > ((int64_t)1 << 33) || p.slots * (p.row_bytes[i] >> 16) > ((int64_t)1 << 30)) return M3_ERR_UNSUPPORTED;
        if (p.slots > 0 && p.data[i] == nullptr) return M3_ERR_NULL;
        if (!on16(p.data[i])) return M3_ERR_ALIGN;
    }
    for (int i = 0; i < p.narrays; ++i)
        for (int j = i + 1; j < p.narrays; ++j)
            if (meet(span(p.data[i], p.slots * p.row_bytes[i]), span(p.data[j], p.slots * p.row_bytes[j])))
                return M3_ERR_ALIAS;
    return M3_OK;
}

bool meets_pool(const m3_pool& p, const Span& s)
{
    for (int i = 0; i < p.narrays; ++i)
        if (meet(span(p.data[i], p.slots * p.row_bytes[i]), s)) return true;
    return false;
}

m3::PoolParams pool_params(const m3_pool& src, const m3_pool& dst)
{
    m3::PoolParams q;
    memset(&q, 0, sizeof(q));
    q.n = dst.narrays;
    int pieces = 0;
    for (int i = 0; i < q.n; ++i) {
        const int64_t r = dst.row_bytes[i];
        q.src[i] = static_cast<const char*>(src.data[i]);
        q.dst[i] = static_cast<char*>(dst.data[i]);
        q.row[i] = r;
        q.unit[i] = r % 16 == 0 ? 16 : r % 4 == 0 ? 4 : r % 2 == 0 ? 2 : 1;
        q.piece0[i] = pieces;
        pieces += (int)((r + m3::kPoolPiece - 1) / m3::kPoolPiece);
        q.ws_off[i] = q.ws_row;
        q.ws_row += (r + 15) / 16 * 16;
    }
    q.piece0[q.n] = pieces;
    q.src_slots = src.slots;
    q.dst_slots = dst.slots;
    return q;
}

// *in_place: dst is src.
m3_status check_copy(const m3_pool_copy_args* a, bool* in_place)
{
    if (a == nullptr) return M3_ERR_NULL;
    m3_status s = check_pool(a->src);
    if (s == M3_OK) s = check_pool(a->dst);
    if (s != M3_OK) return s;
    if (a->src.narrays != a->dst.narrays || a->count < 0) return M3_ERR_SHAPE;
    bool same = a->src.slots == a->dst.slots;
    for (int i = 0; i < a->src.narrays; ++i) {
        if (a->src.row_bytes[i] != a->dst.row_bytes[i]) return M3_ERR_SHAPE;
        same = same && a->src.data[i] == a->dst.data[i];
    }
    if (!same)
        for (int i = 0; i < a->src.narrays; ++i)
            if (meets_pool(a->dst, span(a->src.data[i], a->src.slots * a->src.row_bytes[i]))) return M3_ERR_ALIAS;
    if (a->count > 0 && a->count > kMaxBlocks256 / pool_pieces(a->dst)) return M3_ERR_UNSUPPORTED;
    *in_place = same;
    return M3_OK;
}

size_t copy_workspace(const m3_pool_copy_args* a, bool in_place)
{
    if (!in_place) return 0;
    return (size_t)a->count * (size_t)pool_params(a->src, a->dst).ws_row;
}

}  // namespace

extern "C" {

int m3_delta_supported(int64_t dstate, int64_t headdim, int32_t io_dtype)
{
    return m3::delta_supported(dstate, headdim, io_dtype) ? 1 : 0;
}

size_t m3_delta_workspace_bytes(const m3_delta_args* a)
{
    DeltaPlan pl;
    return plan_delta(a, false, &pl) == M3_OK ? pl.fwd : 0;
}

size_t m3_delta_bwd_workspace_bytes(const m3_delta_bwd_args* a)
{
    DeltaPlan pl;
    return a != nullptr && plan_delta(&a->in, true, &pl) == M3_OK ? pl.bwd : 0;
}

m3_status m3_delta_fwd(const m3_delta_args* a, void* stream)
{
    DeltaPlan pl;
    const m3_status s = plan_delta(a, false, &pl);
    if (s != M3_OK) return s;
    if (a->slots != nullptr && (a->nslots < 0 || a->nslots > ((int64_t)1 << 30))) return M3_ERR_OPTION;
    if (a->batch * a->nheads == 0) return M3_OK;
    const DeltaBytes n = bytes_of(a, pl);
    if (n.vo > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o)) return M3_ERR_NULL;
    const void* al[] = {a->q, a->k, a->v, a->g, a->beta, a->h_in, a->o, a->h_out};
    for (const void* x : al)
        if (!on16(x)) return M3_ERR_ALIGN;
    if (!on4(a->cu_seqlens) || !on4(a->slots)) return M3_ERR_ALIGN;
    if (pl.fwd > 0) {
        if (a->workspace == nullptr || a->workspace_bytes < pl.fwd) return M3_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0) return M3_ERR_ALIGN;
    }
    const Span in[] = {span(a->q, n.qk), span(a->k, n.qk), span(a->v, n.vo), span(a->g, n.gb), span(a->beta, n.gb),
                       span(a->cu_seqlens, n.idx + 4), span(a->slots, n.idx), span(a->h_in, n.rec)};
    const Span out[] = {span(a->o, n.vo), span(a->h_out, n.rec), span(a->workspace, (int64_t)pl.fwd)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 8; ++j)
            if (!(i == 1 && j == 7 && a->h_in == a->h_out) && meet(out[i], in[j])) return M3_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (meet(out[i], out[j])) return M3_ERR_ALIAS;
    }
    m3::DeltaParams p = params_of(a, pl);
    char* w = static_cast<char*>(a->workspace);
    p.tf = reinterpret_cast<m3::bf16*>(w);
    p.af = reinterpret_cast<float*>(w + pl.tri_w);
    p.sc = reinterpret_cast<float*>(w + pl.tri_w + pl.tri_o);
    if (pl.order > 0 && pl.nc > 0) p.order = reinterpret_cast<int*>(w + pl.tri_w + pl.tri_o + pl.sc);
    if (pl.parts) p.carry_in = p.carry_out = reinterpret_cast<float*>(w + pl.tri_w + pl.tri_o + pl.sc + pl.order);
    return status_of(m3::launch_delta_fwd(p, a->io_dtype, static_cast<hipStream_t>(stream)));
}

m3_status m3_delta_step(const m3_delta_step_args* a, void* stream)
{
    if (a == nullptr) return M3_ERR_NULL;
    const m3_status s = check_sizes(a->batch, 1, a->nheads, a->ngroups, a->headdim, a->dstate, a->io_dtype, a->l2norm,
                                    a->scale, a->norm_eps);
    if (s != M3_OK) return s;
    // a wavefront to 32 columns of one row and head, four to a workgroup
    if (a->batch * a->nheads * (a->headdim / 32) > (kMaxThreads - 255) / 64) return M3_ERR_UNSUPPORTED;
    if (a->slots != nullptr && (a->nslots < 0 || a->nslots > ((int64_t)1 << 30))) return M3_ERR_OPTION;
    if (a->batch * a->nheads == 0) return M3_OK;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->h || !a->o) return M3_ERR_NULL;
    const void* al[] = {a->q, a->k, a->v, a->g, a->beta, a->h, a->o};
    for (const void* x : al)
        if (!on16(x)) return M3_ERR_ALIGN;
    if (!on4(a->slots)) return M3_ERR_ALIGN;
    m3_delta_args f;
    memset(&f, 0, sizeof(f));
    f.batch = a->batch; f.seqlen = 1; f.nheads = a->nheads; f.ngroups = a->ngroups;
    f.headdim = a->headdim; f.dstate = a->dstate;
    f.io_dtype = a->io_dtype; f.l2norm = a->l2norm; f.scale = a->scale; f.norm_eps = a->norm_eps;
    f.q = a->q; f.k = a->k; f.v = a->v; f.g = a->g; f.beta = a->beta;
    f.h_in = a->h; f.h_out = a->h; f.o = a->o; f.slots = a->slots; f.nslots = a->nslots;
    DeltaPlan pl;
    memset(&pl, 0, sizeof(pl));
    pl.G = a->ngroups > 0 ? a->ngroups : a->nheads;
    const DeltaBytes n = bytes_of(&f, pl);
    const Span in[] = {span(a->q, n.qk), span(a->k, n.qk), span(a->v, n.vo), span(a->g, n.gb), span(a->beta, n.gb),
                       span(a->slots, n.idx)};
    const Span out[] = {span(a->o, n.vo), span(a->h, n.rec)};
    for (const Span& x : out)
        for (const Span& y : in)
            if (meet(x, y)) return M3_ERR_ALIAS;
    if (meet(out[0], out[1])) return M3_ERR_ALIAS;
    return status_of(m3::launch_delta_step(params_of(&f, pl), a->io_dtype, static_cast<hipStream_t>(stream)));
}

m3_status m3_delta_bwd(const m3_delta_bwd_args* b, void* stream)
{
    if (b == nullptr) return M3_ERR_NULL;
    const m3_delta_args* a = &b->in;
    DeltaPlan pl;
    const m3_status s = plan_delta(a, true, &pl);
    if (s != M3_OK) return s;
    if (a->slots != nullptr || a->h_out != nullptr || a->o != nullptr) return M3_ERR_UNSUPPORTED;
    const DeltaBytes n = bytes_of(a, pl);
    if (a->batch * a->nheads == 0 && n.vo == 0 && n.qk == 0) return M3_OK;
    if (n.vo > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !b->dout || !b->dv || !b->dg || !b->dbeta)) return M3_ERR_NULL;
    if (n.qk > 0 && (!b->dq || !b->dk)) return M3_ERR_NULL;   // (groups without heads: zeros)
    const void* al[] = {a->q, a->k, a->v, a->g, a->beta, a->h_in, b->dout, b->dh_out, b->dq, b->dk, b->dv, b->dg, b->dbeta,
                        b->dh_in};
    for (const void* x : al)
        if (!on16(x)) return M3_ERR_ALIGN;
    if (!on4(a->cu_seqlens)) return M3_ERR_ALIGN;
    if (pl.bwd > 0) {
        if (a->workspace == nullptr || a->workspace_bytes < pl.bwd) return M3_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(a->workspace) & 255u) != 0) return M3_ERR_ALIGN;
    }
    const int64_t e = a->io_dtype == M3_F32 ? 1 : 2;   // float32 values per io value's bytes
    const Span in[] = {span(a->q, n.qk), span(a->k, n.qk), span(a->v, n.vo), span(a->g, n.gb), span(a->beta, n.gb),
                       span(a->cu_seqlens, n.idx + 4), span(a->h_in, n.rec), span(b->dout, n.vo), span(b->dh_out, n.rec)};
    const Span out[] = {span(b->dq, n.qk * e), span(b->dk, n.qk * e), span(b->dv, n.vo * e), span(b->dg, n.gb),
                        span(b->dbeta, n.gb), span(b->dh_in, n.rec), span(a->workspace, (int64_t)pl.bwd)};
    for (int i = 0; i < 7; ++i) {
        for (const Span& y : in)
            if (meet(out[i], y)) return M3_ERR_ALIAS;
        for (int j = i + 1; j < 7; ++j)
            if (meet(out[i], out[j])) return M3_ERR_ALIAS;
    }
    m3::DeltaBwdParams p;
    memset(&p, 0, sizeof(p));
    p.f = params_of(a, pl);
    p.dout = b->dout; p.dh_out = b->dh_out;
    p.dq = b->dq; p.dk = b->dk; p.dv = b->dv; p.dg = b->dg; p.dbeta = b->dbeta; p.dh_in = b->dh_in;
    char* w = static_cast<char*>(a->workspace);
    auto take = [&w](size_t bytes) { char* x = w; w += bytes; return x; };
    p.f.tf = reinterpret_cast<m3::bf16*>(take(pl.tri_w));
    p.f.sc = reinterpret_cast<float*>(take(pl.sc));
    int* const order = reinterpret_cast<int*>(take(pl.order));
    p.f.order = pl.order > 0 && pl.nc > 0 ? order : nullptr;
    p.S = reinterpret_cast<float*>(take(pl.st));
    p.dS = reinterpret_cast<float*>(take(pl.st));
    p.U = reinterpret_cast<float*>(take(pl.rowsP));
    p.dR = reinterpret_cast<float*>(take(pl.rowsP));
    const bool shared = pl.G != a->nheads;
    p.dqe = shared ? reinterpret_cast<float*>(take(pl.heads)) : b->dq;
    p.dke = shared ? reinterpret_cast<float*>(take(pl.heads)) : b->dk;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return status_of(a->io_dtype == M3_F32 ? m3::launch_delta_bwd_f32(p, st) : m3::launch_delta_bwd_bf16(p, st));
}

size_t m3_pool_copy_workspace_bytes(const m3_pool_copy_args* a)
{
    bool in_place = false;
    return check_copy(a, &in_place) == M3_OK ? copy_workspace(a, in_place) : 0;
}

m3_status m3_pool_copy(const m3_pool_copy_args* a, void* stream)
{
    bool in_place = false;
    const m3_status s = check_copy(a, &in_place);
    if (s != M3_OK) return s;
    if (a->count == 0 || a->dst.slots == 0) return M3_OK;
    if (a->src_slot == nullptr || a->dst_slot == nullptr) return M3_ERR_NULL;
    if (!on4(a->src_slot) || !on4(a->dst_slot)) return M3_ERR_ALIGN;
    const size_t need = copy_workspace(a, in_place);
    if (need > 0) {
        if (a->workspace == nullptr || a->workspace_bytes < need) return M3_ERR_WORKSPACE;
        if (!on16(a->workspace)) return M3_ERR_ALIGN;
    }
    const Span ix[] = {span(a->src_slot, a->count * 4), span(a->dst_slot, a->count * 4)}, ws = span(a->workspace, (int64_t)need);
    for (const Span& x : ix)
        if (meets_pool(a->dst, x) || meet(x, ws)) return M3_ERR_ALIAS;
    if (meets_pool(a->dst, ws)) return M3_ERR_ALIAS;
    m3::PoolParams p = pool_params(a->src, a->dst);
    p.ws = static_cast<char*>(a->workspace);
    return status_of(m3::launch_pool_copy(p, a->src_slot, a->dst_slot, a->count, in_place, static_cast<hipStream_t>(stream)));
}

m3_status m3_pool_fork(const m3_pool_fork_args* a, void* stream)
{
    if (a == nullptr) return M3_ERR_NULL;
    const m3_status s = check_pool(a->pool);
    if (s != M3_OK) return s;
    if (a->count < 0) return M3_ERR_SHAPE;
    const int64_t S = a->pool.slots;
    if (a->count > 0 && a->count > kMaxBlocks256 / pool_pieces(a->pool)) return M3_ERR_UNSUPPORTED;
    if (S == 0 && a->count == 0) return M3_OK;
    if ((S > 0 && (!a->live || !a->live_out)) || (a->count > 0 && (!a->parents || !a->children))) return M3_ERR_NULL;
    if (!on4(a->live) || !on4(a->live_out) || !on4(a->parents) || !on4(a->children) || !on4(a->workspace)) return M3_ERR_ALIGN;
    if (a->count > 0 && (a->workspace == nullptr || a->workspace_bytes < (size_t)a->count * 4)) return M3_ERR_WORKSPACE;
    const Span live = span(a->live, S * 4), par = span(a->parents, a->count * 4), out = span(a->live_out, S * 4),
               ch = span(a->children, a->count * 4), ws = span(a->workspace, a->count * 4);
    const Span all[] = {live, par, out, ch, ws};
    for (const Span& x : all)
        if (meets_pool(a->pool, x)) return M3_ERR_ALIAS;
    if ((a->live != a->live_out && meet(live, out)) || meet(par, out) || meet(par, ch) || meet(live, ch) || meet(out, ch) ||
        meet(ws, live) || meet(ws, par) || meet(ws, out) || meet(ws, ch))
        return M3_ERR_ALIAS;
    return status_of(m3::launch_pool_fork(pool_params(a->pool, a->pool), a->live, a->live_out, a->parents, a->children,
                                          static_cast<int*>(a->workspace), a->count, static_cast<hipStream_t>(stream)));
}

m3_status m3_pool_compact(const m3_pool_compact_args* a, void* stream)
{
    if (a == nullptr) return M3_ERR_NULL;
    const m3_status s = check_pool(a->pool);
    if (s != M3_OK) return s;
    const int64_t S = a->pool.slots;
    if (S / 2 > kMaxBlocks256 / pool_pieces(a->pool)) return M3_ERR_UNSUPPORTED;
    if (S > 0 && (!a->live || !a->new_slot)) return M3_ERR_NULL;
    if (!on4(a->live) || !on4(a->live_out) || !on4(a->new_slot) || !on4(a->count) || !on4(a->workspace)) return M3_ERR_ALIGN;
    if (a->workspace == nullptr || a->workspace_bytes < (size_t)(S + 1) * 4) return M3_ERR_WORKSPACE;
    const Span live = span(a->live, S * 4), out = span(a->live_out, S * 4), nw = span(a->new_slot, S * 4),
               ct = span(a->count, 4), ws = span(a->workspace, (S + 1) * 4);
    const Span all[] = {live, out, nw, ct, ws};
    for (const Span& x : all)
        if (meets_pool(a->pool, x)) return M3_ERR_ALIAS;
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (!(i == 0 && j == 1 && a->live == a->live_out) && meet(all[i], all[j])) return M3_ERR_ALIAS;
    return status_of(m3::launch_pool_compact(pool_params(a->pool, a->pool), a->live, a->live_out, a->new_slot, a->count,
                                             static_cast<int*>(a->workspace), static_cast<hipStream_t>(stream)));
}

m3_status m3_pool_free(int32_t* live, int64_t slots, const int32_t* list, int64_t count, void* stream)
{
    if (slots < 0 || count < 0) return M3_ERR_SHAPE;
    if (count > kMaxThreads - 255 || slots > ((int64_t)1 << 30)) return M3_ERR_UNSUPPORTED;
    if (slots == 0 || count == 0) return M3_OK;
    if (live == nullptr || list == nullptr) return M3_ERR_NULL;
    if (!on4(live) || !on4(list)) return M3_ERR_ALIGN;
    if (meet(span(live, slots * 4), span(list, count * 4))) return M3_ERR_ALIAS;
    return status_of(m3::launch_pool_free(live, slots, list, count, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
