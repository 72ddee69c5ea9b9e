// local_api.cu -- entry points of the local attention: host-side validation,
// the choice of kernel path and key-axis splits, workspace layout.
#include <limits.h>

#include "api_util.cuh"
#include "local.cuh"

namespace hsa {
namespace local {

namespace {

constexpr int SMS = 148;                 // B200
constexpr int MAX_POS = 1 << 30;
constexpr size_t HDR = 256;              // status word + padding

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

hsa_status_t check_heads(int H, int Hkv, int d, int dtype, unsigned flags, float scale, int window, int sinks) {
    if (H < 1 || Hkv < 1) return fail(HSA_ERR_INVALID_ARG, "H, Hkv must be >= 1 (H=%d Hkv=%d)", H, Hkv);
    if (H % Hkv != 0) return fail(HSA_ERR_INVALID_ARG, "H=%d is not a multiple of Hkv=%d", H, Hkv);
    if (dtype != HSA_F32 && dtype != HSA_BF16) return fail(HSA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (flags & ~HSA_FLAG_SIMT) return fail(HSA_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (!(scale >= 0.f) || isinf(scale)) return fail(HSA_ERR_INVALID_ARG, "scale must be finite and >= 0");
    if (window < 0 || sinks < 0) return fail(HSA_ERR_INVALID_ARG, "window=%d and sinks=%d must be >= 0", window, sinks);
    if (d != 64 && d != 128) return fail(HSA_ERR_UNSUPPORTED, "d=%d (supported: 64, 128)", d);
    if (H / Hkv > MAX_G) return fail(HSA_ERR_UNSUPPORTED, "G=%d (max %d)", H / Hkv, MAX_G);
    if (Hkv > 65535) return fail(HSA_ERR_UNSUPPORTED, "Hkv=%d (max 65535)", Hkv);
    return HSA_OK;
}

void fill_mask(LocArgs *a, float scale, int window, int sinks) {
    a->scale = scale > 0.f ? scale : 1.f / sqrtf((float)a->d);
    a->scale_log2 = a->scale * 1.4426950408889634f;
    a->window = window > 0 ? window : INT32_MAX;
    a->sinks = window > 0 ? sinks : 0;   // without a window every past key is visible anyway
}

hsa_status_t shape_of(const hsa_window_t *in, LocArgs *a) {
    if (!in) return fail(HSA_ERR_INVALID_ARG, "problem pointer is NULL");
    if (in->B < 0 || in->Tq < 0 || in->Tkv < 0)
        return fail(HSA_ERR_INVALID_ARG, "negative size (B=%d Tq=%d Tkv=%d)", in->B, in->Tq, in->Tkv);
    HSA_TRY(check_heads(in->H, in->Hkv, in->d, in->dtype, in->flags, in->scale, in->window, in->sinks));
    if (in->q_pos0 < 0) return fail(HSA_ERR_INVALID_ARG, "q_pos0 must be >= 0");
    if (in->kv_cap != 0 && in->kv_cap < in->Tkv)
        return fail(HSA_ERR_INVALID_ARG, "kv_cap=%d is below Tkv=%d", in->kv_cap, in->Tkv);
    if (in->B > 65535) return fail(HSA_ERR_UNSUPPORTED, "B=%d (max 65535)", in->B);
    const int cap = in->kv_cap != 0 ? in->kv_cap : in->Tkv;
    if (in->q_pos0 > MAX_POS - (int64_t)in->Tq || cap > MAX_POS)   // the sum itself may not fit 64 bits
        return fail(HSA_ERR_UNSUPPORTED, "positions must stay below 2^30");
    if ((long long)in->B * in->Tq > INT_MAX || (long long)in->B * cap > INT_MAX ||
        (long long)in->B * in->Tq * in->H > (1ll << 33))
        return fail(HSA_ERR_UNSUPPORTED, "too many tokens for 32-bit rows");
    *a = LocArgs{};
    a->B = in->B;
    a->H = in->H;
    a->Hkv = in->Hkv;
    a->G = in->H / in->Hkv;
    a->d = in->d;
    a->max_q = in->Tq;
    a->max_kv = in->Tkv;
    a->rows = in->B * in->Tq;
    a->Tcap = cap;
    a->q_pos0 = (int)in->q_pos0;
    fill_mask(a, in->scale, in->window, in->sinks);
    return HSA_OK;
}

hsa_status_t shape_of(const hsa_paged_t *in, LocArgs *a) {
    if (!in) return fail(HSA_ERR_INVALID_ARG, "problem pointer is NULL");
    if (in->B < 0 || in->rows < 0 || in->max_q < 0 || in->max_kv < 0)
        return fail(HSA_ERR_INVALID_ARG, "negative size (B=%d rows=%d max_q=%d max_kv=%d)", in->B, in->rows, in->max_q,
                    in->max_kv);
    HSA_TRY(check_heads(in->H, in->Hkv, in->d, in->dtype, in->flags, in->scale, in->window, in->sinks));
    if (in->page != 16 && in->page != 32 && in->page != 64 && in->page != 128)
        return fail(HSA_ERR_UNSUPPORTED, "page=%d (supported: 16, 32, 64, 128)", in->page);
    if (in->npages < 1 || in->max_pages < 1)
        return fail(HSA_ERR_INVALID_ARG, "npages=%d and max_pages=%d must be >= 1", in->npages, in->max_pages);
    if (in->B > 65535) return fail(HSA_ERR_UNSUPPORTED, "B=%d (max 65535)", in->B);
    const long long cap = (long long)in->max_pages * in->page;
    if (in->max_kv > cap)
        return fail(HSA_ERR_INVALID_ARG, "max_kv=%d is above max_pages * page = %lld", in->max_kv, cap);
    const long long max_kv = in->max_kv > 0 ? in->max_kv : cap;
    if (max_kv > MAX_POS || in->rows > MAX_POS) return fail(HSA_ERR_UNSUPPORTED, "positions must stay below 2^30");
    if ((long long)in->npages * in->page > INT_MAX || (long long)in->rows * in->H > (1ll << 33))
        return fail(HSA_ERR_UNSUPPORTED, "too many tokens for 32-bit rows");
    *a = LocArgs{};
    a->B = in->B;
    a->H = in->H;
    a->Hkv = in->Hkv;
    a->G = in->H / in->Hkv;
    a->d = in->d;
    a->max_q = in->max_q > 0 && in->max_q < in->rows ? in->max_q : in->rows;
    a->max_kv = (int)max_kv;
    a->rows = in->rows;
    a->paged = 1;
    a->page_shift = in->page == 16 ? 4 : in->page == 32 ? 5 : in->page == 64 ? 6 : 7;
    a->npages = in->npages;
    a->max_pages = in->max_pages;
    fill_mask(a, in->scale, in->window, in->sinks);
    return HSA_OK;
}

hsa_status_t check_ws(size_t need_bytes, void *ws, size_t ws_bytes) {
    if (ws_bytes < need_bytes)
        return fail(HSA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need_bytes);
    if (!ws) return fail(HSA_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws & 255u) return fail(HSA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    return HSA_OK;
}

// int32 arrays only need their element's alignment
hsa_status_t need4(const void *x, const char *name) {
    if (!x) return fail(HSA_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)x & 3u) return fail(HSA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return HSA_OK;
}

hsa_status_t run_forward(LocArgs &a, int dtype, unsigned flags, const void *Q, const void *K, const void *V, void *O,
                         void *ws, size_t ws_bytes, cudaStream_t st) {
    const LocPlan pl = plan_forward(a, dtype, (flags & HSA_FLAG_SIMT) != 0);
    HSA_TRY(check_ws(pl.need, ws, ws_bytes));
    if (a.B == 0 || a.rows == 0 || a.max_q == 0) return HSA_OK;
    a.status = (uint32_t *)ws;
    a.nsplit = pl.nsplit;
    a.opart = (float *)((char *)ws + pl.opart);
    a.lpart = (float *)((char *)ws + pl.lpart);
    a.tc_starts = pl.starts ? (long long *)((char *)ws + pl.starts) : nullptr;
    cudaError_t e = pl.few ? launch_few(a, Q, K, V, O, st)
                    : pl.tc ? launch_tc(a, Q, K, V, O, st)
                            : launch_simt(a, dtype, Q, K, V, O, st);
    if (e == cudaSuccess && a.nsplit > (pl.few ? FEW_CLUSTER : 1)) e = launch_combine(a, dtype, O, st);
    return e == cudaSuccess ? HSA_OK : cuda_fail(e, "local attention kernel launch");
}

}  // namespace

long long most_keys(const LocArgs &a, int tok) {
    if (a.window == INT32_MAX) return a.max_kv;
    const long long w = (long long)a.window + tok - 1 + a.sinks;
    return w < a.max_kv ? w : a.max_kv;
}

// The most bytes beyond the header that plan_forward of a call with a smaller (or equal) B, rows, max_q and max_kv can
// need, so that one workspace serves a server's batches of any size up to its largest.  Smaller calls are split
// more: below, items are work items, and a call of n of them gets at most 2 SMS / n splits.
static size_t forward_most(const LocArgs &a, int dtype, bool simt) {
    if (a.B == 0 || a.max_q == 0 || a.max_kv == 0) return 0;
    auto partials = [&](long long rows) {   // rows: of all heads and splits
        return rows > 0 ? align256((size_t)rows * a.d * sizeof(float)) + align256((size_t)rows * sizeof(float)) : 0;
    };
    auto least = [](long long x, long long y) { return x < y ? x : y; };
    const long long rows = (long long)a.max_q * a.G, heads = (long long)a.B * a.Hkv;
    if (simt || dtype != HSA_BF16) {
        // items of up to 32 rows (64 only where they fill the SMs unsplit), two key tiles per split at least
        const long long block = rows <= 16 ? 16 : 32, nt = ceil_div(most_keys(a, (int)(block / a.G)), 64) + 1;
        return nt / 2 < 2 || a.Hkv > SMS ? 0 : partials(least(2 * SMS * block, heads * rows * least(64, nt / 2)));
    }
    // few rows: partials beyond a cluster's splits
    const int tok = (int)least(a.max_q, 16 / a.G);
    const bool few = ceil_div(most_keys(a, tok), 64) + 1 >= 32 * FEW_CLUSTER && a.Hkv * FEW_CLUSTER < SMS;
    size_t most = few ? partials((long long)tok * a.G * least(2 * SMS, 64 * heads)) : 0;
    if (rows > 16) {
        const TcPlan t = tc_plan_most(a, most_keys(a, 2 * (128 / a.G)));
        const size_t n = align256(t.starts) + align256(t.opart) + align256(t.lpart);
        if (n > most) most = n;
    }
    return most;
}

LocPlan plan_forward(const LocArgs &a, int dtype, bool simt) {
    LocPlan p{};
    p.nsplit = 1;
    p.few = !simt && few_supported(a, dtype);
    p.tc = !p.few && !simt && tc_supported(a, dtype);
    if (p.few) {
        // CTAs of 64-key tiles, two per SM.  A cluster joins up to 8 splits in the same launch; more splits
        // (partials and a second launch, ~3 us) only where 8 leave most SMs without work for long.
        const long long items = (long long)a.Hkv * a.B;
        const int nt = ceil_div(most_keys(a, a.max_q), 64) + 1;
        long long n = items > 0 ? 2 * SMS / items : 1;
        if (n > FEW_CLUSTER && (nt < 32 * FEW_CLUSTER || items * FEW_CLUSTER >= SMS)) n = FEW_CLUSTER;
        if (n > nt) n = nt;
        if (n > 64) n = 64;
        if (n > 1) p.nsplit = (int)n;
    } else if (!p.tc) {
        const int tok = simt_rows(a) / a.G, bk = 64;
        const long long items = (long long)ceil_div(a.max_q, tok) * a.Hkv * a.B;
        // too few blocks to fill the SMs twice: the key axis is split over CTAs as well, two tiles each at least
        const int nt = ceil_div(most_keys(a, tok), bk) + 1;
        if (items > 0 && items < 2 * SMS) {
            int n = 2 * SMS / (int)items;
            if (n > nt / 2) n = nt / 2;
            if (n > 64) n = 64;
            if (n > 1) p.nsplit = n;
        }
    }
    size_t off = HDR;
    p.opart = p.lpart = off;
    if (p.tc) {
        const TcPlan t = tc_plan(a, most_keys(a, 2 * (128 / a.G)));
        if (t.shares) {
            p.starts = off;
            off += align256(t.starts);
            p.opart = off;
            off += align256(t.opart);
            p.lpart = off;
            off += align256(t.lpart);
        }
    } else if (p.nsplit > (p.few ? FEW_CLUSTER : 1)) {
        const size_t r = (size_t)a.B * a.max_q * a.H * p.nsplit;
        off += align256(r * a.d * sizeof(float));
        p.lpart = off;
        off += align256(r * sizeof(float));
    }
    p.need = off;
    const size_t most = HDR + forward_most(a, dtype, simt);
    p.total = off > most ? off : most;
    return p;
}

BwdPlan plan_backward(const LocArgs &a, int dtype, bool simt) {
    BwdPlan p{};
    p.tc = !simt && bwd_tc_supported(a, dtype);
    p.bk = p.tc ? 128 : 64;
    p.nkt = ceil_div(a.max_kv, p.bk);
    // few key tiles: their rows are shared between CTAs as well, two row tiles (tcgen05: four) each at least
    const int tok = 64 / a.G;                      // both paths' row tiles are 64 rows
    long long range = a.window < INT32_MAX ? (long long)a.window + p.bk : a.max_q;
    if (range > a.max_q) range = a.max_q;
    const long long items = (long long)a.B * a.Hkv * p.nkt, want = p.tc ? SMS : 2 * SMS;
    p.nwin = 1;
    if (items > 0 && items < want) {
        long long n = want / items, most = range / ((p.tc ? 4 : 2) * tok);
        if (n > most) n = most;
        if (n > 16) n = 16;
        if (n > 1) p.nwin = (int)n;
    }
    p.win_q = range > 0 ? ceil_div(ceil_div(range, p.nwin), tok) * tok : 1;
    const int sinks = a.sinks < a.max_kv ? a.sinks : a.max_kv;
    if (a.window < INT32_MAX && sinks > 0 && a.max_q > 0 && (long long)a.q_pos0 + a.max_q - 1 >= a.window) {
        p.nst = ceil_div(sinks, p.bk);
        // the far rows of a sink tile in chunks as long as the others, at most 64 of them over all sink tiles
        const int most = 64 / p.nst > 1 ? 64 / p.nst : 1;
        long long fq = p.win_q;
        if (fq < ceil_div(a.max_q, most)) fq = ceil_div(a.max_q, most);
        if (fq > a.max_q) fq = a.max_q;
        p.far_q = (int)fq;
        p.nfar = ceil_div(a.max_q, fq);
    }
    p.npt = p.nwin > 1 ? p.nkt : p.nst;
    size_t off = HDR;
    p.D = off;
    off += align256((size_t)a.rows * a.H * sizeof(float));
    p.part = off;
    if (p.npt > 0) off += align256(2 * (size_t)(p.nwin + p.nfar) * a.B * a.Hkv * p.npt * p.bk * a.d * sizeof(float));
    p.total = off;
    return p;
}

}  // namespace local
}  // namespace hsa

using namespace hsa;
using namespace hsa::local;

extern "C" {

hsa_status_t hsa_window_workspace_size(const hsa_window_t *prob, size_t *bytes) {
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    if (!bytes) return fail(HSA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = plan_forward(a, prob->dtype, (prob->flags & HSA_FLAG_SIMT) != 0).total;
    return HSA_OK;
}

hsa_status_t hsa_window_attend(const hsa_window_t *prob, const void *Q, const void *K, const void *V, void *O,
                               float *lse, void *ws, size_t ws_bytes, void *stream) {
    NvtxRange nvtx_("hsa_window_attend");
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    const bool rows = a.rows > 0;
    HSA_TRY(need(Q, rows, "Q"));
    HSA_TRY(need(K, rows && a.max_kv > 0, "K"));
    HSA_TRY(need(V, rows && a.max_kv > 0, "V"));
    HSA_TRY(need(O, rows, "O"));
    HSA_TRY(need(lse, lse != nullptr, "lse"));
    a.lse = lse;
    return run_forward(a, prob->dtype, prob->flags, Q, K, V, O, ws, ws_bytes, (cudaStream_t)stream);
}

hsa_status_t hsa_window_backward_workspace_size(const hsa_window_t *prob, size_t *bytes) {
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    if (!bytes) return fail(HSA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = plan_backward(a, prob->dtype, (prob->flags & HSA_FLAG_SIMT) != 0).total;
    return HSA_OK;
}

hsa_status_t hsa_window_backward(const hsa_window_t *prob, const void *Q, const void *K, const void *V, const void *O,
                                 const float *lse, const void *dO, void *dQ, void *dK, void *dV, void *ws,
                                 size_t ws_bytes, void *stream) {
    NvtxRange nvtx_("hsa_window_backward");
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    const bool rows = a.rows > 0, kv = (long long)a.B * a.Tcap > 0;
    HSA_TRY(need(Q, rows, "Q"));
    HSA_TRY(need(K, rows && a.max_kv > 0, "K"));
    HSA_TRY(need(V, rows && a.max_kv > 0, "V"));
    HSA_TRY(need(O, rows, "O"));
    HSA_TRY(need(lse, rows, "lse"));
    HSA_TRY(need(dO, rows, "dO"));
    HSA_TRY(need(dQ, rows, "dQ"));
    HSA_TRY(need(dK, kv, "dK"));
    HSA_TRY(need(dV, kv, "dV"));
    const BwdPlan pl = plan_backward(a, prob->dtype, (prob->flags & HSA_FLAG_SIMT) != 0);
    HSA_TRY(check_ws(pl.total, ws, ws_bytes));
    if (a.B == 0) return HSA_OK;
    cudaStream_t st = (cudaStream_t)stream;
    a.status = (uint32_t *)ws;
    a.nsplit = 1;
    a.lse = const_cast<float *>(lse);
    BwdArgs w{};
    w.a = a;
    w.nkt = pl.nkt;
    w.nwin = pl.nwin;
    w.win_q = pl.win_q;
    w.npt = pl.npt;
    w.nst = pl.nst;
    w.nfar = pl.nfar;
    w.far_q = pl.far_q;
    w.D = (float *)((char *)ws + pl.D);
    w.part = (float *)((char *)ws + pl.part);
    cudaError_t e = cudaSuccess;
    // tokens behind the cached ones, and all of them when there is no query
    const int tail = rows ? a.max_kv : 0;
    if (kv && tail < a.Tcap) {
        const size_t row = (size_t)a.Hkv * a.d * (prob->dtype == HSA_BF16 ? 2 : 4), pitch = row * a.Tcap;
        e = cudaMemset2DAsync((char *)dK + tail * row, pitch, 0, row * (a.Tcap - tail), a.B, st);
        if (e == cudaSuccess) e = cudaMemset2DAsync((char *)dV + tail * row, pitch, 0, row * (a.Tcap - tail), a.B, st);
    }
    if (e == cudaSuccess && rows) {
        const bool few = prob->dtype == HSA_BF16;
        if (!few || !few_rowdot_all(a)) e = launch_rowdot(a, prob->dtype, O, dO, w.D, st);
        if (e == cudaSuccess && few) e = launch_few_rowdot(a, Q, K, V, dO, w.D, st);
        if (e == cudaSuccess)
            e = pl.tc ? launch_bwd_tc(w, Q, K, V, dO, dQ, dK, dV, st)
                      : launch_bwd_simt(w, prob->dtype, Q, K, V, dO, dQ, dK, dV, st);
        if (e == cudaSuccess) e = launch_bwd_join(w, pl.bk, prob->dtype, dK, dV, st);
    }
    return e == cudaSuccess ? HSA_OK : cuda_fail(e, "local attention backward launch");
}

hsa_status_t hsa_rope_init(hsa_rope_t *r) {
    if (!r) return fail(HSA_ERR_INVALID_ARG, "rope is NULL");
    if (r->rot < 2 || r->rot > 128 || r->rot % 2) return fail(HSA_ERR_INVALID_ARG, "rot=%d must be even, 2 .. 128", r->rot);
    if (r->interleaved != 0 && r->interleaved != 1)
        return fail(HSA_ERR_INVALID_ARG, "interleaved=%d must be 0 or 1", r->interleaved);
    if (r->scaling < HSA_ROPE_NONE || r->scaling > HSA_ROPE_BANDS)
        return fail(HSA_ERR_INVALID_ARG, "unknown scaling %d", r->scaling);
    if (!(r->theta > 1.0) || isinf(r->theta)) return fail(HSA_ERR_INVALID_ARG, "theta must be finite and > 1");
    if (!(r->factor >= 1.0) || isinf(r->factor)) return fail(HSA_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (!(r->mscale >= 0.0) || isinf(r->mscale)) return fail(HSA_ERR_INVALID_ARG, "mscale must be finite and >= 0");
    const bool turns = r->scaling == HSA_ROPE_YARN || r->scaling == HSA_ROPE_BANDS;
    double low = r->low, high = r->high;
    if (turns) {
        if (r->orig_len < 1) return fail(HSA_ERR_INVALID_ARG, "orig_len=%d must be >= 1 for this scaling", r->orig_len);
        if (low == 0.0 && high == 0.0) {
            low = 1.0;
            high = r->scaling == HSA_ROPE_YARN ? 32.0 : 4.0;
        }
        if (!(low > 0.0) || !(high > low) || isinf(high))
            return fail(HSA_ERR_INVALID_ARG, "0 < low < high is needed (low=%g high=%g)", low, high);
    }
    if (r->scaling == HSA_ROPE_NTK && r->rot == 2)
        return fail(HSA_ERR_INVALID_ARG, "NTK scaling needs rot > 2");
    const double TWO_PI = 6.283185307179586476925286766559, n = r->rot;
    const double theta = r->scaling == HSA_ROPE_NTK ? r->theta * pow(r->factor, n / (n - 2.0)) : r->theta;
    double lo = 0, hi = 0;
    if (r->scaling == HSA_ROPE_YARN) {
        // the pair index that makes t turns within orig_len: n ln(orig_len / 2 pi t) / (2 ln theta)
        lo = floor(n * log(r->orig_len / (high * TWO_PI)) / (2.0 * log(theta)));
        hi = ceil(n * log(r->orig_len / (low * TWO_PI)) / (2.0 * log(theta)));
        if (lo < 0) lo = 0;
        if (hi > n - 1) hi = n - 1;
    }
    for (int i = 0; i < 64; ++i) {
        double f = 0.0;
        if (i < r->rot / 2) {
            f = pow(theta, -2.0 * i / n);
            if (r->scaling == HSA_ROPE_LINEAR) {
                f /= r->factor;
            } else if (r->scaling == HSA_ROPE_YARN) {
                double u = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
                u = u < 0 ? 0 : u > 1 ? 1 : u;
                f = u * f / r->factor + (1.0 - u) * f;
            } else if (r->scaling == HSA_ROPE_BANDS) {
                const double t = r->orig_len * f / TWO_PI;
                double u = (t - low) / (high - low);
                u = u < 0 ? 0 : u > 1 ? 1 : u;
                f = (1.0 - u) * f / r->factor + u * f;
            }
        }
        r->inv_freq[i] = f;
    }
    r->mult = r->mscale > 0.0 ? r->mscale : r->scaling == HSA_ROPE_YARN ? 0.1 * log(r->factor) + 1.0 : 1.0;
    return HSA_OK;
}

}  // extern "C"

namespace {

hsa_status_t check_head_count(long long heads) {
    if (heads > 16383) return fail(HSA_ERR_UNSUPPORTED, "%lld heads in one call (max 16383)", heads);
    return HSA_OK;
}

hsa_status_t rope_args(const hsa_rope_t *rope, int d, RopeArgs *r) {
    if (!rope) return fail(HSA_ERR_INVALID_ARG, "rope is NULL");
    if (rope->rot < 2 || rope->rot > d || rope->rot % 2)
        return fail(HSA_ERR_INVALID_ARG, "rot=%d must be even and at most d=%d", rope->rot, d);
    if (!(rope->mult > 0.0)) return fail(HSA_ERR_INVALID_ARG, "rope was not set up by hsa_rope_init");
    for (int i = 0; i < 64; ++i) r->f[i] = rope->inv_freq[i] * 0.15915494309189533576888376337251;   // turns per token
    r->mult = (float)rope->mult;
    r->rot = rope->rot;
    r->interleaved = rope->interleaved;
    r->sgn = 1.f;
    return HSA_OK;
}

}  // namespace

extern "C" {

hsa_status_t hsa_rope(const hsa_rope_t *rope, const hsa_window_t *prob, const int32_t *pos, int inverse, const void *Q,
                      const void *K, void *Qr, void *Kr, void *stream) {
    NvtxRange nvtx_("hsa_rope");
    if (!prob) return fail(HSA_ERR_INVALID_ARG, "problem pointer is NULL");
    hsa_window_t pr{};   // the fields that count here; the others may hold anything
    pr.B = prob->B;
    pr.Tq = prob->Tq;
    pr.H = pr.Hkv = 1;   // the two head counts have nothing to do with each other here
    pr.d = prob->d;
    pr.q_pos0 = prob->q_pos0;
    pr.dtype = prob->dtype;
    LocArgs a;
    HSA_TRY(shape_of(&pr, &a));
    const long long H = prob->H, Hkv = prob->Hkv;
    if (H < 1 || Hkv < 1) return fail(HSA_ERR_INVALID_ARG, "H, Hkv must be >= 1 (H=%lld Hkv=%lld)", H, Hkv);
    RopeArgs r;
    HSA_TRY(rope_args(rope, a.d, &r));
    HSA_TRY(check_head_count((Q ? H : 0) + (K ? Hkv : 0)));
    const bool rows = a.rows > 0;
    if (rows && !Q && !K) return fail(HSA_ERR_INVALID_ARG, "Q and K are both NULL");
    HSA_TRY(need(Q, Q != nullptr, "Q"));
    HSA_TRY(need(K, K != nullptr, "K"));
    HSA_TRY(need(Qr, rows && Q, "Qr"));
    HSA_TRY(need(Kr, rows && K, "Kr"));
    if (pos) HSA_TRY(need4(pos, "pos"));
    if (!rows) return HSA_OK;
    if (inverse) r.sgn = -1.f;
    cudaError_t e = launch_rope(r, prob->dtype, a.B, a.max_q, (int)H, (int)Hkv, a.d, a.q_pos0, pos, Q, K, Qr, Kr,
                                (cudaStream_t)stream);
    return e == cudaSuccess ? HSA_OK : cuda_fail(e, "rope kernel launch");
}

hsa_status_t hsa_paged_append(const hsa_paged_t *prob, const hsa_rope_t *rope, const void *k_new, const void *v_new,
                              const void *Q, void *Qr, const int32_t *q_start, const int32_t *kv_len,
                              const int32_t *table, void *Kp, void *Vp, void *ws, size_t ws_bytes, void *stream) {
    NvtxRange nvtx_("hsa_paged_append");
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    RopeArgs r;
    if (rope) HSA_TRY(rope_args(rope, a.d, &r));
    HSA_TRY(check_head_count((Q ? a.H : 0) + 2ll * a.Hkv));
    const bool any = a.rows > 0 && a.B > 0;
    HSA_TRY(need(k_new, any, "k_new"));
    HSA_TRY(need(v_new, any, "v_new"));
    HSA_TRY(need(Kp, any, "Kp"));
    HSA_TRY(need(Vp, any, "Vp"));
    HSA_TRY(need(Q, Q != nullptr, "Q"));
    HSA_TRY(need(Qr, any && Q, "Qr"));
    if (any) {
        HSA_TRY(need4(q_start, "q_start"));
        HSA_TRY(need4(kv_len, "kv_len"));
        HSA_TRY(need4(table, "table"));
    }
    HSA_TRY(check_ws(HDR, ws, ws_bytes));
    if (!any) return HSA_OK;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.status = (uint32_t *)ws;
    cudaError_t e = launch_append(rope ? &r : nullptr, a, prob->dtype, k_new, v_new, Q, Qr, Kp, Vp, (cudaStream_t)stream);
    return e == cudaSuccess ? HSA_OK : cuda_fail(e, "paged append kernel launch");
}

hsa_status_t hsa_paged_workspace_size(const hsa_paged_t *prob, size_t *bytes) {
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    if (!bytes) return fail(HSA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = plan_forward(a, prob->dtype, (prob->flags & HSA_FLAG_SIMT) != 0).total;
    return HSA_OK;
}

hsa_status_t hsa_paged_attend(const hsa_paged_t *prob, const void *Q, const void *Kp, const void *Vp,
                              const int32_t *q_start, const int32_t *kv_len, const int32_t *table, void *O, void *ws,
                              size_t ws_bytes, void *stream) {
    NvtxRange nvtx_("hsa_paged_attend");
    LocArgs a;
    HSA_TRY(shape_of(prob, &a));
    const bool any = a.rows > 0 && a.B > 0;
    HSA_TRY(need(Q, any, "Q"));
    HSA_TRY(need(Kp, any, "Kp"));
    HSA_TRY(need(Vp, any, "Vp"));
    HSA_TRY(need(O, any, "O"));
    if (any) {
        HSA_TRY(need4(q_start, "q_start"));
        HSA_TRY(need4(kv_len, "kv_len"));
        HSA_TRY(need4(table, "table"));
    }
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    return run_forward(a, prob->dtype, prob->flags, Q, Kp, Vp, O, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
