// local.cuh -- shared pieces of the local attention (sliding window with
// sinks, contiguous or paged K/V): the kernels' view of a call, the geometry of
// its visibility mask in key tiles, and the internal launch interface.
#pragma once

#include "common.cuh"

namespace hsa {
namespace local {

// One call of hsa_window_attend or hsa_paged_attend as the kernels see it.
// Rows are (token, head of the group) pairs of one kv head; tokens of all
// sequences are numbered row0(b) + t.
struct LocArgs {
    int B, H, Hkv, G, d;
    int max_q;             // most new tokens of one sequence (contiguous: Tq)
    int max_kv;            // most cached tokens of one sequence (contiguous: Tkv)
    int rows;              // tokens in Q / O over all sequences
    int Tcap;              // contiguous: K/V tokens per sequence
    int q_pos0;            // contiguous: position of row 0
    int window;            // INT32_MAX = none
    int sinks;
    float scale, scale_log2;
    int paged, page_shift, npages, max_pages;
    const int32_t *q_start, *kv_len, *table;
    int nsplit;            // key-axis splits per (sequence, kv head, row tile)
    int by_rows;           // CUDA-core forward: row tiles numbered over all sequences (tile_by_row)
    float *opart, *lpart;  // split partials: [nsplit][B][max_q][H][d] and [nsplit][B][max_q][H] (tcgen05: by slot)
    long long *tc_starts;  // tcgen05: starts of the blocks' key tiles when CTAs take equal shares of them; else null
    float *lse;            // optional output
    uint32_t *status;
};

// One sequence of the call.
struct Seq {
    int row0, n;    // its tokens in Q / O
    int pos0, kv;   // position of its first token (may be negative), cached tokens
};

__device__ __forceinline__ Seq seq_of(const LocArgs &a, int b) {
    Seq s;
    if (!a.paged) {
        s.row0 = b * a.max_q;
        s.n = a.max_q;
        s.pos0 = a.q_pos0;
        s.kv = a.max_kv;
        return s;
    }
    // lengths are device data: anything outside the call's bounds is cut to them and recorded
    const int r0 = a.q_start[b], r1 = a.q_start[b + 1], kv = a.kv_len[b];
    s.row0 = min(max(r0, 0), a.rows);
    const int r1c = min(max(r1, s.row0), a.rows);
    s.n = min(r1c - s.row0, a.max_q);
    s.kv = min(max(kv, 0), a.max_kv);
    s.pos0 = s.kv - s.n;
    if (s.row0 != r0 || s.row0 + s.n != r1 || s.kv != kv) atomicOr(a.status, DEV_BAD_INDEX);
    return s;
}

// Row tiles of `tok` tokens numbered over all sequences: those of sequence b start at q_start[b] / tok + b, which leaves
// each room enough (rounding down may leave one too many).  False: tile x has no tokens.
__device__ __forceinline__ bool tile_by_row(const LocArgs &a, int x, int tok, int *b, int *blk) {
    auto first = [&](int i) { return min(max(a.q_start[i], 0), a.rows) / tok + i; };
    int lo = 0, hi = a.B - 1;   // the last b that starts at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    *b = lo;
    *blk = x - first(lo);
    return *blk >= 0;
}

// Row of the K/V tensors (in tokens) that holds token u of sequence b, or -1
// if its page number is outside the pool.
__device__ __forceinline__ long long kv_row(const LocArgs &a, int b, int u) {
    if (!a.paged) return (long long)b * a.Tcap + dbg_clamp(u, 0, a.Tcap, a.status);
    const int at = (int)dbg_clamp(u >> a.page_shift, 0, a.max_pages, a.status);
    const int pg = a.table[(long long)b * a.max_pages + at];
    if ((unsigned)pg >= (unsigned)a.npages) {
        atomicOr(a.status, DEV_BAD_INDEX);
        return -1;
    }
    return ((long long)pg << a.page_shift) + (u & ((1 << a.page_shift) - 1));
}

// First row of the split partials of token t of sequence b (one row per head).  Numbered by sequence, not by row of Q:
// rows behind the last sequence, of which there may be any number, have none.
__device__ __forceinline__ long long part_row(const LocArgs &a, int split, int b, int t) {
    return (((long long)split * a.B + b) * a.max_q + t) * a.H;
}

__host__ __device__ __forceinline__ bool visible(int p, int u, int kv, int window, int sinks) {
    return u <= p && u < kv && (p - u < window || u < sinks);
}

// The key tiles (BK keys each, aligned to BK) that the queries at positions
// pa .. pb reach: first those that only hold sinks, then the window's.
struct Tiles {
    int lo, hi;       // window keys [lo, hi)
    int ns;           // sink keys [0, ns) before the window (ns <= lo)
    int nst, wt0, nt; // tiles of the sinks, first window tile, tiles in all
    __host__ __device__ __forceinline__ int tile(int i) const { return i < nst ? i : wt0 + i - nst; }
};

template <int BK> __host__ __device__ __forceinline__ Tiles tiles_of(int pa, int pb, int kv, int window, int sinks) {
    Tiles t;
    t.hi = pb + 1 < kv ? pb + 1 : kv;
    if (t.hi < 0) t.hi = 0;
    t.lo = pa >= window ? pa - window + 1 : 0;   // window may be INT32_MAX
    if (t.lo > t.hi) t.lo = t.hi;
    t.ns = sinks < t.lo ? sinks : t.lo;
    t.wt0 = t.lo / BK;
    const int wt1 = t.hi > t.lo ? (t.hi + BK - 1) / BK : t.wt0;
    t.nst = (t.ns + BK - 1) / BK;
    if (t.hi > t.lo && t.nst > t.wt0) t.nst = t.wt0;   // the first window tile holds the last sinks too
    t.nt = t.nst + wt1 - t.wt0;
    return t;
}

// Keys of tile [u0, u0 + BK) that some query of the block sees lie in [a, b) or below ns.
// (Others are loaded as zeros: nothing of theirs reaches a sum, NaN included.)
__host__ __device__ __forceinline__ bool key_live(const Tiles &t, int u) { return u < t.hi && (u >= t.lo || u < t.ns); }

// Split s of the nt tiles: [i0, i1).
__host__ __device__ __forceinline__ void split_range(int nt, int nsplit, int s, int *i0, int *i1) {
    const int per = (nt + nsplit - 1) / nsplit;
    *i0 = s * per < nt ? s * per : nt;
    *i1 = *i0 + per < nt ? *i0 + per : nt;
}

// Backward, dK and dV: the work items of a key tile.  The queries inside its window are
// cut into nwin chunks of win_q tokens (1 unless few tiles would leave SMs idle); the key tiles
// that hold sinks are seen by every later query too, in nfar more chunks of far_q tokens.  A
// tile of several items is written as fp32 partials, one slot per item, that bwd_join_kernel adds
// in slot order.
struct BwdArgs {
    LocArgs a;                       // contiguous view; a.lse = the forward's
    int nkt;                         // key tiles over Tkv
    int nwin, win_q;
    int nst;                         // key tiles that hold sinks and have a far part (0: none)
    int nfar, far_q;
    int npt;                         // key tiles written as partials: the first npt
    float *D;                        // [B][Tq][H] row sums of dO o O (few keys: of P o dP)
    float *part;                     // [2 (dK, dV)][nwin + nfar][B][Hkv][npt * BK][d]
};

// Work item x (of nkt * nwin + nst * nfar): its key tile, its slot and its query tokens [ta, tb).
struct KvRange {
    int kt, slot, ta, tb;
};
__host__ __device__ __forceinline__ KvRange kv_range(const BwdArgs &w, const Seq &s, int x, int bk) {
    KvRange r;
    const bool far = x >= w.nkt * w.nwin;
    int c;
    if (far) {
        x -= w.nkt * w.nwin;
        r.kt = x / w.nfar;
        c = x % w.nfar;
        r.slot = w.nwin + c;
    } else {
        r.kt = x / w.nwin;
        r.slot = c = x % w.nwin;
    }
    const int u0 = r.kt * bk, ul = (u0 + bk < s.kv ? u0 + bk : s.kv) - 1;
    const long long n = s.n, t0 = u0 > s.pos0 ? u0 - s.pos0 : 0;
    // first token beyond the window of every key of the tile
    long long edge = w.a.window < INT32_MAX ? (long long)ul + w.a.window - s.pos0 : n;
    edge = edge < 0 ? 0 : edge > n ? n : edge;
    long long lo = far ? (edge > t0 ? edge : t0) : t0;
    const long long hi = far ? n : edge, step = far ? w.far_q : w.win_q;
    lo += c * step;
    const long long end = lo + step < hi ? lo + step : hi;
    r.ta = (int)(lo < n ? lo : n);
    r.tb = (int)(end > r.ta ? end : r.ta);
    return r;
}

struct LocPlan {
    bool tc, few;          // forward path: tcgen05 tiles, few-row kernel; neither: CUDA-core tiles
    int nsplit;
    size_t opart, lpart, starts;   // offsets; starts 0: no shares
    size_t need, total;            // what this call uses; enough for every call of smaller B, rows, max_q and max_kv too
};
LocPlan plan_forward(const LocArgs &a, int dtype, bool simt);

struct BwdPlan {
    bool tc;
    int nkt, nwin, win_q, nst, nfar, far_q, npt, bk;
    size_t D, part, total;
};
BwdPlan plan_backward(const LocArgs &a, int dtype, bool simt);

int simt_rows(const LocArgs &a);   // rows per block of the CUDA-core forward: 16, 32 or 64
cudaError_t launch_simt(const LocArgs &a, int dtype, const void *Q, const void *K, const void *V, void *O,
                        cudaStream_t st);
constexpr int FEW_CLUSTER = 8;   // splits that the few-row kernel joins within a cluster
bool few_supported(const LocArgs &a, int dtype);
cudaError_t launch_few(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st);
bool tc_supported(const LocArgs &a, int dtype);
struct TcPlan {
    bool shares;                    // CTAs take equal shares of all key tiles; else whole items
    size_t starts, opart, lpart;    // bytes
};
TcPlan tc_plan(const LocArgs &a, long long most_keys);   // most_keys: that one block can see
TcPlan tc_plan_most(const LocArgs &a, long long most_keys);   // the most that tc_plan of a smaller call can need
cudaError_t launch_tc(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st);
cudaError_t launch_combine(const LocArgs &a, int dtype, void *O, cudaStream_t st);
cudaError_t launch_rowdot(const LocArgs &a, int dtype, const void *O, const void *dO, float *D, cudaStream_t st);
// bf16: D of the rows that see few keys
bool few_rowdot_all(const LocArgs &a);   // that is every row
cudaError_t launch_few_rowdot(const LocArgs &a, const void *Q, const void *K, const void *V, const void *dO, float *D,
                              cudaStream_t st);
cudaError_t launch_bwd_simt(const BwdArgs &w, int dtype, const void *Q, const void *K, const void *V, const void *dO,
                            void *dQ, void *dK, void *dV, cudaStream_t st);
bool bwd_tc_supported(const LocArgs &a, int dtype);
cudaError_t launch_bwd_tc(const BwdArgs &w, const void *Q, const void *K, const void *V, const void *dO, void *dQ,
                          void *dK, void *dV, cudaStream_t st);
cudaError_t launch_bwd_join(const BwdArgs &w, int bk, int dtype, void *dK, void *dV, cudaStream_t st);

struct RopeArgs {
    double f[64];
    float mult;
    int rot, interleaved;
    float sgn;             // +1 forward, -1 transpose
};
cudaError_t launch_rope(const RopeArgs &r, int dtype, int B, int T, int H, int Hkv, int d, int pos0,
                        const int32_t *pos, const void *Q, const void *K, void *Qr, void *Kr, cudaStream_t st);
cudaError_t launch_append(const RopeArgs *r, const LocArgs &a, int dtype, const void *k, const void *v, const void *Q,
                          void *Qr, void *Kp, void *Vp, cudaStream_t st);

}  // namespace local
}  // namespace hsa
