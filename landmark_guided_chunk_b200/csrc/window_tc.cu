// window_tc.cu -- sliding-window attention with sinks on tcgen05: bf16 rows by
// the hundred (prompts, chunks of new tokens), contiguous or paged K/V.
//
// A persistent CTA per SM takes work items: two tiles of 128 rows of one kv head
// (row = token x query head of the group, so the G heads of a group share each
// K/V tile) against the key tiles (128 keys) that the two tiles' window reaches.
// One pass with a running maximum m and sum l per row:
//   S = Q K^T (TMEM), P = exp2(scale_log2 S - m), l += sum P, O += P V (TMEM)
// m is only moved, and O rescaled by 2^(m_old - m_new), when a row's maximum has
// grown by more than 8 in log2: any reference gives the same quotient O / l, P
// stays below 2^8, and most tiles then need no pass over O.
//
// Roles: two softmax warpgroups (one per row tile, thread = row), a loader warp
// (TMA), an MMA warp, and a warp that zeroes dead V rows of tiles at the edges of
// the visible range (what no query sees must not reach a sum: 0 x NaN).  The MMA
// warp alternates the tiles: PV0(i) QK0(i+1) PV1(i) QK1(i+1), so one tile's
// softmax runs under the other's products.  P overwrites S in TMEM as bf16 and is
// the A operand of PV from there.
//
// Bound: the chain scores, softmax, product, next scores of a row tile.  A pair of tiles takes about 3400 cycles, its
// products 2080; with no softmax arithmetic at all the loop still takes 781 of 890 us (16384 tokens, window 4096).
// 32 + 8 heads of 128, sinks 4: 65536 tokens, window 4096: 4.4 ms among calls with new inputs, 0.97 PFLOP/s of visible
// pairs (58% of the measured 1.68; 3.9 ms while the clock holds); 16384 tokens: 0.90 ms; window 512: 0.215 ms (a
// fifth of its keys are masked and an item's start and end cost four key tiles); head dim 64, window 4096: 0.82 ms.
#include <limits.h>

#include "local.cuh"
#include "local_sm100.cuh"

namespace hsa {
namespace local {

namespace {

using namespace sm100;

constexpr int BK = 128;          // keys per tile
constexpr int MR = 128;          // rows per tile
constexpr int NT = 384;
constexpr float RESCALE = 8.f;   // growth of the maximum (log2) that is let pass

template <int D> struct Cfg {
    static constexpr int NBX = D / 64;                 // 64-column boxes per row
    static constexpr int TILE = 128 * D * 2;           // bytes of a Q, K or V tile
    static constexpr int QB = 2;                       // buffers of the two Q tiles
    static constexpr int NST = D == 128 ? 3 : 8;       // K/V ring stages (one Q buffer and 5 stages: 908 -> 927 us)
};

struct Share {
    int g, j, i, left;   // block, kv head, key tile to start with; key tiles to take
};

struct __align__(8) Bars {
    uint64_t q_full[2][2], q_empty[2][2], kv_full[8], kv_empty[8], land[8];   // q: [buffer][tile]
    uint64_t s_full[2], p_full[2][2], o_full[2], done;                        // p: [tile][half of its keys]
    uint64_t out_full[2][2];      // [Q buffer][tile]: the next item's output may be ready before this one's is looked for
    uint32_t tmem_base;
    uint32_t step;                // K and V tiles that the loader has issued
    int abort;
    Share share;
    int row[2][MR];               // token of each row's output (-1: padding)
};

// The key tiles of an item: the sinks' (from 0), then the window's, which start at
// its first key (paged: at that key's page) and not at a multiple of 128, so that a
// short window takes few of them.  A last tile is cut to a multiple of 16 keys.
struct KeyTiles {
    int lo, hi, ns;      // live keys: [lo, hi) and [0, ns), ns <= lo
    int send, base;      // sink tiles cover [0, send), window tiles [base, hi)
    int nst, nt;
    __device__ __forceinline__ int start(int i) const { return i < nst ? i * BK : base + (i - nst) * BK; }
    __device__ __forceinline__ int width(int i) const {
        const int n = (i < nst ? send : hi) - start(i);
        return n >= BK ? BK : (n + 15) & ~15;
    }
    __device__ __forceinline__ bool live(int u) const { return u < hi && (u >= lo || u < ns); }
    // keys of the tile that are brought in though no query of the item sees them
    __device__ __forceinline__ bool has_dead(int i) const {
        const int u0 = start(i), u1 = u0 + width(i);
        return i < nst ? u1 > ns : u1 > hi || (u0 < lo && !(ns >= lo));
    }
};

__device__ __forceinline__ KeyTiles key_tiles(int pa, int pb, int kv, int window, int sinks, int align) {
    KeyTiles t;
    t.hi = max(0, min(pb + 1, kv));
    t.lo = min(pa >= window ? pa - window + 1 : 0, t.hi);   // window may be INT32_MAX
    t.ns = min(sinks, t.lo);
    t.base = t.lo & ~(align - 1);
    t.send = min(t.ns, t.base);
    if (t.hi == t.lo) t.base = t.hi, t.send = t.ns;
    t.nst = (t.send + BK - 1) / BK;
    t.nt = t.nst + (t.hi - t.base + BK - 1) / BK;
    return t;
}

struct Item {
    int b, j, t0, ntile;          // ntile: row tiles with tokens (0: nothing to do)
    int i0, i1;                   // key tiles to do
    int slot;                     // partials' slot of an item that is shared with other CTAs; -1: all of it is this CTA's
    Seq s;
    KeyTiles tl;
};

// Block g of two row tiles: (sequence, block of 2 tok tokens); without a window, later blocks see more keys:
// longest first.
__device__ __forceinline__ void block_of(const LocArgs &a, int g, int tok, int nblk, Item *it) {
    const int blk = nblk - 1 - g % nblk;
    it->b = g / nblk;
    it->s = seq_of(a, it->b);
    it->t0 = blk * 2 * tok;
    const int left = it->s.n - it->t0;
    it->ntile = left <= 0 ? 0 : left <= tok ? 1 : 2;
    const int pa = it->s.pos0 + it->t0, pb = it->s.pos0 + min(it->s.n, it->t0 + 2 * tok) - 1;
    it->tl = key_tiles(pa, pb, it->s.kv, a.window, a.sinks, a.paged ? 1 << a.page_shift : 1);
    if (it->ntile == 0) it->tl.nt = 0;
}

// Which items a CTA takes.  Many items: every gridDim.x-th one.  Few: the key tiles of all items in a row, cut into
// equal shares, one per CTA (lengths differ, and whole items would leave most SMs waiting for the longest); an item
// that a cut goes through is written as partials and joined by join_kernel.
// LOOSE steps over a sequence's blocks without tokens, which come first: for paged calls whose max_q is far above most
// sequences' tokens (launch_tc).
template <bool LOOSE> struct Walk {
    Share s;             // shares: what is left; else s.g: the next item
    bool first;
    __device__ __forceinline__ bool next(const LocArgs &a, bool shares, int tok, int nblk, int nitems, Item *it) {
        if (!shares) {
            if (s.g >= nitems) return false;
            it->j = s.g % a.Hkv;
            block_of(a, s.g / a.Hkv, tok, nblk, it);
            it->i0 = 0;
            it->i1 = it->tl.nt;
            it->slot = -1;
            if (LOOSE && it->ntile == 0) {   // past this item and the others
                const int first = (it->b * nblk + nblk - (it->s.n + 2 * tok - 1) / (2 * tok)) * a.Hkv;
                s.g += (first - s.g - 1) / (int)gridDim.x * (int)gridDim.x;
            }
            s.g += gridDim.x;
            return true;
        }
        if (s.left <= 0) return false;
        int weight;
        while (true) {
            block_of(a, s.g, tok, nblk, it);
            weight = it->ntile == 0 ? 0 : max(it->tl.nt, 1);   // a block that sees no key still writes its zeros
            if (weight > 0) break;
            ++s.g;
        }
        const int take = min(s.left, weight - s.i);
        it->j = s.j;
        it->i0 = s.i;
        it->i1 = min(s.i + take, it->tl.nt);
        it->slot = take < weight ? 2 * (int)blockIdx.x + (first ? 0 : 1) : -1;
        first = false;
        s.left -= take;
        s.i += take;
        if (s.i == weight) {
            s.i = 0;
            if (++s.j == a.Hkv) {
                s.j = 0;
                ++s.g;
            }
        }
        return true;
    }
};

constexpr int SHARE_LEAST = 8;   // key tiles per CTA at least: a cut's partials and their join cost about four

// One warp: the sum of all blocks' tiles times kv heads, and this CTA's share of them.  CTA 0 leaves the blocks'
// starts in `starts` (int64 [blocks + 1], then the tiles per CTA) for the join.
__device__ __forceinline__ Share find_share(const LocArgs &a, int tok, int nblk, long long *starts) {
    const int lane = threadIdx.x & 31, nb = a.B * nblk;
    auto weight_of = [&](int g) -> int {
        if (g >= nb) return 0;
        Item it;
        block_of(a, g, tok, nblk, &it);
        return it.ntile == 0 ? 0 : max(it.tl.nt, 1) * a.Hkv;
    };
    long long total = 0;
    for (int g0 = 0; g0 < nb; g0 += 32) total += __reduce_add_sync(FULL, (unsigned)weight_of(g0 + lane));
    const long long per = max((long long)SHARE_LEAST, (total + gridDim.x - 1) / gridDim.x);   // tiles per CTA
    const int c = blockIdx.x;
    Share sh{0, 0, 0, 0};
    const long long s0 = min(total, c * per), s1 = min(total, s0 + per);
    long long at = 0;
    for (int g0 = 0; g0 < nb; g0 += 32) {
        const int wl = weight_of(g0 + lane);
        int inc = wl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += y;
        }
        const long long before = at + inc - wl;
        if (c == 0 && g0 + lane < nb) starts[g0 + lane] = before;
        if (s0 < s1 && wl > 0 && before <= s0 && s0 < before + wl) {
            const int tiles = wl / a.Hkv, off = (int)(s0 - before);
            sh.g = g0 + lane;
            sh.j = off / tiles;
            sh.i = off % tiles;
            sh.left = (int)(s1 - s0);
        }
        at += __shfl_sync(FULL, inc, 31);
    }
    if (c == 0 && lane == 0) {
        starts[nb] = total;
        starts[nb + 1] = per;
    }
    sh.g = (int)__reduce_max_sync(FULL, (unsigned)sh.g);   // one lane has found it, the others hold zeros
    sh.j = (int)__reduce_max_sync(FULL, (unsigned)sh.j);
    sh.i = (int)__reduce_max_sync(FULL, (unsigned)sh.i);
    sh.left = (int)__reduce_max_sync(FULL, (unsigned)sh.left);
    return sh;
}

constexpr int JOIN_ROWS = 4;   // blocks per row tile

// Joins the partials of the items that the shares cut: O = sum exp(lse_i - lse) O_i, in order of the pieces.  Four
// blocks per (item, row tile).
template <int D>
__global__ void __launch_bounds__(256)
    window_join_kernel(const __grid_constant__ LocArgs a, __nv_bfloat16 *__restrict__ O, int tok, int nblk, const long long *starts) {
    const int nb = a.B * nblk, g = blockIdx.x / a.Hkv, j = blockIdx.x % a.Hkv;
    const int t = blockIdx.y / JOIN_ROWS, r0 = blockIdx.y % JOIN_ROWS * (MR / JOIN_ROWS);   // row tile, first of its rows here
    const long long s = starts[g], e = starts[g + 1], per = starts[nb + 1];
    if (e == s) return;
    const long long tiles = (e - s) / a.Hkv, i0 = s + j * tiles, i1 = i0 + tiles;
    // CTA of a tile (exact: both numbers are far below 2^53)
    auto cta_of = [&](long long x) -> int { return (int)((double)x / (double)per); };
    const int c0 = cta_of(i0), pieces = cta_of(i1 - 1) - c0 + 1;
    if (pieces == 1) return;
    // the piece is its CTA's first item unless that CTA started before it
    __shared__ int slot[148];
    if (threadIdx.x < pieces)
        slot[threadIdx.x] = 2 * (c0 + (int)threadIdx.x) + ((c0 + (int)threadIdx.x) * per >= i0 ? 0 : 1);
    __syncthreads();
    Item it;
    block_of(a, g, tok, nblk, &it);
    // a thread: four columns of every 256 / (D / 4)-th row
    constexpr int TPR = D / 4, RPB = 256 / TPR;
    const int col = threadIdx.x % TPR * 4;
#pragma unroll 2
    for (int r = r0 + threadIdx.x / TPR; r < min(r0 + MR / JOIN_ROWS, tok * a.G); r += RPB) {
        const int token = it.t0 + t * tok + r / a.G;
        if (token >= it.s.n) continue;
        const long long rt = t * MR + r;
        float mx = -INFINITY;
        for (int k = 0; k < pieces; ++k) mx = fmaxf(mx, a.lpart[(long long)slot[k] * 2 * MR + rt]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        if (mx != -INFINITY) {
#pragma unroll 4
            for (int k = 0; k < pieces; ++k) {
                const long long at = (long long)slot[k] * 2 * MR + rt;
                const float w = expf(a.lpart[at] - mx);
                const float4 v = *reinterpret_cast<const float4 *>(a.opart + at * D + col);
                l += w;
                acc.x = fmaf(w, v.x, acc.x);
                acc.y = fmaf(w, v.y, acc.y);
                acc.z = fmaf(w, v.z, acc.z);
                acc.w = fmaf(w, v.w, acc.w);
            }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long row = (long long)(it.s.row0 + token) * a.H + j * a.G + r % a.G;
        *reinterpret_cast<uint2 *>(O + row * D + col) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (col == 0 && a.lse) a.lse[row] = l > 0.f ? mx + logf(l) : -INFINITY;
    }
}

template <int D, bool LOOSE>
__global__ void __launch_bounds__(NT, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      __nv_bfloat16 *__restrict__ O,
                      const __grid_constant__ LocArgs a, int tok, int nblk, int nitems, long long *starts) {
    typedef Cfg<D> C;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base;                       // QB buffers x 2 tiles: Q, then the item's output
    uint8_t *sKV = base + 2 * C::QB * C::TILE;   // NST tiles
    Bars *bar = reinterpret_cast<Bars *>(sKV + C::NST * C::TILE);
    volatile int *abort = &bar->abort;
    volatile uint32_t *step = &bar->step;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // rows that no box covers (G does not divide 128) stay zero
    for (int i = threadIdx.x; i < 2 * C::QB * C::TILE / 16; i += NT) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            for (int x = 0; x < 2; ++x) {
                mbar_init(&bar->q_full[x][t], 1);
                mbar_init(&bar->q_empty[x][t], 1);
                mbar_init(&bar->p_full[t][x], 4);
                mbar_init(&bar->out_full[x][t], 4);
            }
            mbar_init(&bar->s_full[t], 1);
            mbar_init(&bar->o_full[t], 1);
        }
        for (int s = 0; s < C::NST; ++s) {
            mbar_init(&bar->kv_full[s], 1);
            mbar_init(&bar->kv_empty[s], 1);
            mbar_init(&bar->land[s], 1);
        }
        mbar_init(&bar->done, 1);
        bar->step = 0;
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bar->tmem_base, 512);
        tmem_relinquish();
    }
    const bool shares = starts != nullptr;
    if (warp == 10) {
        const Share sh = shares ? find_share(a, tok, nblk, starts) : Share{(int)blockIdx.x, 0, 0, 0};
        if (lane == 0) bar->share = sh;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: S/P tiles at 0 and 128, O tiles at 256 and 256 + D

    if (warp < 8) {
        reg_inc<216>();
        // ---------------------------------------------------------------- softmax: thread = row of tile t
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sS = tmem + lane_off + t * 128, sO = tmem + lane_off + 256 + t * D;
        const int rt = r / a.G;                  // token in the tile
        uint32_t n = 0, na = 0;                  // tiles of S, items with keys so far
        bool ok = true;
        Item it;
        for (Walk<LOOSE> walk{bar->share, true}; ok && walk.next(a, shares, tok, nblk, nitems, &it);) {
            const bool any = it.i1 > it.i0;
            if (t >= it.ntile) {
                na += any;
                continue;
            }
            const int tt = it.t0 + t * tok;                  // the tile's first token
            const bool live = rt < tok && tt + rt < it.s.n;
            const int p = it.s.pos0 + tt + rt;
            // visible keys of this row: [wa, we], and the sinks (<= we as well); padding rows mask nothing
            const int we = live ? min(p, it.s.kv - 1) : INT32_MAX, wa = live && p >= a.window ? p - a.window + 1 : 0;
            // the row's place in O, kept out of the registers until the epilogue
            bar->row[t][r] = live ? (it.s.row0 + tt + rt) : -1;
            const KeyTiles tl = it.tl;
            const int i0 = it.i0, i1 = it.i1;
            float m = -INFINITY;
            uint64_t l2 = 0;   // row sum in two parts
            for (int i = i0; i < i1; ++i, ++n) {
                const int u0 = tl.start(i), nc = tl.width(i);
                // (the second tile's warps have passed over items of one tile)
                if (!(ok = mbar_wait_ahead(&bar->s_full[t], n & 1, abort, status, step))) break;
                tc_fence_after();
                uint32_t sr[4][32];
                const int end = min(we, (i < tl.nst ? tl.send : tl.hi) - 1);   // keys past a cut tile belong to others
                const bool full = __all_sync(FULL, u0 + 127 <= end && (u0 >= wa || u0 + 127 < a.sinks));
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tmem_ld32(sS, sr[0]);
                tmem_ld32(sS + 32, sr[1]);
                tmem_wait_ld(sr[0]);
                tmem_wait_ld(sr[1]);
                tmem_ld32(sS + 64, sr[2]);   // land while the first half is looked at
                tmem_ld32(sS + 96, sr[3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (!full) {
                        // bits of columns 32 q ..: c <= end and (c >= wa or c < sinks)
                        auto below = [&](int x) -> uint32_t {   // columns below key x
                            const int y = x - u0 - 32 * q;
                            return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u;
                        };
                        uint32_t w = ~below(wa) | below(a.sinks);
                        if (end < u0 + 128) w &= below(end + 1);
#pragma unroll
                        for (int c = 0; c < 32; ++c) sr[q][c] = (w >> c) & 1u ? sr[q][c] : 0xff800000u;
                    }
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(sr[q][c]), __uint_as_float(sr[q][c + 1]));
                    if (q == 1) {
                        tmem_wait_ld(sr[2]);
                        tmem_wait_ld(sr[3]);
                    }
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                const bool grow = top > m + RESCALE;   // from m = -inf: with the first visible key
                if (__any_sync(FULL, grow)) {
                    const float f = grow ? ex2(m - top) : 1.f;   // 0 from -inf
                    m = grow ? top : m;
                    l2 = fma2(l2, pair(f, f), 0);
                    if (i > i0) {
                        // O holds the sums so far: wait for the last product, rescale the rows that need it
                        if (!(ok = mbar_wait(&bar->o_full[t], (n - 1) & 1, abort, status))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            tmem_ld16(sO + q * 16, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            tmem_st16(sO + q * 16, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), mr2 = pair(-ref, -ref);
                uint64_t l3 = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (32 * q < nc) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float x, y;
                            unpair(fma2(pair(__uint_as_float(sr[q][c]), __uint_as_float(sr[q][c + 1])), sc2, mr2), x, y);
                            x = ex2(x);
                            y = ex2(y);
                            if (c & 2) l3 = add2(l3, pair(x, y));
                            else l2 = add2(l2, pair(x, y));
                            pk[c / 2] = pack_bf16x2(x, y);   // the tensor cores take P as bf16
                        }
                        tmem_st16(sS + q * 16, pk);   // over columns of S, which are all in registers
                    }
                    if (q & 1) {   // the product over this half of the keys can start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar->p_full[t][q >> 1]);
                    }
                }
                l2 = add2(l2, l3);
            }
            if (!ok) break;
            // epilogue: O / l, or the split's partial and its lse
            float la, lb;
            unpair(l2, la, lb);
            const float l = la + lb;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            if (any) {
                if (!(ok = mbar_wait(&bar->o_full[t], (n - 1) & 1, abort, status))) break;
                tc_fence_after();
            }
            const int token = *(volatile int *)&bar->row[t][r];
            const bool out = token >= 0;
            const long long row = (long long)token * a.H + it.j * a.G + r % a.G;
            const long long prow = (long long)it.slot * 2 * MR + t * MR + r;
            // whole tiles go out by TMA from the Q buffer, which no product reads any more
            const bool whole = it.slot < 0 && it.t0 + (t + 1) * tok <= it.s.n;
            uint8_t *stage = sQ + (na % C::QB * 2 + t) * C::TILE + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (any) {
                    tmem_ld32(sO + q * 32, o);
                    tmem_wait_ld(o);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = l > 0.f ? __float_as_uint(__uint_as_float(o[c]) * inv) : 0u;
                if (it.slot >= 0) {
                    if (out) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.opart + prow * D + q * 32);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(O + row * D + q * 32);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t h[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            h[x] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * x]), __uint_as_float(o[8 * c + 2 * x + 1]));
                        const uint4 v = make_uint4(h[0], h[1], h[2], h[3]);
                        if (any && whole && out)
                            *reinterpret_cast<uint4 *>(stage + (q >> 1) * 16384 + ((((q & 1) * 4 + c) ^ (r & 7)) << 4)) = v;
                        else if (out && !(any && whole))
                            dst[c] = v;
                    }
                }
            }
            if (any) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->out_full[na % C::QB][t]);
                ++na;
            }
            tc_fence_before();   // these reads come before the next item's product into O (through p_full)
            if (out) {
                const float lse = l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
                if (it.slot >= 0)
                    a.lpart[prow] = lse;
                else if (a.lse)
                    a.lse[row] = lse;
            }
        }
    } else {
        reg_dec<64>();
        if (warp == 8) {
            // ------------------------------------------------------------ loader
            const int psize = a.paged ? 1 << a.page_shift : 64;   // rows per box (a page, or 64)
            const uint32_t qbytes = (uint32_t)(tok * a.G) * 128u * C::NBX;
            uint32_t na = 0, nkv = 0;            // items with keys, K/V tiles so far
            uint32_t last_land = 0;              // bit s: stage s was last filled through land[s]
            uint32_t land_par = 0;               // bit s: parity of land[s]'s next phase
            uint32_t qpar = 0;                   // bit 2 x + t: parity of q_full[x][t]'s next phase (and of q_empty's last)
            uint32_t qused = 0;                  // bit 2 x + t: filled before
            bool ok = true;
            Item it;
            for (Walk<LOOSE> walk{bar->share, true}; ok && walk.next(a, shares, tok, nblk, nitems, &it);) {
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                for (int i = it.i0; i < it.i1 && ok; ++i) {
                    const int u0 = it.tl.start(i);
                    const int nbox = (it.tl.width(i) + psize - 1) / psize;
                    // this lane's box: its row in the K/V tensor; a bad page is read past the end, as zeros
                    int row = 0x7fffff00;
                    if (lane < nbox) {
                        const long long x = kv_row(a, it.b, u0 + lane * psize);
                        if (x >= 0) row = (int)x;
                    }
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        const int s = nkv % C::NST;
                        if (nkv >= (uint32_t)C::NST &&
                            !(ok = mbar_wait(&bar->kv_empty[s], (nkv / C::NST - 1) & 1, abort, status)))
                            break;
                        const bool dead = kv == 1 && it.tl.has_dead(i);
                        uint64_t *full = dead ? &bar->land[s] : &bar->kv_full[s];
                        if (dead) {
                            last_land |= 1u << s;
                            land_par ^= 1u << s;
                        } else {
                            last_land &= ~(1u << s);
                        }
                        if (lane == 0) mbar_expect_tx(full, (uint32_t)(nbox * psize) * 128u * C::NBX);
                        __syncwarp();
                        if (lane < nbox) {
                            uint8_t *dst = sKV + s * C::TILE + lane * psize * 128;
                            for (int x = 0; x < C::NBX; ++x)
                                tma_load_3d(dst + x * 16384, kv ? &tmV : &tmK, 64 * x, it.j, row, full);
                        }
                        ++nkv;
                        if (lane == 0) *step = nkv;
                        if (kv == 0 && i == it.i0) {
                            // the item's query tiles, into the buffer that the item before last has left
                            const int x = na++ % C::QB;
                            for (int t = 0; t < it.ntile && ok; ++t) {
                                const uint32_t bit = 1u << (2 * x + t);
                                if ((qused & bit) &&
                                    !(ok = mbar_wait(&bar->q_empty[x][t], (qpar & bit) ? 0 : 1, abort, status)))
                                    break;
                                qused |= bit;
                                qpar ^= bit;
                                if (lane == 0) {
                                    mbar_expect_tx(&bar->q_full[x][t], qbytes);
                                    for (int y = 0; y < C::NBX; ++y)
                                        tma_load_3d(sQ + (x * 2 + t) * C::TILE + y * 16384, &tmQ, 64 * y, it.j * a.G,
                                                    it.s.row0 + it.t0 + t * tok, &bar->q_full[x][t]);
                                }
                            }
                        }
                    }
                }
            }
            // wind down: every load issued has landed
            for (int x = 0; x < 4; ++x)
                if (qused >> x & 1) mbar_drain(&bar->q_full[x >> 1][x & 1], (qpar >> x & 1) ^ 1);
            for (int s = 0; s < C::NST; ++s) {
                const uint32_t uses = nkv > (uint32_t)s ? (nkv - 1 - s) / C::NST + 1 : 0;
                if (uses == 0) continue;
                if (last_land >> s & 1) mbar_drain(&bar->land[s], (land_par >> s & 1) ^ 1);
                else mbar_drain(&bar->kv_full[s], (uses - 1) & 1);
            }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer (the whole warp, one lane elected)
            constexpr uint32_t idesc_o = idesc_bf16_f32(MR, D, 0, 1);
            const uint32_t q0 = smem_u32(sQ), kv0 = smem_u32(sKV);
            uint32_t qpar = 0, p_par = 0, kvpar = 0, na = 0, head = 0;   // bits: parities of the next phases
            bool ok = true;
            Item it;
            for (Walk<LOOSE> walk{bar->share, true}; ok && walk.next(a, shares, tok, nblk, nitems, &it);) {
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                const int nt = it.i1 - it.i0, x = na++ % C::QB;   // key tiles, Q buffer
                // ring stages of K and V of tile i and of K of tile i + 1
                auto after = [](uint32_t st) { return st + 1 == C::NST ? 0u : st + 1; };
                auto wait_kv = [&](uint32_t st) {
                    const bool r = mbar_wait(&bar->kv_full[st], kvpar >> st & 1, abort, status);
                    kvpar ^= 1u << st;
                    return r;
                };
                auto qk = [&](int t, uint32_t st, int width, auto &&wait) -> bool {
                    const uint64_t qd = desc_kmajor_sw128(q0 + uniform(x * 2 + t) * C::TILE);
                    const uint64_t kd = desc_kmajor_sw128(kv0 + uniform(st) * C::TILE);
                    const uint32_t id = uniform(idesc_bf16_f32(MR, width, 0, 0)), dst = uniform(t) * 128;
                    if (!wait()) return false;   // the operands' addresses are ready before the operands
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {   // 16 columns a step, 64 to a box
                            constexpr uint32_t step = 32 >> 4, box = 16384 >> 4;
                            umma_bf16(tmem + dst, qd + (kk >> 2) * box + (kk & 3) * step,
                                      kd + (kk >> 2) * box + (kk & 3) * step, id, kk != 0);
                        }
                        umma_commit(&bar->s_full[t]);
                        if (t == it.ntile - 1) umma_commit(&bar->kv_empty[st]);
                    }
                    __syncwarp();
                    return true;
                };
                auto pv = [&](int t, int h, uint32_t st, int w16, bool first, auto &&wait) -> bool {
                    const uint64_t vd = desc_mnmajor_sw128(kv0 + uniform(st) * C::TILE, 16384, 1024);
                    const uint32_t ut = uniform(t), acc = uniform(first ? 0 : 1);
                    if (!wait()) return false;
                    tc_fence_after();
                    if (elect_one()) {
                        // 16 keys a step: 2048 bytes down V, 8 columns along P
                        if (w16 == BK / 16) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16_ts(tmem + 256 + ut * D, tmem + ut * 128 + (h * 4 + kk) * 8,
                                             vd + (h * 4 + kk) * (2048 >> 4), idesc_o, kk == 0 ? (h ? 1 : acc) : 1);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                if (h * 4 + kk < w16)
                                    umma_bf16_ts(tmem + 256 + ut * D, tmem + ut * 128 + (h * 4 + kk) * 8,
                                                 vd + (h * 4 + kk) * (2048 >> 4), idesc_o, kk == 0 ? (h ? 1 : acc) : 1);
                        }
                        if (h == 1) {
                            umma_commit(&bar->o_full[t]);
                            if (t == it.ntile - 1) umma_commit(&bar->kv_empty[st]);
                        }
                    }
                    __syncwarp();
                    return true;
                };
                // first scores of both tiles
                uint32_t ks = head;
                ok = wait_kv(ks);
                for (int t = 0; t < it.ntile && ok; ++t) {
                    ok = qk(t, ks, it.tl.width(it.i0), [&] {
                        return mbar_wait(&bar->q_full[x][t], qpar >> (2 * x + t) & 1, abort, status);
                    });
                    qpar ^= 1u << (2 * x + t);
                }
                for (int i = 0; i < nt && ok; ++i) {
                    const uint32_t vs = after(ks), kn = after(vs);
                    const int w16 = it.tl.width(it.i0 + i) >> 4;
                    for (int t = 0; t < it.ntile && ok; ++t) {
                        // P comes in halves
                        ok = pv(t, 0, vs, w16, i == 0, [&] {
                            return (t > 0 || wait_kv(vs)) && mbar_wait(&bar->p_full[t][0], p_par >> t & 1, abort, status);
                        });
                        ok = ok && pv(t, 1, vs, w16, i == 0, [&] {
                            return mbar_wait(&bar->p_full[t][1], p_par >> t & 1, abort, status);
                        });
                        p_par ^= 1u << t;
                        if (i + 1 < nt) ok = ok && qk(t, kn, it.tl.width(it.i0 + i + 1), [&] { return t > 0 || wait_kv(kn); });
                    }
                    ks = kn;
                    head = after(vs);
                }
            }
            if (elect_one()) umma_commit(&bar->done);
            __syncwarp();
            mbar_drain(&bar->done, 0);
        } else if (warp == 11) {
            // ------------------------------------------------------------ output tiles, and the release of their buffers
            uint32_t na = 0, par = 0;
            bool ok = true;
            Item it;
            for (Walk<LOOSE> walk{bar->share, true}; ok && walk.next(a, shares, tok, nblk, nitems, &it);) {
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                const int x = na++ % C::QB;
                for (int t = 0; t < it.ntile; ++t) {
                    const int bit = 2 * x + t;
                    if (!(ok = mbar_wait_ahead(&bar->out_full[x][t], par >> bit & 1, abort, status, step))) break;
                    par ^= 1u << bit;
                    if (lane == 0) {
                        if (it.slot < 0 && it.t0 + (t + 1) * tok <= it.s.n) {
                            for (int y = 0; y < C::NBX; ++y)
                                tma_store_3d(&tmO, sQ + (x * 2 + t) * C::TILE + y * 16384, 64 * y, it.j * a.G,
                                             it.s.row0 + it.t0 + t * tok);
                            bulk_commit();
                            bulk_wait_read();
                        }
                        mbar_arrive(&bar->q_empty[x][t]);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 10) {
            // ------------------------------------------------------------ zeroes dead V rows at the range's edges
            uint32_t nkv = 0, land_par = 0;
            bool ok = true;
            Item it;
            for (Walk<LOOSE> walk{bar->share, true}; ok && walk.next(a, shares, tok, nblk, nitems, &it);) {
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                for (int i = it.i0; i < it.i1 && ok; ++i, nkv += 2) {
                    if (!it.tl.has_dead(i)) continue;
                    const int u0 = it.tl.start(i), width = it.tl.width(i);
                    const int s = (nkv + 1) % C::NST;
                    if (!(ok = mbar_wait_ahead(&bar->land[s], land_par >> s & 1, abort, status, step))) break;
                    land_par ^= 1u << s;
                    uint8_t *v = sKV + s * C::TILE;
                    // 8 lanes per 128-byte row
                    for (int r = lane >> 3; r < width; r += 4)
                        if (!it.tl.live(u0 + r))
                            for (int x = 0; x < C::NBX; ++x)
                                reinterpret_cast<uint4 *>(v + x * 16384 + r * 128)[lane & 7] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->kv_full[s]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

bool tc_supported(const LocArgs &a, int dtype) {
    if (dtype != HSA_BF16 || a.max_kv == 0 || a.max_q == 0) return false;
    // items are numbered in 32 bits, with room for a step past the last (a loose max_q of very many sequences)
    const int tok = MR / a.G, nblk = (a.max_q + 2 * tok - 1) / (2 * tok);
    return (long long)a.B * nblk * a.Hkv <= INT_MAX - 148;
}

cudaError_t launch_tc(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st) {
    const int tok = MR / a.G, nblk = (a.max_q + 2 * tok - 1) / (2 * tok);
    const long long items = (long long)a.B * nblk * a.Hkv;
    long long *starts = a.tc_starts;
    CUtensorMap mq, mk, mv, mo;
    const uint64_t d = a.d;
    const uint64_t qd[3] = {d, (uint64_t)a.H, (uint64_t)a.rows}, qs[2] = {d * 2, (uint64_t)a.H * d * 2};
    const uint32_t qb[3] = {64, (uint32_t)a.G, (uint32_t)tok};
    const uint64_t kvrows = a.paged ? (uint64_t)a.npages << a.page_shift : (uint64_t)a.B * a.Tcap;
    const uint64_t kd[3] = {d, (uint64_t)a.Hkv, kvrows}, ks[2] = {d * 2, (uint64_t)a.Hkv * d * 2};
    const uint32_t kb[3] = {64, 1, a.paged ? 1u << a.page_shift : 64u};
    cudaError_t e = make_tmap_3d(&mq, Q, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mo, O, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mk, K, kd, ks, kb);
    if (e == cudaSuccess) e = make_tmap_3d(&mv, V, kd, ks, kb);
    if (e != cudaSuccess) return e;
    // shares: every SM may get one, however few the items
    const int grid = items < 148 && !starts ? (int)items : 148;
    auto go = [&](auto kern, int tile, int tiles) {
        const size_t smem = 1024 + (size_t)tiles * tile + sizeof(Bars);
        cudaError_t x = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (x != cudaSuccess) return x;
        kern<<<grid, NT, smem, st>>>(mq, mk, mv, mo, (__nv_bfloat16 *)O, a, tok, nblk, (int)items, starts);
        return cudaGetLastError();
    };
    // Far more items than the rows can fill: the walk that steps over the empty ones.  It makes an item's start longer
    // (300 items of 6 key tiles: 35.2 -> 36.9 us), so only where they are most.  20000 single tokens: max_q 20399
    // (318 blocks each) 40.6 -> 13.9 ms, max_q 300 (5 blocks) 1.45 -> 1.73 ms.
    const bool loose = a.paged && (long long)a.B * nblk > 16 * (a.rows / (2ll * tok) + a.B);
    auto by_walk = [&](auto kern, auto kern_loose, int tile, int tiles) {
        return loose ? go(kern_loose, tile, tiles) : go(kern, tile, tiles);
    };
    e = a.d == 64 ? by_walk(window_fwd_kernel<64, false>, window_fwd_kernel<64, true>, Cfg<64>::TILE, 2 * Cfg<64>::QB + Cfg<64>::NST)
                  : by_walk(window_fwd_kernel<128, false>, window_fwd_kernel<128, true>, Cfg<128>::TILE,
                            2 * Cfg<128>::QB + Cfg<128>::NST);
    if (e != cudaSuccess || !starts) return e;
    const dim3 jg((unsigned)items, 2 * JOIN_ROWS);
    if (a.d == 64) window_join_kernel<64><<<jg, 256, 0, st>>>(a, (__nv_bfloat16 *)O, tok, nblk, starts);
    else window_join_kernel<128><<<jg, 256, 0, st>>>(a, (__nv_bfloat16 *)O, tok, nblk, starts);
    return cudaGetLastError();
}

static int share_items(const LocArgs &a) { return (a.paged ? 16 : 2) * 148; }   // fewer items than these are shared
constexpr long long SHARE_BLOCKS = 1024;

static void share_bytes(const LocArgs &a, long long blocks, long long items, long long most_keys, TcPlan *p) {
    p->starts = (size_t)(blocks + 2) * sizeof(long long);
    // two slots (first and last item) for each CTA that can get a share
    long long ctas = items * (most_keys / BK + 3) / SHARE_LEAST + 1;
    if (ctas > 148) ctas = 148;
    p->opart = (size_t)(2 * ctas) * 2 * MR * a.d * sizeof(float);
    p->lpart = (size_t)(2 * ctas) * 2 * MR * sizeof(float);
}

TcPlan tc_plan(const LocArgs &a, long long most_keys) {
    const int tok = MR / a.G, nblk = (a.max_q + 2 * tok - 1) / (2 * tok);
    const long long blocks = (long long)a.B * nblk, items = blocks * a.Hkv;
    TcPlan p{};
    // Shares where whole items would leave SMs idle: fewer than two items per SM, or 16 where the lengths are not
    // known here.  More items balance by themselves and run faster whole, since neighbouring CTAs then read the same
    // keys (2048 items of 33 tiles: 890 us whole, 1148 us shared); items of fewer than 16 key tiles are not worth
    // their cuts and the second launch (300 of 6 tiles: 35 us whole, 53 us and the join shared; but 136 of 113 to 256: 833 us and 492 us).
    // The scan of the blocks' lengths, one warp per CTA, is kept to 1024 blocks.
    p.shares = items > 0 && items < share_items(a) && blocks <= SHARE_BLOCKS && most_keys >= 16 * BK;
    if (p.shares) share_bytes(a, blocks, items, most_keys, &p);
    return p;
}

TcPlan tc_plan_most(const LocArgs &a, long long most_keys) {
    const int tok = MR / a.G, nblk = (a.max_q + 2 * tok - 1) / (2 * tok);
    const long long blocks = (long long)a.B * nblk, items = blocks * a.Hkv;
    TcPlan p{};
    p.shares = items > 0 && a.Hkv < share_items(a) && most_keys >= 16 * BK;
    if (p.shares)
        share_bytes(a, blocks < SHARE_BLOCKS ? blocks : SHARE_BLOCKS, items < share_items(a) ? items : share_items(a), most_keys, &p);
    return p;
}

}  // namespace local
}  // namespace hsa
