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
    static constexpr int NST = D == 128 ? 4 : 8;       // K/V ring stages
};

struct __align__(8) Bars {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], land[8];
    uint64_t s_full[2], p_full[2], o_full[2], done;
    uint32_t tmem_base;
    int abort;
};

struct Item {
    int b, j, split, t0, ntile;   // ntile: row tiles with tokens (0: nothing to do)
    int i0, i1;                   // key tiles of this split
    Seq s;
    Tiles tl;
};

__device__ __forceinline__ Item item_of(const LocArgs &a, int idx, int tok, int nblk) {
    Item it;
    it.j = idx % a.Hkv;
    idx /= a.Hkv;
    it.split = idx % a.nsplit;
    idx /= a.nsplit;
    const int blk = nblk - 1 - idx % nblk;   // without a window, later blocks see more keys: longest first
    it.b = idx / nblk;
    it.s = seq_of(a, it.b);
    it.t0 = blk * 2 * tok;
    const int left = it.s.n - it.t0;
    it.ntile = left <= 0 ? 0 : left <= tok ? 1 : 2;
    const int pa = it.s.pos0 + it.t0, pb = it.s.pos0 + min(it.s.n, it.t0 + 2 * tok) - 1;
    it.tl = tiles_of<BK>(pa, pb, it.s.kv, a.window, a.sinks);
    split_range(it.tl.nt, a.nsplit, it.split, &it.i0, &it.i1);
    return it;
}

// Whether tile [u0, u0 + 128) holds keys that no query of the item sees, and which
// the loader still brings in.
__device__ __forceinline__ bool has_dead(const Tiles &t, int u0) {
    return u0 + BK > t.hi || (u0 < t.lo && !(u0 + BK <= t.ns));
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, __nv_bfloat16 *__restrict__ O,
                      const __grid_constant__ LocArgs a, int tok, int nblk, int nitems) {
    typedef Cfg<D> C;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base;                       // 2 tiles
    uint8_t *sKV = base + 2 * C::TILE;        // NST tiles
    Bars *bar = reinterpret_cast<Bars *>(sKV + C::NST * C::TILE);
    volatile int *abort = &bar->abort;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // rows that no box covers (G does not divide 128) stay zero
    for (int i = threadIdx.x; i < 2 * C::TILE / 16; i += NT) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar->q_full[t], 1);
            mbar_init(&bar->q_empty[t], 1);
            mbar_init(&bar->s_full[t], 1);
            mbar_init(&bar->p_full[t], 4);
            mbar_init(&bar->o_full[t], 1);
        }
        for (int s = 0; s < C::NST; ++s) {
            mbar_init(&bar->kv_full[s], 1);
            mbar_init(&bar->kv_empty[s], 1);
            mbar_init(&bar->land[s], 1);
        }
        mbar_init(&bar->done, 1);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bar->tmem_base, 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;   // S/P tiles at 0 and 128, O tiles at 256 and 256 + D

    if (warp < 8) {
        reg_inc<216>();
        // ---------------------------------------------------------------- softmax: thread = row of tile t
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sS = tmem + lane_off + t * 128, sO = tmem + lane_off + 256 + t * D;
        const int rt = r / a.G, rg = r % a.G;   // token in the tile, head in the group
        uint32_t n = 0;                          // tiles of S seen so far
        bool ok = true;
        for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
            const Item it = item_of(a, idx, tok, nblk);
            if (t >= it.ntile) continue;
            const int tt = it.t0 + t * tok;                  // the tile's first token
            const int te = min(it.s.n, tt + tok);
            const int pa = it.s.pos0 + tt, pb = it.s.pos0 + te - 1;
            const bool live = rt < tok && tt + rt < te;
            const int p = live ? pa + rt : -1;
            // visible keys of this row: [wa, we], and those below sk (<= we as well)
            const int we = min(p, it.s.kv - 1), wa = p >= a.window ? p - a.window + 1 : 0, sk = a.sinks;
            float m = -INFINITY;
            uint64_t l2 = 0;   // row sum, two halves
            for (int i = it.i0; i < it.i1; ++i, ++n) {
                const int u0 = it.tl.tile(i) * BK;
                if (!(ok = mbar_wait(&bar->s_full[t], n & 1, abort, status))) break;
                tc_fence_after();
                uint32_t sr[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(sS + q * 32, sr[q]);
                tmem_wait_ld();
                if (!tile_full(pa, pb, u0, BK, it.s.kv, a.window, a.sinks)) {
                    const int e = we - u0, f = wa - u0, k = sk - u0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // bits of columns 32 q ..: c <= e and (c >= f or c < k)
                        auto below = [&](int x) -> uint32_t {   // columns c < x
                            const int y = x - 32 * q;
                            return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u;
                        };
                        const uint32_t w = below(e + 1) & (~below(f) | below(k));
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            sr[q][c] = (w >> c) & 1u ? sr[q][c] : 0xff800000u;
                    }
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = __uint_as_float(sr[q][0]);
#pragma unroll
                    for (int c = 1; c < 32; ++c) mx[q] = fmaxf(mx[q], __uint_as_float(sr[q][c]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                const bool grow = top > m + RESCALE || (m == -INFINITY && top > m);
                float f = 1.f;
                if (grow) {
                    f = ex2(m - top);   // 0 from -inf
                    m = top;
                    l2 = fma2(l2, pair(f, f), 0);
                }
                if (i > it.i0 && __any_sync(FULL, grow)) {
                    // O holds the sums so far: wait for the last product, rescale the rows that need it
                    if (!(ok = mbar_wait(&bar->o_full[t], (n - 1) & 1, abort, status))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tmem_ld16(sO + q * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                        tmem_st16(sO + q * 16, o);
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), mr2 = pair(-ref, -ref);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float x, y;
                        unpair(fma2(pair(__uint_as_float(sr[q][c]), __uint_as_float(sr[q][c + 1])), sc2, mr2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        l2 = add2(l2, pair(x, y));
                        pk[c / 2] = pack_bf16x2(x, y);   // the tensor cores take P as bf16
                    }
                    tmem_st16(sS + q * 16, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full[t]);
            }
            if (!ok) break;
            // epilogue: O / l, or the split's partial and its lse
            float la, lb;
            unpair(l2, la, lb);
            const float l = la + lb;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const bool any = it.i1 > it.i0;
            if (any) {
                if (!(ok = mbar_wait(&bar->o_full[t], (n - 1) & 1, abort, status))) break;
                tc_fence_after();
            }
            const long long row = live ? (long long)(it.s.row0 + tt + rt) * a.H + it.j * a.G + rg : 0;
            const long long prow = (long long)it.split * a.rows * a.H + row;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (any) {
                    tmem_ld32(sO + q * 32, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = l > 0.f ? __float_as_uint(__uint_as_float(o[c]) * inv) : 0u;
                if (live) {
                    if (a.nsplit > 1) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.opart + prow * D + q * 32);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(O + row * D + q * 32);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t h[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                h[x] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * x]), __uint_as_float(o[8 * c + 2 * x + 1]));
                            dst[c] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                }
            }
            tc_fence_before();   // these reads come before the next item's product into O (through p_full)
            if (live) {
                const float lse = l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
                if (a.nsplit > 1)
                    a.lpart[prow] = lse;
                else if (a.lse)
                    a.lse[row] = lse;
            }
        }
    } else {
        reg_dec<64>();
        if (warp == 8) {
            // ------------------------------------------------------------ loader
            const int psize = a.paged ? 1 << a.page_shift : BK;
            const int ppt = BK / psize;          // boxes per tile (pages, or one)
            const uint32_t qbytes = (uint32_t)(tok * a.G) * 128u * C::NBX;
            uint32_t nq0 = 0, nq1 = 0, nkv = 0;
            uint32_t last_land = 0;              // bit s: stage s was last filled through land[s]
            uint32_t land_par = 0;               // bit s: parity of land[s]'s next phase
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const Item it = item_of(a, idx, tok, nblk);
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                for (int i = it.i0; i < it.i1 && ok; ++i) {
                    const int u0 = it.tl.tile(i) * BK;
                    // this lane's box: its row in the K/V tensor; past the end (zeros) where nothing is visible
                    int row = 0x7fffff00;
                    if (lane < ppt) {
                        const int ua = u0 + lane * psize, ub = ua + psize;   // keys [ua, ub)
                        const bool use = ua < it.tl.hi && (ub > it.tl.lo || ua < it.tl.ns);
                        if (!a.paged)
                            row = it.b * a.Tcap + ua;
                        else if (use) {
                            const long long x = kv_row(a, it.b, ua);
                            if (x >= 0) row = (int)x;
                        }
                    }
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        if (kv == 0 && i == it.i0) {
                            // the item's query tiles, before its first keys
                            for (int t = 0; t < it.ntile && ok; ++t) {
                                const uint32_t n = t ? nq1++ : nq0++;
                                if (n > 0 && !(ok = mbar_wait(&bar->q_empty[t], (n - 1) & 1, abort, status))) {
                                    --(t ? nq1 : nq0);
                                    break;
                                }
                                if (lane == 0) {
                                    mbar_expect_tx(&bar->q_full[t], qbytes);
                                    for (int x = 0; x < C::NBX; ++x)
                                        tma_load_3d(sQ + t * C::TILE + x * 16384, &tmQ, 64 * x, it.j * a.G,
                                                    it.s.row0 + it.t0 + t * tok, &bar->q_full[t]);
                                }
                            }
                            if (!ok) break;
                        }
                        const int s = nkv % C::NST;
                        if (nkv >= (uint32_t)C::NST &&
                            !(ok = mbar_wait(&bar->kv_empty[s], (nkv / C::NST - 1) & 1, abort, status)))
                            break;
                        const bool dead = kv == 1 && has_dead(it.tl, u0);
                        uint64_t *full = dead ? &bar->land[s] : &bar->kv_full[s];
                        if (dead) {
                            last_land |= 1u << s;
                            land_par ^= 1u << s;
                        } else {
                            last_land &= ~(1u << s);
                        }
                        if (lane == 0) mbar_expect_tx(full, C::TILE);
                        __syncwarp();
                        if (lane < ppt) {
                            uint8_t *dst = sKV + s * C::TILE + lane * psize * 128;
                            for (int x = 0; x < C::NBX; ++x)
                                tma_load_3d(dst + x * 16384, kv ? &tmV : &tmK, 64 * x, it.j, row, full);
                        }
                        ++nkv;
                    }
                }
            }
            // wind down: every load issued has landed
            if (nq0 > 0) mbar_drain(&bar->q_full[0], (nq0 - 1) & 1);
            if (nq1 > 0) mbar_drain(&bar->q_full[1], (nq1 - 1) & 1);
            for (int s = 0; s < C::NST; ++s) {
                const uint32_t uses = nkv > (uint32_t)s ? (nkv - 1 - s) / C::NST + 1 : 0;
                if (uses == 0) continue;
                if (last_land >> s & 1) mbar_drain(&bar->land[s], (land_par >> s & 1) ^ 1);
                else mbar_drain(&bar->kv_full[s], (uses - 1) & 1);
            }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                const uint32_t idesc_s = idesc_bf16_f32(MR, BK, 0, 0), idesc_o = idesc_bf16_f32(MR, D, 0, 1);
                uint32_t nq = 0, np = 0, nkv = 0;   // bit t: parity of tile t's next phase
                bool ok = true;
                for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                    const Item it = item_of(a, idx, tok, nblk);
                    if (it.ntile == 0 || it.i0 >= it.i1) continue;
                    const int nt = it.i1 - it.i0;
                    const uint32_t kv0 = nkv;   // tile i: K is fill kv0 + 2 i, V the one after
                    nkv += 2 * nt;
                    auto stage = [&](uint32_t f) { return smem_u32(sKV + (f % C::NST) * C::TILE); };
                    auto wait_kv = [&](uint32_t f) {
                        return mbar_wait(&bar->kv_full[f % C::NST], (f / C::NST) & 1, abort, status);
                    };
                    auto qk = [&](int t, int i) {
                        const uint32_t qa = smem_u32(sQ + t * C::TILE), kb = stage(kv0 + 2 * i);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
                            umma_bf16(tmem + t * 128, desc_kmajor_sw128(qa + o), desc_kmajor_sw128(kb + o), idesc_s,
                                      kk != 0);
                        }
                        umma_commit(&bar->s_full[t]);
                        if (i == nt - 1) umma_commit(&bar->q_empty[t]);
                        if (t == it.ntile - 1) umma_commit(&bar->kv_empty[(kv0 + 2 * i) % C::NST]);
                    };
                    // first scores of both tiles
                    for (int t = 0; t < it.ntile && ok; ++t) {
                        ok = mbar_wait(&bar->q_full[t], nq >> t & 1, abort, status);
                        nq ^= 1u << t;
                        if (ok && t == 0) ok = wait_kv(kv0);
                        if (!ok) break;
                        tc_fence_after();
                        qk(t, 0);
                    }
                    for (int i = 0; i < nt && ok; ++i) {
                        for (int t = 0; t < it.ntile; ++t) {
                            if (!(ok = mbar_wait(&bar->p_full[t], np >> t & 1, abort, status))) break;
                            np ^= 1u << t;
                            if (t == 0 && !(ok = wait_kv(kv0 + 2 * i + 1))) break;
                            tc_fence_after();
                            const uint32_t vb = stage(kv0 + 2 * i + 1);
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                umma_bf16_ts(tmem + 256 + t * D, tmem + t * 128 + kk * 8,
                                             desc_mnmajor_sw128(vb + kk * 16 * 128, 16384, 1024), idesc_o,
                                             i != 0 || kk != 0);
                            umma_commit(&bar->o_full[t]);
                            if (t == it.ntile - 1) umma_commit(&bar->kv_empty[(kv0 + 2 * i + 1) % C::NST]);
                            if (i + 1 < nt) {
                                if (t == 0 && !(ok = wait_kv(kv0 + 2 * i + 2))) break;
                                tc_fence_after();
                                qk(t, i + 1);
                            }
                        }
                    }
                }
                umma_commit(&bar->done);
                mbar_drain(&bar->done, 0);
            }
        } else if (warp == 10) {
            // ------------------------------------------------------------ zeroes dead V rows at the range's edges
            uint32_t nkv = 0, land_par = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const Item it = item_of(a, idx, tok, nblk);
                if (it.ntile == 0 || it.i0 >= it.i1) continue;
                for (int i = it.i0; i < it.i1 && ok; ++i, nkv += 2) {
                    const int u0 = it.tl.tile(i) * BK;
                    if (!has_dead(it.tl, u0)) continue;
                    const int s = (nkv + 1) % C::NST;
                    if (!(ok = mbar_wait(&bar->land[s], land_par >> s & 1, abort, status))) break;
                    land_par ^= 1u << s;
                    uint8_t *v = sKV + s * C::TILE;
                    // 8 lanes per 128-byte row
                    for (int r = lane >> 3; r < BK; r += 4)
                        if (!key_live(it.tl, u0 + r))
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
    return dtype == HSA_BF16 && a.max_kv > 0 && a.max_q > 0;
}

cudaError_t launch_tc(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st) {
    const int tok = MR / a.G, nblk = (a.max_q + 2 * tok - 1) / (2 * tok);
    const long long items = (long long)a.B * nblk * a.Hkv * a.nsplit;
    CUtensorMap mq, mk, mv;
    const uint64_t d = a.d;
    const uint64_t qd[3] = {d, (uint64_t)a.H, (uint64_t)a.rows}, qs[2] = {d * 2, (uint64_t)a.H * d * 2};
    const uint32_t qb[3] = {64, (uint32_t)a.G, (uint32_t)tok};
    const uint64_t kvrows = a.paged ? (uint64_t)a.npages << a.page_shift : (uint64_t)a.B * a.Tcap;
    const uint64_t kd[3] = {d, (uint64_t)a.Hkv, kvrows}, ks[2] = {d * 2, (uint64_t)a.Hkv * d * 2};
    const uint32_t kb[3] = {64, 1, a.paged ? 1u << a.page_shift : (uint32_t)BK};
    cudaError_t e = make_tmap_3d(&mq, Q, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mk, K, kd, ks, kb);
    if (e == cudaSuccess) e = make_tmap_3d(&mv, V, kd, ks, kb);
    if (e != cudaSuccess) return e;
    const int grid = items < 148 ? (int)items : 148;
    auto go = [&](auto kern, int tile, int nst) {
        const size_t smem = 1024 + (size_t)(2 + nst) * tile + sizeof(Bars);
        cudaError_t x = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (x != cudaSuccess) return x;
        kern<<<grid, NT, smem, st>>>(mq, mk, mv, (__nv_bfloat16 *)O, a, tok, nblk, (int)items);
        return cudaGetLastError();
    };
    return a.d == 64 ? go(window_fwd_kernel<64>, Cfg<64>::TILE, Cfg<64>::NST)
                     : go(window_fwd_kernel<128>, Cfg<128>::TILE, Cfg<128>::NST);
}

}  // namespace local
}  // namespace hsa
