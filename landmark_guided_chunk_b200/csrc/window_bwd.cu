// window_bwd.cu -- backward of the sliding-window attention on tcgen05 (bf16).
//
// With P = exp2(scale_log2 S - lse_log2), S = Q K^T, dP = dO V^T, D = rowsum(dO o O):
//   dS = P o (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// Two kernels, each writing its outputs once, so that no sum depends on the order of
// atomics: window_dq_kernel runs over the key tiles of a row tile (three products per
// 128 x 128 tile), window_dkv_kernel over the row tiles of a key tile, transposed
// (S^T = K Q^T: four products).  Seven products against the five of one fused kernel,
// whose S, dP, dK, dV already fill the 512 TMEM columns, so that dQ would have to leave
// the chip as fp32 atomics for every tile (64 KB against 5 x 4 MFLOP).
//
// A row is (token, head of the group), so a key tile's dK and dV add over the G heads
// by themselves.  Rows and keys that nothing sees are masked to P = dS = 0.
//
// Roles in both: two elementwise warpgroups, each with one half of the tile's columns
// (lse is known: no row maximum to share), a loader warp (TMA), an MMA warp (converged,
// one lane elected), a helper warp.
#include <stddef.h>

#include "local.cuh"
#include "local_sm100.cuh"

namespace hsa {
namespace local {

namespace {

using namespace sm100;

constexpr int BK = 128;   // keys per tile
constexpr int MR = 128;   // rows per tile
constexpr int NT = 384;

template <int D> struct Cfg {
    static constexpr int NBX = D / 64, TILE = 128 * D * 2;
};

// ---------------------------------------------------------------------------- shared pieces

// (d_tmem) = A B^T, both K-major tiles of 128 x D in shared memory; N = width of B
template <int D> __device__ __forceinline__ void mma_nt(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint64_t ad = desc_kmajor_sw128(a), bd = desc_kmajor_sw128(b);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        constexpr uint32_t step = 32 >> 4, box = 16384 >> 4;
        umma_bf16(d_tmem, ad + (kk >> 2) * box + (kk & 3) * step, bd + (kk >> 2) * box + (kk & 3) * step, idesc, kk != 0);
    }
}
// (d_tmem) (+)= A B: A bf16 in TMEM (64 columns a half: 32 for data), B a tile of 128 x D in shared memory, rows
// contracted; the first `steps` of 8 steps of 16
template <int D>
__device__ __forceinline__ void mma_tn(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t accumulate, int steps) {
    constexpr uint32_t idesc = idesc_bf16_f32(MR, D, 0, 1);
    const uint64_t bd = desc_mnmajor_sw128(b, 16384, 1024);
    if (steps == 8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(d_tmem, a_tmem + (kk >> 2) * 64 + (kk & 3) * 8, bd + kk * (2048 >> 4), idesc,
                         kk == 0 ? accumulate : 1);
    } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            if (kk < steps)
                umma_bf16_ts(d_tmem, a_tmem + (kk >> 2) * 64 + (kk & 3) * 8, bd + kk * (2048 >> 4), idesc,
                             kk == 0 ? accumulate : 1);
    }
}

// 32 columns of an fp32 accumulator, times f, to 32 consecutive elements: bf16 or fp32
__device__ __forceinline__ void put32(uint32_t taddr, float f, __nv_bfloat16 *h, float *w, bool live) {
    uint32_t o[32];
    tmem_ld32(taddr, o);
    tmem_wait_ld(o);
    if (!live) return;
    if (w) {
#pragma unroll
        for (int c = 0; c < 32; c += 4)
            *reinterpret_cast<float4 *>(w + c) =
                make_float4(__uint_as_float(o[c]) * f, __uint_as_float(o[c + 1]) * f, __uint_as_float(o[c + 2]) * f,
                            __uint_as_float(o[c + 3]) * f);
    } else {
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
            uint32_t x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[y] = pack_bf16x2(__uint_as_float(o[c + 2 * y]) * f, __uint_as_float(o[c + 2 * y + 1]) * f);
            *reinterpret_cast<uint4 *>(h + c) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
}

// bits of columns 32 q .. 32 q + 31 in [c0, c1)
__device__ __forceinline__ uint32_t bits(int c0, int c1, int q) {
    auto below = [](int y) -> uint32_t { return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u; };
    return below(c1 - 32 * q) & ~below(c0 - 32 * q);
}

// The key tiles of a row tile: the sinks' from 0, then the window's from its first key;
// the last of each is cut to a multiple of 16 keys.
struct KeyTiles {
    int lo, hi, ns, nst, nt;
    __device__ __forceinline__ int start(int i) const { return i < nst ? i * BK : lo + (i - nst) * BK; }
    __device__ __forceinline__ int end(int i) const { return min(start(i) + BK, i < nst ? ns : hi); }
    __device__ __forceinline__ int width(int i) const { return (end(i) - start(i) + 15) & ~15; }
};

__device__ __forceinline__ KeyTiles key_tiles(int pa, int pb, int kv, int window, int sinks) {
    KeyTiles t;
    t.hi = max(0, min(pb + 1, kv));
    t.lo = min(pa >= window ? pa - window + 1 : 0, t.hi);   // window may be INT32_MAX
    t.ns = min(sinks, t.lo);
    t.nst = (t.ns + BK - 1) / BK;
    t.nt = t.nst + (t.hi - t.lo + BK - 1) / BK;
    return t;
}

// ---------------------------------------------------------------------------- dQ

constexpr int KST = 3, VST = 2;   // ring stages: K stays until dS K, V only until dO V^T

struct __align__(8) DqBars {
    uint64_t q_full, q_empty, k_full[KST], k_empty[KST], land[KST], v_full[VST], v_empty[VST];
    uint64_t s_full[2], dp_full, dp_empty, ds_full[2], dq_full, done;
    uint32_t tmem_base;
    int abort;
};

struct DqItem {
    int b, j, t0, te;
    Seq s;
    KeyTiles tl;
};

__device__ __forceinline__ DqItem dq_item(const LocArgs &a, int idx, int tok, int nblk) {
    DqItem it;
    it.j = idx % a.Hkv;
    idx /= a.Hkv;
    const int blk = nblk - 1 - idx % nblk;   // without a window, later rows see more keys: longest first
    it.b = idx / nblk;
    it.s = seq_of(a, it.b);
    it.t0 = blk * tok;
    it.te = min(it.s.n, it.t0 + tok);
    it.tl = key_tiles(it.s.pos0 + it.t0, it.s.pos0 + it.te - 1, it.s.kv, a.window, a.sinks);
    return it;
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     __nv_bfloat16 *__restrict__ dQ, const __grid_constant__ BwdArgs w, int tok, int nblk, int nitems) {
    typedef Cfg<D> C;
    const LocArgs &a = w.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sG = sQ + C::TILE, *sK = sG + C::TILE, *sV = sK + KST * C::TILE;
    DqBars *bar = reinterpret_cast<DqBars *>(sV + VST * C::TILE);
    volatile int *abort = &bar->abort;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows that no box covers (G does not divide 128) stay zero
    for (int i = threadIdx.x; i < 2 * C::TILE / 16; i += NT) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, 1);
        mbar_init(&bar->q_empty, 1);
        for (int s = 0; s < KST; ++s) {
            mbar_init(&bar->k_full[s], 1);
            mbar_init(&bar->k_empty[s], 1);
            mbar_init(&bar->land[s], 1);
        }
        for (int s = 0; s < VST; ++s) {
            mbar_init(&bar->v_full[s], 1);
            mbar_init(&bar->v_empty[s], 1);
            mbar_init(&bar->s_full[s], 1);
            mbar_init(&bar->ds_full[s], 8);
        }
        mbar_init(&bar->dp_full, 1);
        mbar_init(&bar->dp_empty, 8);
        mbar_init(&bar->dq_full, 1);
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
    // all 512 TMEM columns are this CTA's: S (then dS) at 0 and 128, dP at 256, dQ at 384
    if (warp < 8) {
        reg_inc<208>();
        // ---------------------------------------------------------------- elementwise: thread = half a row
        const int hf = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16, cols = lane_off + 64 * hf;
        uint32_t n = 0, ni = 0;
        bool ok = true;
        for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
            const DqItem it = dq_item(a, idx, tok, nblk);
            const int t = it.t0 + r / a.G;
            const bool live = r < tok * a.G && t < it.te;
            const int p = it.s.pos0 + t;
            const int we = live ? min(p, it.s.kv - 1) : -1, wa = live && p >= a.window ? p - a.window + 1 : 0;
            const long long row = live ? (long long)(it.s.row0 + t) * a.H + it.j * a.G + r % a.G : 0;
            const float lse2 = live ? a.lse[row] * 1.4426950408889634f : 0.f, dd = live ? w.D[row] : 0.f;
            for (int i = 0; i < it.tl.nt; ++i, ++n) {
                const uint32_t sS = cols + (n & 1) * 128;
                const int u0 = it.tl.start(i) + 64 * hf, nc = it.tl.end(i) - u0;   // columns of this half
                if (!(ok = mbar_wait(&bar->s_full[n & 1], (n >> 1) & 1, abort, status))) break;
                tc_fence_after();
                uint32_t x[2][32];
                // visible: c <= we - u0, c < nc, and (c >= wa - u0 or c < sinks - u0)
                const int c1 = min(we + 1 - u0, nc);
                const bool full = __all_sync(FULL, c1 >= 64 && (wa <= u0 || u0 + 64 <= a.sinks));
                if (nc > 0) {
                    tmem_ld32(sS, x[0]);
                    tmem_ld32(sS + 32, x[1]);
                    tmem_wait_ld(x[0]);
                    tmem_wait_ld(x[1]);
                    const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), ml2 = pair(-lse2, -lse2);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t m = full ? ~0u : bits(0, c1, q) & (bits(wa - u0, 64, q) | bits(0, a.sinks - u0, q));
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float y, z;
                            unpair(fma2(pair(__uint_as_float(x[q][c]), __uint_as_float(x[q][c + 1])), sc2, ml2), y, z);
                            x[q][c] = __float_as_uint(ex2(y));
                            x[q][c + 1] = __float_as_uint(ex2(z));
                        }
                        if (!full) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[q][c] = (m >> c) & 1u ? x[q][c] : 0u;
                        }
                    }
                }
                if (!(ok = mbar_wait(&bar->dp_full, n & 1, abort, status))) break;
                tc_fence_after();
                if (nc > 0) {
                    uint32_t g[2][32];
                    tmem_ld32(cols + 256, g[0]);
                    tmem_ld32(cols + 288, g[1]);
                    tmem_wait_ld(g[0]);
                    tmem_wait_ld(g[1]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->dp_empty);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            // P = 0 where masked: whatever dP holds there (NaN included) must not come through
                            float y = __uint_as_float(x[q][c]) * (__uint_as_float(g[q][c]) - dd);
                            float z = __uint_as_float(x[q][c + 1]) * (__uint_as_float(g[q][c + 1]) - dd);
                            if (!full) {
                                y = x[q][c] ? y : 0.f;
                                z = x[q][c + 1] ? z : 0.f;
                            }
                            pk[c / 2] = pack_bf16x2(y, z);   // the tensor cores take dS as bf16
                        }
                        tmem_st16(sS + q * 16, pk);
                    }
                    tmem_wait_st();
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->dp_empty);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->ds_full[n & 1]);
            }
            if (!ok) break;
            const bool any = it.tl.nt > 0;
            if (any) {
                if (!(ok = mbar_wait(&bar->dq_full, ni++ & 1, abort, status))) break;
                tc_fence_after();
            }
            __nv_bfloat16 *dst = dQ + row * D + hf * (D / 2);
            if (any) {
                for (int q = 0; q < D / 64; ++q) put32(lane_off + 384 + hf * (D / 2) + q * 32, a.scale, dst + q * 32, nullptr, live);
                tc_fence_before();
            } else if (live) {
                for (int c = 0; c < D / 2; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        reg_dec<80>();
        if (warp == 8) {
            // ------------------------------------------------------------ loader
            uint32_t nq = 0, nk = 0, land_par = 0, last_land = 0;
            const uint32_t qbytes = (uint32_t)(tok * a.G) * 128u * C::NBX;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                for (int i = 0; i < it.tl.nt && ok; ++i, ++nk) {
                    const int u0 = it.tl.start(i), nbox = (it.tl.width(i) + 63) / 64;
                    const int row = it.b * a.Tcap + u0;
                    const uint32_t bytes = (uint32_t)nbox * 64u * 128u * C::NBX;
                    const uint32_t ks = nk % KST, vs = nk % VST;
                    if (nk >= KST && !(ok = mbar_wait(&bar->k_empty[ks], (nk / KST - 1) & 1, abort, status))) break;
                    // K rows past the tile's end would meet dS = 0 as B rows: the helper zeroes them first
                    const bool dead = it.tl.end(i) < u0 + it.tl.width(i);
                    uint64_t *full = dead ? &bar->land[ks] : &bar->k_full[ks];
                    if (dead) {
                        land_par ^= 1u << ks;
                        last_land |= 1u << ks;
                    } else {
                        last_land &= ~(1u << ks);
                    }
                    if (lane == 0) {
                        mbar_expect_tx(full, bytes);
                        for (int y = 0; y < nbox; ++y)
                            for (int x = 0; x < C::NBX; ++x)
                                tma_load_3d(sK + ks * C::TILE + x * 16384 + y * 8192, &tmK, 64 * x, it.j, row + 64 * y, full);
                    }
                    if (i == 0) {
                        if (nq > 0 && !(ok = mbar_wait(&bar->q_empty, (nq - 1) & 1, abort, status))) {
                            ++nk;
                            break;
                        }
                        ++nq;
                        if (lane == 0) {
                            mbar_expect_tx(&bar->q_full, 2 * qbytes);
                            for (int x = 0; x < C::NBX; ++x) {
                                tma_load_3d(sQ + x * 16384, &tmQ, 64 * x, it.j * a.G, it.s.row0 + it.t0, &bar->q_full);
                                tma_load_3d(sG + x * 16384, &tmG, 64 * x, it.j * a.G, it.s.row0 + it.t0, &bar->q_full);
                            }
                        }
                    }
                    if (nk >= VST && !(ok = mbar_wait(&bar->v_empty[vs], (nk / VST - 1) & 1, abort, status))) {
                        ++nk;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(&bar->v_full[vs], bytes);
                        for (int y = 0; y < nbox; ++y)
                            for (int x = 0; x < C::NBX; ++x)
                                tma_load_3d(sV + vs * C::TILE + x * 16384 + y * 8192, &tmV, 64 * x, it.j, row + 64 * y,
                                            &bar->v_full[vs]);
                    }
                }
            }
            // wind down: what was issued has landed (bounded; in a clean run all of it was waited for already)
            if (nq > 0) mbar_drain(&bar->q_full, (nq - 1) & 1);
            for (uint32_t s = 0; s < KST; ++s) {
                const uint32_t uses = nk > s ? (nk - 1 - s) / KST + 1 : 0;
                if (uses == 0) continue;
                if (last_land >> s & 1) mbar_drain(&bar->land[s], (land_par >> s & 1) ^ 1);
                else mbar_drain(&bar->k_full[s], (uses - 1) & 1);
            }
            if (ok)
                for (uint32_t s = 0; s < VST; ++s) {
                    const uint32_t uses = nk > s ? (nk - 1 - s) / VST + 1 : 0;
                    if (uses) mbar_drain(&bar->v_full[s], (uses - 1) & 1);
                }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer
            const uint32_t q0 = smem_u32(sQ), g0 = smem_u32(sG), k0 = smem_u32(sK), v0 = smem_u32(sV);
            uint32_t n = 0, nq = 0;   // tiles before this item, items with tiles
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                const int nt = it.tl.nt;
                if (nt == 0) continue;
                auto qk = [&](int i) -> bool {
                    const uint32_t f = n + i;
                    if (!mbar_wait(&bar->k_full[f % KST], (f / KST) & 1, abort, status)) return false;
                    tc_fence_after();
                    const uint32_t kb = k0 + uniform(f % KST) * C::TILE, id = uniform(idesc_bf16_f32(MR, it.tl.width(i), 0, 0)),
                                   dst = uniform(f & 1) * 128;
                    if (elect_one()) {
                        mma_nt<D>(dst, q0, kb, id);
                        umma_commit(&bar->s_full[f & 1]);
                    }
                    __syncwarp();
                    return true;
                };
                auto dp = [&](int i) -> bool {
                    const uint32_t f = n + i;
                    if (!mbar_wait(&bar->v_full[f % VST], (f / VST) & 1, abort, status)) return false;
                    if (f > 0 && !mbar_wait(&bar->dp_empty, (f - 1) & 1, abort, status)) return false;
                    tc_fence_after();
                    const uint32_t vb = v0 + uniform(f % VST) * C::TILE, id = uniform(idesc_bf16_f32(MR, it.tl.width(i), 0, 0));
                    if (elect_one()) {
                        mma_nt<D>(256, g0, vb, id);
                        umma_commit(&bar->dp_full);
                        umma_commit(&bar->v_empty[f % VST]);
                        if (i == nt - 1) umma_commit(&bar->q_empty);
                    }
                    __syncwarp();
                    return true;
                };
                if (!(ok = mbar_wait(&bar->q_full, nq++ & 1, abort, status))) break;
                ok = qk(0) && (nt < 2 || qk(1)) && dp(0);
                for (int i = 0; i < nt && ok; ++i) {
                    const uint32_t f = n + i;
                    if (i + 1 < nt && !(ok = dp(i + 1))) break;
                    if (!(ok = mbar_wait(&bar->ds_full[f & 1], (f >> 1) & 1, abort, status))) break;
                    tc_fence_after();
                    const uint32_t kb = k0 + uniform(f % KST) * C::TILE, src = uniform(f & 1) * 128, acc = uniform(i > 0);
                    const int steps = it.tl.width(i) >> 4;
                    if (elect_one()) {
                        mma_tn<D>(384, src, kb, acc, steps);
                        umma_commit(&bar->k_empty[f % KST]);
                        if (i == nt - 1) umma_commit(&bar->dq_full);
                    }
                    __syncwarp();
                    if (i + 2 < nt) ok = qk(i + 2);
                }
                n += nt;
            }
            if (elect_one()) umma_commit(&bar->done);
            __syncwarp();
            mbar_drain(&bar->done, 0);
        } else if (warp == 10) {
            // ------------------------------------------------------------ zeroes K rows past a tile's end
            uint32_t nk = 0, land_par = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                for (int i = 0; i < it.tl.nt && ok; ++i, ++nk) {
                    const int used = it.tl.end(i) - it.tl.start(i), width = it.tl.width(i);
                    if (used == width) continue;
                    const uint32_t ks = nk % KST;
                    if (!(ok = mbar_wait(&bar->land[ks], land_par >> ks & 1, abort, status))) break;
                    land_par ^= 1u << ks;
                    for (int r = used + (lane >> 3); r < width; r += 4)
                        for (int x = 0; x < C::NBX; ++x)
                            reinterpret_cast<uint4 *>(sK + ks * C::TILE + x * 16384 + r * 128)[lane & 7] =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->k_full[ks]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

// ---------------------------------------------------------------------------- dK, dV

constexpr int RST = 2;   // ring stages of row tiles (Q and dO, with their lse and D)

struct __align__(16) KvBars {
    uint64_t kv_full, kv_empty, r_full[RST], r_empty[RST], st_full[RST], st_empty[RST];
    uint64_t s_full, p_full, dp_full, ds_full, acc_full, done;
    uint32_t tmem_base;
    int abort;
    alignas(16) float lse2[RST][MR];   // minus lse in log2; read as float4
    alignas(16) float dd[RST][MR];
};
static_assert(offsetof(KvBars, lse2) % 16 == 0 && offsetof(KvBars, dd) % 16 == 0, "vector loads");

struct KvItem {
    int b, j, kt, far, u0, ta, tb;   // key tile, far chunk (-1: the window's rows), first key, query tokens [ta, tb)
    Seq s;
    int nt;                          // row tiles
};

__device__ __forceinline__ KvItem kv_item(const BwdArgs &w, int idx, int tok) {
    const LocArgs &a = w.a;
    KvItem it;
    it.j = idx % a.Hkv;
    idx /= a.Hkv;
    it.b = idx % a.B;
    it.kt = idx / a.B;   // early keys first: without a window they are seen by the most rows
    it.far = -1;
    if (it.kt >= w.nkt) {
        it.far = (it.kt - w.nkt) % w.nfar;
        it.kt = (it.kt - w.nkt) / w.nfar;
    }
    it.s = seq_of(a, it.b);
    it.u0 = it.kt * BK;
    const int ul = min(it.u0 + BK, it.s.kv) - 1;
    it.ta = max(0, it.u0 - it.s.pos0);
    it.tb = it.s.n;
    if (a.window < INT32_MAX) {
        const long long edge = (long long)ul + a.window - it.s.pos0;   // first token beyond the window of every key
        if (it.far < 0) {
            it.tb = (int)max(0ll, min((long long)it.s.n, edge));
        } else {
            const long long f0 = max(0ll, max((long long)it.ta, edge));
            it.ta = (int)min((long long)it.s.n, f0 + (long long)it.far * w.far_q);
            it.tb = (int)min((long long)it.s.n, f0 + (long long)(it.far + 1) * w.far_q);
        }
    }
    it.nt = it.tb > it.ta ? (it.tb - it.ta + tok - 1) / tok : 0;
    return it;
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      __nv_bfloat16 *__restrict__ dK, __nv_bfloat16 *__restrict__ dV, const __grid_constant__ BwdArgs w,
                      int tok, int nitems) {
    typedef Cfg<D> C;
    const LocArgs &a = w.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sK = base, *sV = sK + C::TILE, *sR = sV + C::TILE;   // sR: RST x (Q, dO)
    KvBars *bar = reinterpret_cast<KvBars *>(sR + RST * 2 * C::TILE);
    volatile int *abort = &bar->abort;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows that no box covers (G does not divide 128) stay zero
    for (int i = threadIdx.x; i < RST * 2 * C::TILE / 16; i += NT)
        reinterpret_cast<uint4 *>(sR)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        mbar_init(&bar->kv_full, 1);
        mbar_init(&bar->kv_empty, 1);
        for (int s = 0; s < RST; ++s) {
            mbar_init(&bar->r_full[s], 1);
            mbar_init(&bar->r_empty[s], 1);
            mbar_init(&bar->st_full[s], 1);
            mbar_init(&bar->st_empty[s], 8);
        }
        mbar_init(&bar->s_full, 1);
        mbar_init(&bar->p_full, 8);
        mbar_init(&bar->dp_full, 1);
        mbar_init(&bar->ds_full, 8);
        mbar_init(&bar->acc_full, 1);
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
    // all 512 TMEM columns are this CTA's: S^T (then P^T) at 0, dP^T (then dS^T) at 128, dV at 256, dK at 256 + D
    if (warp < 8) {
        reg_inc<208>();
        // ---------------------------------------------------------------- elementwise: thread = key, half of the rows
        const int hf = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16, cols = lane_off + 64 * hf;
        uint32_t n = 0, ni = 0;
        bool ok = true;
        for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
            const KvItem it = kv_item(w, idx, tok);
            const int u = it.u0 + r;
            const bool live = u < it.s.kv;
            for (int i = 0; i < it.nt; ++i, ++n) {
                const int st = n % RST;
                const int t0 = it.ta + i * tok, ntok = min(tok, it.tb - t0), pt = it.s.pos0 + t0;
                // columns (row token * G + head) that see this key: [c0, c1)
                const int after = min(max(u - pt, 0), tok);
                const int last = u < a.sinks ? ntok : min(ntok, (int)max(0ll, min((long long)tok, (long long)u + a.window - pt)));
                const int c0 = after * a.G - 64 * hf, c1 = live ? last * a.G - 64 * hf : -64;
                const bool full = __all_sync(FULL, c0 <= 0 && c1 >= 64);
                if (!(ok = mbar_wait(&bar->st_full[st], (n / RST) & 1, abort, status))) break;
                if (!(ok = mbar_wait(&bar->s_full, n & 1, abort, status))) break;
                tc_fence_after();
                uint32_t x[2][32];
                tmem_ld32(cols, x[0]);
                tmem_ld32(cols + 32, x[1]);
                tmem_wait_ld(x[0]);
                tmem_wait_ld(x[1]);
                const uint64_t sc2 = pair(a.scale_log2, a.scale_log2);
                const float4 *ls = reinterpret_cast<const float4 *>(&bar->lse2[st][64 * hf]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 l4 = ls[q * 8 + c / 4];   // negated
                        float y, z;
                        unpair(fma2(pair(__uint_as_float(x[q][c]), __uint_as_float(x[q][c + 1])), sc2, pair(l4.x, l4.y)), y, z);
                        x[q][c] = __float_as_uint(ex2(y));
                        x[q][c + 1] = __float_as_uint(ex2(z));
                        unpair(fma2(pair(__uint_as_float(x[q][c + 2]), __uint_as_float(x[q][c + 3])), sc2, pair(l4.z, l4.w)), y, z);
                        x[q][c + 2] = __float_as_uint(ex2(y));
                        x[q][c + 3] = __float_as_uint(ex2(z));
                    }
                    if (!full) {
                        const uint32_t m = bits(c0, c1, q);
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[q][c] = (m >> c) & 1u ? x[q][c] : 0u;
                    }
#pragma unroll
                    for (int c = 0; c < 32; c += 2)   // the tensor cores take P as bf16
                        pk[c / 2] = pack_bf16x2(__uint_as_float(x[q][c]), __uint_as_float(x[q][c + 1]));
                    tmem_st16(cols + q * 16, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full);
                if (!(ok = mbar_wait(&bar->dp_full, n & 1, abort, status))) break;
                tc_fence_after();
                const float4 *ds = reinterpret_cast<const float4 *>(&bar->dd[st][64 * hf]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t g[32], pk[16];
                    tmem_ld32(cols + 128 + q * 32, g);
                    tmem_wait_ld(g);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 d4 = ds[q * 8 + c / 4];
                        float e[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            e[y] = __uint_as_float(x[q][c + y]) * (__uint_as_float(g[c + y]) - e[y]);
                            if (!full) e[y] = x[q][c + y] ? e[y] : 0.f;   // masked: whatever dP holds there
                        }
                        pk[c / 2] = pack_bf16x2(e[0], e[1]);   // the tensor cores take dS as bf16
                        pk[c / 2 + 1] = pack_bf16x2(e[2], e[3]);
                    }
                    tmem_st16(cols + 128 + q * 16, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar->st_empty[st]);
                    mbar_arrive(&bar->ds_full);
                }
            }
            if (!ok) break;
            if (it.nt > 0) {
                if (!(ok = mbar_wait(&bar->acc_full, ni++ & 1, abort, status))) break;
                tc_fence_after();
            }
            // this half's columns of dK and dV: the outputs, or fp32 partials of a sink tile
            const bool part = it.kt < w.nst;
            const long long psz = (long long)a.B * a.Hkv * w.nst * BK * D;
            const long long prow = part ? (((long long)it.b * a.Hkv + it.j) * w.nst * BK + u) * D + hf * (D / 2) : 0;
            float *pk = part ? w.part + (it.far + 1) * psz + prow : nullptr;
            float *pv = part ? pk + (w.nfar + 1) * psz : nullptr;
            const long long at = live ? (((long long)it.b * a.Tcap + u) * a.Hkv + it.j) * D + hf * (D / 2) : 0;
            if (it.nt > 0) {
                for (int q = 0; q < D / 64; ++q) {
                    const uint32_t c = hf * (D / 2) + q * 32;
                    put32(lane_off + 256 + c, 1.f, dV + at + q * 32, part ? pv + q * 32 : nullptr, live);
                    put32(lane_off + 256 + D + c, a.scale, dK + at + q * 32, part ? pk + q * 32 : nullptr, live);
                }
                tc_fence_before();
            } else if (live) {
                for (int c = 0; c < D / 2; c += 8) {
                    if (part) {
                        *reinterpret_cast<float4 *>(pk + c) = *reinterpret_cast<float4 *>(pk + c + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
                        *reinterpret_cast<float4 *>(pv + c) = *reinterpret_cast<float4 *>(pv + c + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
                    } else {
                        *reinterpret_cast<uint4 *>(dK + at + c) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dV + at + c) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
        }
    } else {
        reg_dec<80>();
        if (warp == 8) {
            // ------------------------------------------------------------ loader
            uint32_t ni = 0, n = 0;
            const uint32_t rbytes = (uint32_t)(tok * a.G) * 128u * C::NBX;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                if (it.nt == 0) continue;
                if (ni > 0 && !(ok = mbar_wait(&bar->kv_empty, (ni - 1) & 1, abort, status))) break;
                ++ni;
                if (lane == 0) {
                    mbar_expect_tx(&bar->kv_full, 2 * C::TILE);
                    for (int y = 0; y < 2; ++y)
                        for (int x = 0; x < C::NBX; ++x) {
                            const int row = it.b * a.Tcap + it.u0 + 64 * y;
                            tma_load_3d(sK + x * 16384 + y * 8192, &tmK, 64 * x, it.j, row, &bar->kv_full);
                            tma_load_3d(sV + x * 16384 + y * 8192, &tmV, 64 * x, it.j, row, &bar->kv_full);
                        }
                }
                for (int i = 0; i < it.nt && ok; ++i) {
                    const uint32_t st = n % RST;
                    if (n >= RST && !(ok = mbar_wait(&bar->r_empty[st], (n / RST - 1) & 1, abort, status))) break;
                    if (lane == 0) {
                        uint8_t *dst = sR + st * 2 * C::TILE;
                        const int row = it.s.row0 + it.ta + i * tok;
                        mbar_expect_tx(&bar->r_full[st], 2 * rbytes);
                        for (int x = 0; x < C::NBX; ++x) {
                            tma_load_3d(dst + x * 16384, &tmQ, 64 * x, it.j * a.G, row, &bar->r_full[st]);
                            tma_load_3d(dst + C::TILE + x * 16384, &tmG, 64 * x, it.j * a.G, row, &bar->r_full[st]);
                        }
                    }
                    ++n;
                }
            }
            // wind down: what was issued has landed
            if (ni > 0) mbar_drain(&bar->kv_full, (ni - 1) & 1);
            for (uint32_t s = 0; s < RST; ++s) {
                const uint32_t uses = n > s ? (n - 1 - s) / RST + 1 : 0;
                if (uses) mbar_drain(&bar->r_full[s], (uses - 1) & 1);
            }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA issuer
            constexpr uint32_t idesc = idesc_bf16_f32(BK, MR, 0, 0);
            const uint32_t k0 = smem_u32(sK), v0 = smem_u32(sV), r0 = smem_u32(sR);
            uint32_t n = 0, ni = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                if (it.nt == 0) continue;
                if (!(ok = mbar_wait(&bar->kv_full, ni++ & 1, abort, status))) break;
                auto scores = [&](uint32_t f) -> bool {
                    if (!mbar_wait(&bar->r_full[f % RST], (f / RST) & 1, abort, status)) return false;
                    tc_fence_after();
                    const uint32_t rb = r0 + uniform(f % RST) * 2 * C::TILE;
                    if (elect_one()) {
                        mma_nt<D>(0, k0, rb, idesc);
                        umma_commit(&bar->s_full);
                    }
                    __syncwarp();
                    return true;
                };
                auto dp = [&](uint32_t f, bool last) {
                    const uint32_t rb = r0 + uniform(f % RST) * 2 * C::TILE + C::TILE;
                    if (elect_one()) {
                        mma_nt<D>(128, v0, rb, idesc);
                        umma_commit(&bar->dp_full);
                        if (last) umma_commit(&bar->kv_empty);
                    }
                    __syncwarp();
                };
                if (!(ok = scores(n))) break;
                dp(n, it.nt == 1);
                for (int i = 0; i < it.nt; ++i, ++n) {
                    if (!(ok = mbar_wait(&bar->p_full, n & 1, abort, status))) break;
                    tc_fence_after();
                    const uint32_t rb = r0 + uniform(n % RST) * 2 * C::TILE, acc = uniform(i > 0);
                    if (elect_one()) mma_tn<D>(256, 0, rb + C::TILE, acc, 8);   // dV += P^T dO
                    __syncwarp();
                    if (i + 1 < it.nt && !(ok = scores(n + 1))) break;
                    if (!(ok = mbar_wait(&bar->ds_full, n & 1, abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_tn<D>(256 + D, 128, rb, acc, 8);   // dK += dS^T Q
                        umma_commit(&bar->r_empty[n % RST]);
                        if (i == it.nt - 1) umma_commit(&bar->acc_full);
                    }
                    __syncwarp();
                    if (i + 1 < it.nt) dp(n + 1, i + 2 == it.nt);
                }
            }
            if (elect_one()) umma_commit(&bar->done);
            __syncwarp();
            mbar_drain(&bar->done, 0);
        } else if (warp == 10) {
            // ------------------------------------------------------------ lse and D of each row tile
            uint32_t n = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                for (int i = 0; i < it.nt && ok; ++i, ++n) {
                    const int t0 = it.ta + i * tok;
                    float l[4], d[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int c = lane + 32 * x, t = t0 + c / a.G;
                        const bool in = c < tok * a.G && t < it.tb;
                        const long long row = in ? (long long)(it.s.row0 + t) * a.H + it.j * a.G + c % a.G : 0;
                        l[x] = in ? a.lse[row] * -1.4426950408889634f : 0.f;
                        d[x] = in ? w.D[row] : 0.f;
                    }
                    const int st = n % RST;
                    if (n >= RST && !(ok = mbar_wait(&bar->st_empty[st], (n / RST - 1) & 1, abort, status))) break;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        bar->lse2[st][lane + 32 * x] = l[x];
                        bar->dd[st][lane + 32 * x] = d[x];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->st_full[st]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

}  // namespace

bool bwd_tc_supported(const LocArgs &a, int dtype) { return dtype == HSA_BF16 && a.max_kv > 0 && a.max_q > 0; }

cudaError_t launch_bwd_tc(const BwdArgs &w, const void *Q, const void *K, const void *V, const void *dO, void *dQ,
                          void *dK, void *dV, cudaStream_t st) {
    const LocArgs &a = w.a;
    const int tok = MR / a.G, nblk = (a.max_q + tok - 1) / tok;
    CUtensorMap mq, mg, mk, mv;
    const uint64_t d = a.d;
    const uint64_t qd[3] = {d, (uint64_t)a.H, (uint64_t)a.rows}, qs[2] = {d * 2, (uint64_t)a.H * d * 2};
    const uint32_t qb[3] = {64, (uint32_t)a.G, (uint32_t)tok};
    const uint64_t kd[3] = {d, (uint64_t)a.Hkv, (uint64_t)a.B * a.Tcap}, ks[2] = {d * 2, (uint64_t)a.Hkv * d * 2};
    const uint32_t kb[3] = {64, 1, 64};
    cudaError_t e = make_tmap_3d(&mq, Q, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mg, dO, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mk, K, kd, ks, kb);
    if (e == cudaSuccess) e = make_tmap_3d(&mv, V, kd, ks, kb);
    if (e != cudaSuccess) return e;
    const long long nq = (long long)a.B * nblk * a.Hkv, nk = (long long)a.B * (w.nkt + w.nst * w.nfar) * a.Hkv;
    auto go = [&](auto dq, auto dkv, int tile) {
        const size_t s1 = 1024 + (size_t)(2 + KST + VST) * tile + sizeof(DqBars);
        const size_t s2 = 1024 + (size_t)(2 + 2 * RST) * tile + sizeof(KvBars);
        cudaError_t x = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s1);
        if (x == cudaSuccess) x = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s2);
        if (x != cudaSuccess) return x;
        dkv<<<(unsigned)(nk < 148 ? nk : 148), NT, s2, st>>>(mq, mg, mk, mv, (__nv_bfloat16 *)dK, (__nv_bfloat16 *)dV, w,
                                                             tok, (int)nk);
        dq<<<(unsigned)(nq < 148 ? nq : 148), NT, s1, st>>>(mq, mg, mk, mv, (__nv_bfloat16 *)dQ, w, tok, nblk, (int)nq);
        return cudaGetLastError();
    };
    return a.d == 64 ? go(window_dq_kernel<64>, window_dkv_kernel<64>, Cfg<64>::TILE)
                     : go(window_dq_kernel<128>, window_dkv_kernel<128>, Cfg<128>::TILE);
}

}  // namespace local
}  // namespace hsa
