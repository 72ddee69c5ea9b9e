// window_bwd.cu -- backward of the sliding-window attention on tcgen05 (bf16).
//
// With P = exp2(scale_log2 S - lse_log2), S = Q K^T, dP = dO V^T, D = rowsum(dO o O)
// (few keys: rowsum(P o dP), few_rowdot_kernel):
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
// Roles in both: four elementwise warpgroups (two take every other tile, each thread half of
// a row's 64 columns), a loader warp (TMA), two or three MMA warps (converged, one lane
// elected; a product that waits for its operands must not hold up the others), a helper
// warp.  Tiles are 128 x 64, so that S and dP fit TMEM twice next to the accumulators.
//
// Bound: the hand-offs between product and elementwise warps, then the products.  16384
// tokens, window 2048, 32 + 8 heads of 128: dK, dV 1.12 ms (its products alone 0.77, its
// elementwise part alone 0.84), dQ 0.81 ms (0.55, 0.61); with tiles of 128 x 128 and two
// elementwise warpgroups on the same tile 1.30 and 0.76.
#include <stddef.h>

#include "local.cuh"
#include "local_sm100.cuh"

namespace hsa {
namespace local {

namespace {

using namespace sm100;

constexpr int MR = 128;   // rows of an accumulator: query rows (dQ) or keys (dK, dV)
constexpr int RR = 64;    // the other side's rows per tile: keys (dQ) or query rows (dK, dV)

template <int D> struct Cfg {
    static constexpr int NBX = D / 64, TILE = MR * D * 2, RT = RR * D * 2;   // bytes of the two kinds of tile
};

// ---------------------------------------------------------------------------- shared pieces

// (d_tmem) = A B^T: A a K-major tile of 128 x D, B one of 64 x D in shared memory; N in idesc.  The descriptors are
// made before the issuing lane is elected: inside its branch they would count as per-thread values.
template <int D>
__device__ __forceinline__ void mma_nt(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        constexpr uint32_t step = 32 >> 4, abox = 16384 >> 4, bbox = RR * 128 >> 4;
        umma_bf16(d_tmem, ad + (kk >> 2) * abox + (kk & 3) * step, bd + (kk >> 2) * bbox + (kk & 3) * step, idesc, kk != 0);
    }
}
// (d_tmem) (+)= A B: A bf16 in TMEM, B a tile of 64 x D in shared memory, rows contracted; the first `steps` of
// 4 steps of 16.  The two halves of A's columns (one per warpgroup) start 32 TMEM columns apart.
template <int D>
__device__ __forceinline__ void mma_tn(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, uint32_t accumulate, int steps) {
    constexpr uint32_t idesc = idesc_bf16_f32(MR, D, 0, 1);
    if (steps == 4) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ts(d_tmem, a_tmem + kk / 2 * 32 + kk % 2 * 8, bd + kk * (2048 >> 4), idesc, kk == 0 ? accumulate : 1);
    } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            if (kk < steps)
                umma_bf16_ts(d_tmem, a_tmem + kk / 2 * 32 + kk % 2 * 8, bd + kk * (2048 >> 4), idesc, kk == 0 ? accumulate : 1);
    }
}
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr) { return desc_mnmajor_sw128(saddr, RR * 128, 1024); }

// N (16 or 32) columns of an fp32 accumulator, times f, to consecutive elements: bf16, or fp32 partials
template <int N>
__device__ __forceinline__ void put(uint32_t taddr, float f, __nv_bfloat16 *h, float *w, bool live) {
    uint32_t o[N];
    if constexpr (N == 32) tmem_ld32(taddr, o);
    else tmem_ld16(taddr, o);
    tmem_wait_ld(o);
    if (!live) return;
    if (w) {
#pragma unroll
        for (int c = 0; c < N; c += 4)
            *reinterpret_cast<float4 *>(w + c) =
                make_float4(__uint_as_float(o[c]) * f, __uint_as_float(o[c + 1]) * f, __uint_as_float(o[c + 2]) * f,
                            __uint_as_float(o[c + 3]) * f);
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            uint32_t x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[y] = pack_bf16x2(__uint_as_float(o[c + 2 * y]) * f, __uint_as_float(o[c + 2 * y + 1]) * f);
            *reinterpret_cast<uint4 *>(h + c) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
}

// bits of columns 0 .. 31 in [c0, c1)
__device__ __forceinline__ uint32_t bits(int c0, int c1) {
    auto below = [](int y) -> uint32_t { return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u; };
    return below(c1) & ~below(c0);
}

// One thread's 32 columns of a tile.  First half: P = exp2(scale_log2 S + nl) in x, where `full` or bit set in m.
__device__ __forceinline__ void make_p(uint32_t (&x)[32], uint64_t sc2, const float *nl, bool rowwise, bool full, uint32_t m) {
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const float4 l4 = rowwise ? make_float4(*nl, *nl, *nl, *nl) : *reinterpret_cast<const float4 *>(nl + c);
        float y, z;
        unpair(fma2(pair(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, pair(l4.x, l4.y)), y, z);
        x[c] = __float_as_uint(ex2(y));
        x[c + 1] = __float_as_uint(ex2(z));
        unpair(fma2(pair(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2, pair(l4.z, l4.w)), y, z);
        x[c + 2] = __float_as_uint(ex2(y));
        x[c + 3] = __float_as_uint(ex2(z));
    }
    if (!full) {
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = (m >> c) & 1u ? x[c] : 0u;
    }
}
// Second half: dS = P (dP - D) as bf16 pairs (the tensor cores take it so); where masked, whatever dP holds there
// (NaN included) must not come through.
__device__ __forceinline__ void make_ds(const uint32_t (&x)[32], const uint32_t (&g)[32], const float *nd, bool rowwise, bool full,
                                        uint32_t m, uint32_t (&pk)[16]) {
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const float4 d4 = rowwise ? make_float4(*nd, *nd, *nd, *nd) : *reinterpret_cast<const float4 *>(nd + c);
        float e[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            e[y] = __uint_as_float(x[c + y]) * (__uint_as_float(g[c + y]) - e[y]);
            if (!full) e[y] = (m >> (c + y)) & 1u ? e[y] : 0.f;
        }
        pk[c / 2] = pack_bf16x2(e[0], e[1]);
        pk[c / 2 + 1] = pack_bf16x2(e[2], e[3]);
    }
}

// The key tiles of a row tile: the sinks' from 0, then the window's from its first key;
// the last of each is cut to a multiple of 16 keys.
struct KeyTiles {
    int lo, hi, ns, nst, nt;
    __device__ __forceinline__ int start(int i) const { return i < nst ? i * RR : lo + (i - nst) * RR; }
    __device__ __forceinline__ int end(int i) const { return min(start(i) + RR, i < nst ? ns : hi); }
    __device__ __forceinline__ int width(int i) const { return (end(i) - start(i) + 15) & ~15; }
};

__device__ __forceinline__ KeyTiles key_tiles(int pa, int pb, int kv, int window, int sinks) {
    KeyTiles t;
    t.hi = max(0, min(pb + 1, kv));
    t.lo = min(pa >= window ? pa - window + 1 : 0, t.hi);   // window may be INT32_MAX
    t.ns = min(sinks, t.lo);
    t.nst = (t.ns + RR - 1) / RR;
    t.nt = t.nst + (t.hi - t.lo + RR - 1) / RR;
    return t;
}

// ---------------------------------------------------------------------------- dQ

constexpr int NTQ = 768;          // a warp for each of the three products
constexpr int KST = 6, VST = 4;   // ring stages: K stays until dS K, V only until dO V^T
constexpr int QSB = 4;            // TMEM buffers of S: a tile's columns are held until dS K has read dS from them

struct __align__(8) DqBars {
    uint64_t q_full, q_empty, k_full[KST], k_empty[KST], land[KST], v_full[VST], v_empty[VST];
    uint64_t s_full[QSB], s_empty[QSB], ds_full[QSB], dp_full[2], dp_empty[2], dq_full, dq_empty, done[4];   // [TMEM buffer]
    uint32_t tmem_base;
    uint32_t step;   // K tiles that the loader has issued
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
__global__ void __launch_bounds__(NTQ, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     __nv_bfloat16 *__restrict__ dQ, const __grid_constant__ BwdArgs w, int tok, int nblk, int nitems) {
    typedef Cfg<D> C;
    const LocArgs &a = w.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sG = sQ + C::TILE, *sK = sG + C::TILE, *sV = sK + KST * C::RT;
    DqBars *bar = reinterpret_cast<DqBars *>(sV + VST * C::RT);
    volatile int *abort = &bar->abort;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows that no box covers (G does not divide 128) stay zero
    for (int i = threadIdx.x; i < 2 * C::TILE / 16; i += NTQ) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, 1);
        mbar_init(&bar->q_empty, 2);   // S and dP
        for (int s = 0; s < KST; ++s) {
            mbar_init(&bar->k_full[s], 1);
            mbar_init(&bar->k_empty[s], 1);
            mbar_init(&bar->land[s], 1);
        }
        for (int s = 0; s < VST; ++s) {
            mbar_init(&bar->v_full[s], 1);
            mbar_init(&bar->v_empty[s], 1);
        }
        for (int s = 0; s < QSB; ++s) {
            mbar_init(&bar->s_full[s], 1);
            mbar_init(&bar->s_empty[s], 1);
            mbar_init(&bar->ds_full[s], 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar->dp_full[s], 1);
            mbar_init(&bar->dp_empty[s], 8);
        }
        for (int s = 0; s < 4; ++s) mbar_init(&bar->done[s], 1);
        mbar_init(&bar->dq_full, 1);
        mbar_init(&bar->dq_empty, 16);
        bar->step = 0;
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(&bar->tmem_base, 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 TMEM columns are this CTA's: four buffers of S (then dS) at 0 .., two of dP at 256 / 320; dQ at 384
    if (warp < 16) {
        reg_inc<96>();
        // ---------------------------------------------------------------- elementwise: thread = half a row of every other tile
        const int pr = warp >> 3, hf = warp >> 2 & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16, cP = lane_off + 256 + pr * 64 + hf * 32;
        uint32_t n = 0, ni = 0;
        bool ok = true;
        const uint64_t sc2 = pair(a.scale_log2, a.scale_log2);
        for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
            const DqItem it = dq_item(a, idx, tok, nblk);
            const int t = it.t0 + r / a.G;
            const bool live = r < tok * a.G && t < it.te;
            const int p = it.s.pos0 + t;
            const int we = live ? min(p, it.s.kv - 1) : -1, wa = live && p >= a.window ? p - a.window + 1 : 0;
            const long long row = live ? (long long)(it.s.row0 + t) * a.H + it.j * a.G + r % a.G : 0;
            const float nl = live ? a.lse[row] * -1.4426950408889634f : 0.f, dd = live ? w.D[row] : 0.f;
            const KeyTiles tl = it.tl;
            for (int i = 0; i < tl.nt; ++i, ++n) {
                if ((int)(n & 1) != pr) continue;
                // visible columns: c <= we - u0, before the tile's end, and (c >= wa - u0 or c < sinks - u0)
                const int u0 = tl.start(i) + 32 * hf, c1 = min(we + 1, tl.end(i)) - u0;
                const bool full = __all_sync(FULL, c1 >= 32 && (wa <= u0 || u0 + 32 <= a.sinks));
                const uint32_t m = full ? ~0u : bits(0, c1) & (bits(wa - u0, 32) | bits(0, a.sinks - u0));
                const uint32_t sb = n % QSB, cS = lane_off + sb * 64 + hf * 32;
                if (!(ok = mbar_wait(&bar->s_full[sb], (n / QSB) & 1, abort, status))) break;
                tc_fence_after();
                uint32_t x[32], g[32], pk[16];
                tmem_ld32(cS, x);
                tmem_wait_ld(x);
                make_p(x, sc2, &nl, true, full, m);
                if (!(ok = mbar_wait(&bar->dp_full[pr], (n >> 1) & 1, abort, status))) break;
                tc_fence_after();
                tmem_ld32(cP, g);
                tmem_wait_ld(g);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->dp_empty[pr]);
                make_ds(x, g, &dd, true, full, m, pk);
                tmem_st16(cS, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->ds_full[sb]);
            }
            if (!ok) break;
            // epilogue: a quarter of the columns per warpgroup
            constexpr int QC = D / 4;
            const int col = (warp >> 2) * QC;
            __nv_bfloat16 *dst = dQ + row * D + col;
            if (tl.nt > 0) {
                if (!(ok = mbar_wait(&bar->dq_full, ni++ & 1, abort, status))) break;
                tc_fence_after();
                put<QC>(lane_off + 384 + col, a.scale, dst, nullptr, live);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->dq_empty);
            } else if (live) {
                for (int c = 0; c < QC; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        reg_dec<48>();
        if (warp == 16) {
            // ------------------------------------------------------------ loader
            uint32_t nq = 0, nk = 0, nv = 0, land_par = 0, last_land = 0;
            const uint32_t qbytes = (uint32_t)(tok * a.G) * 128u * C::NBX;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                for (int i = 0; i < it.tl.nt; ++i) {
                    const int row = it.b * a.Tcap + it.tl.start(i);
                    const uint32_t ks = nk % KST, vs = nv % VST;
                    if (nk >= KST && !(ok = mbar_wait(&bar->k_empty[ks], (nk / KST - 1) & 1, abort, status))) break;
                    // K rows past the tile's end would meet dS = 0 as B rows: the helper zeroes them first
                    const bool dead = it.tl.end(i) < it.tl.start(i) + it.tl.width(i);
                    uint64_t *full = dead ? &bar->land[ks] : &bar->k_full[ks];
                    if (dead) {
                        land_par ^= 1u << ks;
                        last_land |= 1u << ks;
                    } else {
                        last_land &= ~(1u << ks);
                    }
                    if (lane == 0) {
                        mbar_expect_tx(full, C::RT);
                        for (int x = 0; x < C::NBX; ++x)
                            tma_load_3d(sK + ks * C::RT + x * RR * 128, &tmK, 64 * x, it.j, row, full);
                    }
                    ++nk;
                    if (lane == 0) *(volatile uint32_t *)&bar->step = nk;
                    if (i == 0) {
                        if (nq > 0 && !(ok = mbar_wait(&bar->q_empty, (nq - 1) & 1, abort, status))) break;
                        ++nq;
                        if (lane == 0) {
                            mbar_expect_tx(&bar->q_full, 2 * qbytes);
                            for (int x = 0; x < C::NBX; ++x) {
                                tma_load_3d(sQ + x * 16384, &tmQ, 64 * x, it.j * a.G, it.s.row0 + it.t0, &bar->q_full);
                                tma_load_3d(sG + x * 16384, &tmG, 64 * x, it.j * a.G, it.s.row0 + it.t0, &bar->q_full);
                            }
                        }
                    }
                    if (nv >= VST && !(ok = mbar_wait(&bar->v_empty[vs], (nv / VST - 1) & 1, abort, status))) break;
                    if (lane == 0) {
                        mbar_expect_tx(&bar->v_full[vs], C::RT);
                        for (int x = 0; x < C::NBX; ++x)
                            tma_load_3d(sV + vs * C::RT + x * RR * 128, &tmV, 64 * x, it.j, row, &bar->v_full[vs]);
                    }
                    ++nv;
                }
            }
            // wind down: what was issued has landed
            if (nq > 0) mbar_drain(&bar->q_full, (nq - 1) & 1);
            for (uint32_t s = 0; s < KST; ++s) {
                const uint32_t uses = nk > s ? (nk - 1 - s) / KST + 1 : 0;
                if (uses == 0) continue;
                if (last_land >> s & 1) mbar_drain(&bar->land[s], (land_par >> s & 1) ^ 1);
                else mbar_drain(&bar->k_full[s], (uses - 1) & 1);
            }
            for (uint32_t s = 0; s < VST; ++s) {
                const uint32_t uses = nv > s ? (nv - 1 - s) / VST + 1 : 0;
                if (uses) mbar_drain(&bar->v_full[s], (uses - 1) & 1);
            }
        } else if (warp == 17) {
            // ------------------------------------------------------------ MMA issuer of S
            const uint32_t k0 = smem_u32(sK);
            const uint64_t qd = desc_kmajor_sw128(smem_u32(sQ));
            uint32_t f = 0, nq = 0;   // tiles, items with tiles so far
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                const int nt = it.tl.nt;
                if (nt == 0) continue;
                if (!(ok = mbar_wait(&bar->q_full, nq++ & 1, abort, status))) break;
                for (int i = 0; i < nt; ++i, ++f) {
                    // once the product that read the last dS from these columns is done
                    const uint32_t ks = f % KST, sb = f % QSB;
                    const uint64_t kd = desc_kmajor_sw128(k0 + uniform(ks) * C::RT);
                    const uint32_t id = uniform(idesc_bf16_f32(MR, it.tl.width(i), 0, 0)), dst = uniform(sb) * 64;
                    if (!(ok = mbar_wait(&bar->k_full[ks], (f / KST) & 1, abort, status))) break;
                    if (f >= QSB && !(ok = mbar_wait(&bar->s_empty[sb], (f / QSB - 1) & 1, abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_nt<D>(dst, qd, kd, id);
                        umma_commit(&bar->s_full[sb]);
                        if (i == nt - 1) umma_commit(&bar->q_empty);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) umma_commit(&bar->done[0]);
            __syncwarp();
            mbar_drain(&bar->done[0], 0);
        } else if (warp == 20) {
            // ------------------------------------------------------------ MMA issuer of dP
            const uint32_t v0 = smem_u32(sV);
            const uint64_t gd = desc_kmajor_sw128(smem_u32(sG));
            uint32_t f = 0, nq = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                const int nt = it.tl.nt;
                if (nt == 0) continue;
                if (!(ok = mbar_wait(&bar->q_full, nq++ & 1, abort, status))) break;
                for (int i = 0; i < nt; ++i, ++f) {
                    // once dP(f - 2) has been read
                    const uint32_t vs = f % VST, sb = f & 1;
                    const uint64_t vd = desc_kmajor_sw128(v0 + uniform(vs) * C::RT);
                    const uint32_t id = uniform(idesc_bf16_f32(MR, it.tl.width(i), 0, 0)), dst = 256 + uniform(sb) * 64;
                    if (!(ok = mbar_wait(&bar->v_full[vs], (f / VST) & 1, abort, status))) break;
                    if (f >= 2 && !(ok = mbar_wait(&bar->dp_empty[sb], ((f >> 1) - 1) & 1, abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_nt<D>(dst, gd, vd, id);
                        umma_commit(&bar->dp_full[sb]);
                        umma_commit(&bar->v_empty[vs]);
                        if (i == nt - 1) umma_commit(&bar->q_empty);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) umma_commit(&bar->done[2]);
            __syncwarp();
            mbar_drain(&bar->done[2], 0);
        } else if (warp == 18) {
            // ------------------------------------------------------------ MMA issuer of dQ
            const uint32_t k0 = smem_u32(sK);
            uint32_t f = 0, nq = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                const int nt = it.tl.nt;
                if (nt == 0) continue;
                // the previous item's dQ has left TMEM
                if (nq > 0 && !(ok = mbar_wait(&bar->dq_empty, (nq - 1) & 1, abort, status))) break;
                ++nq;
                for (int i = 0; i < nt; ++i, ++f) {
                    const uint32_t ks = f % KST, sb = f % QSB;
                    const uint64_t kd = desc_rows(k0 + uniform(ks) * C::RT);
                    const uint32_t src = uniform(sb) * 64, acc = uniform(i > 0);
                    const int steps = it.tl.width(i) >> 4;
                    if (!(ok = mbar_wait(&bar->ds_full[sb], (f / QSB) & 1, abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_tn<D>(384, src, kd, acc, steps);
                        umma_commit(&bar->s_empty[sb]);
                        umma_commit(&bar->k_empty[ks]);
                        if (i == nt - 1) umma_commit(&bar->dq_full);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) umma_commit(&bar->done[1]);
            __syncwarp();
            mbar_drain(&bar->done[1], 0);
        } else if (warp == 19) {
            // ------------------------------------------------------------ zeroes K rows past a tile's end
            uint32_t nk = 0, land_par = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const DqItem it = dq_item(a, idx, tok, nblk);
                for (int i = 0; i < it.tl.nt && ok; ++i, ++nk) {
                    const int used = it.tl.end(i) - it.tl.start(i), width = it.tl.width(i);
                    if (used == width) continue;
                    const uint32_t ks = nk % KST;
                    if (!(ok = mbar_wait_ahead(&bar->land[ks], land_par >> ks & 1, abort, status, &bar->step))) break;
                    land_par ^= 1u << ks;
                    for (int r = used + (lane >> 3); r < width; r += 4)
                        for (int x = 0; x < C::NBX; ++x)
                            reinterpret_cast<uint4 *>(sK + ks * C::RT + x * RR * 128 + r * 128)[lane & 7] =
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
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

// ---------------------------------------------------------------------------- dK, dV

constexpr int NTK = 640;   // two warps for the four products, each issuing what is due first: more warps measured slower
constexpr int RST = 4;   // ring stages of row tiles (Q and dO, with their lse and D)

struct __align__(16) KvBars {
    uint64_t kv_full, kv_empty, r_full[RST], r_empty[RST], st_full[RST], st_empty[RST];
    uint64_t s_full[2], s_empty[2], p_full[2], dp_full[2], dp_empty[2], ds_full[2], acc_full, acc_empty, done[2];   // [TMEM buffer]
    uint32_t tmem_base;
    int abort;
    alignas(16) float lse2[RST][RR];   // minus lse in log2; read as float4
    alignas(16) float dd[RST][RR];
};
static_assert(offsetof(KvBars, lse2) % 16 == 0 && offsetof(KvBars, dd) % 16 == 0, "vector loads");

struct KvItem {
    int b, j, kt, slot, u0, ta, tb;   // key tile, its partials' slot, first key, query tokens [ta, tb)
    Seq s;
    int nt;                           // row tiles
};

__device__ __forceinline__ KvItem kv_item(const BwdArgs &w, int idx, int tok) {
    const LocArgs &a = w.a;
    KvItem it;
    it.j = idx % a.Hkv;
    idx /= a.Hkv;
    it.b = idx % a.B;
    it.s = seq_of(a, it.b);
    const KvRange r = kv_range(w, it.s, idx / a.B, MR);   // early keys first: without a window the most rows see them
    it.kt = r.kt;
    it.slot = r.slot;
    it.u0 = r.kt * MR;
    it.ta = r.ta;
    it.tb = r.tb;
    it.nt = (it.tb - it.ta + tok - 1) / tok;
    return it;
}

template <int D>
__global__ void __launch_bounds__(NTK, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      __nv_bfloat16 *__restrict__ dK, __nv_bfloat16 *__restrict__ dV, const __grid_constant__ BwdArgs w,
                      int tok, int nitems) {
    typedef Cfg<D> C;
    const LocArgs &a = w.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int RT = C::RT;   // bytes of a row tile of Q or dO
    uint8_t *sK = base, *sV = sK + C::TILE, *sR = sV + C::TILE;   // sR: RST x (Q, dO)
    KvBars *bar = reinterpret_cast<KvBars *>(sR + RST * 2 * RT);
    volatile int *abort = &bar->abort;
    uint32_t *status = a.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows that no box covers (G does not divide 64) stay zero
    for (int i = threadIdx.x; i < RST * 2 * RT / 16; i += NTK) reinterpret_cast<uint4 *>(sR)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        mbar_init(&bar->kv_full, 1);
        mbar_init(&bar->kv_empty, 1);
        for (int s = 0; s < RST; ++s) {
            mbar_init(&bar->r_full[s], 1);
            mbar_init(&bar->r_empty[s], 1);
            mbar_init(&bar->st_full[s], 1);
            mbar_init(&bar->st_empty[s], 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar->s_full[s], 1);
            mbar_init(&bar->s_empty[s], 1);
            mbar_init(&bar->p_full[s], 8);
            mbar_init(&bar->dp_full[s], 1);
            mbar_init(&bar->dp_empty[s], 1);
            mbar_init(&bar->ds_full[s], 8);
            mbar_init(&bar->done[s], 1);
        }
        mbar_init(&bar->acc_full, 1);
        mbar_init(&bar->acc_empty, 16);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(&bar->tmem_base, 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 TMEM columns are this CTA's: two buffers of S^T (then P^T) at 0 / 64 and of dP^T (then dS^T) at
    // 128 / 192; dV at 256, dK at 256 + D
    if (warp < 16) {
        reg_inc<104>();
        // ---------------------------------------------------------------- elementwise: thread = key, half of every other tile
        const int pr = warp >> 3, hf = warp >> 2 & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16, cS = lane_off + pr * 64 + hf * 32, cP = cS + 128;
        uint32_t n = 0, ni = 0;
        bool ok = true;
        const uint64_t sc2 = pair(a.scale_log2, a.scale_log2);
        for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
            const KvItem it = kv_item(w, idx, tok);
            const int u = it.u0 + r;
            const bool live = u < it.s.kv;
            const int nt = it.nt, tb = it.tb, ta = it.ta, p0 = it.s.pos0;
            for (int i = 0; i < nt; ++i, ++n) {
                if ((int)(n & 1) != pr) continue;
                const int st = n % RST, t0 = ta + i * tok, pt = p0 + t0;
                // whole tiles first: every key of the tile is seen by every row
                const bool full = t0 + tok <= tb && tok * a.G == RR && it.u0 + MR <= it.s.kv && it.u0 + MR - 1 <= pt &&
                                  (pt + tok - 1 - it.u0 < a.window || it.u0 + MR <= a.sinks);
                uint32_t m = ~0u;
                if (!full) {
                    // columns (row token * G + head) that see this key: [c0, c1)
                    const int ntok = min(tok, tb - t0), after = min(max(u - pt, 0), tok);
                    const int last = u < a.sinks ? ntok : min(ntok, (int)max(0ll, min((long long)tok, (long long)u + a.window - pt)));
                    m = bits(after * a.G - 32 * hf, live ? last * a.G - 32 * hf : 0);
                }
                if (!(ok = mbar_wait(&bar->st_full[st], (n / RST) & 1, abort, status))) break;
                if (!(ok = mbar_wait(&bar->s_full[pr], (n >> 1) & 1, abort, status))) break;
                tc_fence_after();
                uint32_t x[32], g[32], pk[16];
                tmem_ld32(cS, x);
                tmem_wait_ld(x);
                make_p(x, sc2, &bar->lse2[st][32 * hf], false, full, m);
#pragma unroll
                for (int c = 0; c < 32; c += 2)   // the tensor cores take P as bf16
                    pk[c / 2] = pack_bf16x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                tmem_st16(cS, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full[pr]);
                if (!(ok = mbar_wait(&bar->dp_full[pr], (n >> 1) & 1, abort, status))) break;
                tc_fence_after();
                tmem_ld32(cP, g);
                tmem_wait_ld(g);
                make_ds(x, g, &bar->dd[st][32 * hf], false, full, m, pk);
                tmem_st16(cP, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar->st_empty[st]);
                    mbar_arrive(&bar->ds_full[pr]);
                }
            }
            if (!ok) break;
            if (it.nt > 0) {
                if (!(ok = mbar_wait(&bar->acc_full, ni++ & 1, abort, status))) break;
                tc_fence_after();
            }
            // this warpgroup's quarter of the columns of dK and dV: the outputs, or fp32 partials
            constexpr int QC = D / 4;
            const int col = (warp >> 2) * QC;
            const bool part = it.kt < w.npt;
            const long long psz = (long long)a.B * a.Hkv * w.npt * MR * D;
            const long long prow = part ? (((long long)it.b * a.Hkv + it.j) * w.npt * MR + u) * D + col : 0;
            float *pk = part ? w.part + it.slot * psz + prow : nullptr;
            float *pv = part ? pk + (w.nwin + w.nfar) * psz : nullptr;
            const long long at = live ? (((long long)it.b * a.Tcap + u) * a.Hkv + it.j) * D + col : 0;
            if (it.nt > 0) {
                put<QC>(lane_off + 256 + col, 1.f, dV + at, pv, live);
                put<QC>(lane_off + 256 + D + col, a.scale, dK + at, pk, live);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->acc_empty);
            } else if (live) {
                for (int c = 0; c < QC; c += 8) {
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
        reg_dec<64>();
        if (warp == 16) {
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
                        uint8_t *dst = sR + st * 2 * RT;
                        const int row = it.s.row0 + it.ta + i * tok;
                        mbar_expect_tx(&bar->r_full[st], 2 * rbytes);
                        for (int x = 0; x < C::NBX; ++x) {
                            tma_load_3d(dst + x * RR * 128, &tmQ, 64 * x, it.j * a.G, row, &bar->r_full[st]);
                            tma_load_3d(dst + RT + x * RR * 128, &tmG, 64 * x, it.j * a.G, row, &bar->r_full[st]);
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
        } else if (warp == 17) {
            // ------------------------------------------------------------ MMA issuer of S^T and dP^T: whichever is due first
            constexpr uint32_t idesc = idesc_bf16_f32(MR, RR, 0, 0);
            const uint32_t r0 = smem_u32(sR);
            const uint64_t kd = desc_kmajor_sw128(smem_u32(sK)), vd = desc_kmajor_sw128(smem_u32(sV));
            uint32_t n = 0, ni = 0;   // row tiles before this item, items with tiles so far
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                const uint32_t nt = it.nt;
                if (nt == 0) continue;
                if (!(ok = mbar_wait(&bar->kv_full, ni++ & 1, abort, status))) break;
                PollLimit limit;
                for (uint32_t is = 0, ip = 0; ip < nt;) {
                    bool moved = false;
                    if (is < nt) {   // S, once the product that read P(f - 2) from its columns is done
                        const uint32_t f = n + is, st = f % RST, sb = f & 1;
                        if (mbar_test_warp(&bar->r_full[st], (f / RST) & 1) &&
                            (f < 2 || mbar_test_warp(&bar->s_empty[sb], ((f >> 1) - 1) & 1))) {
                            const uint64_t qd = desc_kmajor_sw128(r0 + uniform(st) * 2 * RT);
                            const uint32_t dst = uniform(sb) * 64;
                            tc_fence_after();
                            if (elect_one()) {
                                mma_nt<D>(dst, kd, qd, idesc);
                                umma_commit(&bar->s_full[sb]);
                            }
                            __syncwarp();
                            ++is;
                            moved = true;
                        }
                    }
                    if (ip < is) {   // dP, once the product that read dS(f - 2) from its columns is done
                        const uint32_t f = n + ip, st = f % RST, sb = f & 1;
                        if (f < 2 || mbar_test_warp(&bar->dp_empty[sb], ((f >> 1) - 1) & 1)) {
                            const uint64_t gd = desc_kmajor_sw128(r0 + uniform(st) * 2 * RT + RT);
                            const uint32_t dst = 128 + uniform(sb) * 64;
                            tc_fence_after();
                            if (elect_one()) {
                                mma_nt<D>(dst, vd, gd, idesc);
                                umma_commit(&bar->dp_full[sb]);
                                if (ip == nt - 1) umma_commit(&bar->kv_empty);
                            }
                            __syncwarp();
                            ++ip;
                            moved = true;
                        }
                    }
                    if (moved) limit.progress();
                    else if (limit.expired(abort, status)) {
                        ok = false;
                        break;
                    }
                }
                n += nt;
            }
            if (elect_one()) umma_commit(&bar->done[0]);
            __syncwarp();
            mbar_drain(&bar->done[0], 0);
        } else if (warp == 18) {
            // ------------------------------------------------------------ MMA issuer of dV and dK: whichever is due first
            const uint32_t r0 = smem_u32(sR);
            uint32_t n = 0, ni = 0;
            bool ok = true;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                const uint32_t nt = it.nt;
                if (nt == 0) continue;
                // the previous item's sums have left TMEM
                if (ni > 0 && !(ok = mbar_wait(&bar->acc_empty, (ni - 1) & 1, abort, status))) break;
                ++ni;
                PollLimit limit;
                for (uint32_t iv = 0, ik = 0; ik < nt;) {
                    bool moved = false;
                    if (iv < nt) {
                        const uint32_t f = n + iv, st = f % RST, sb = f & 1;
                        if (mbar_test_warp(&bar->p_full[sb], (f >> 1) & 1)) {
                            const uint64_t gd = desc_rows(r0 + uniform(st) * 2 * RT + RT);
                            const uint32_t src = uniform(sb) * 64, acc = uniform(iv > 0);
                            tc_fence_after();
                            if (elect_one()) {
                                mma_tn<D>(256, src, gd, acc, 4);   // dV += P^T dO
                                umma_commit(&bar->s_empty[sb]);
                            }
                            __syncwarp();
                            ++iv;
                            moved = true;
                        }
                    }
                    if (ik < iv) {
                        const uint32_t f = n + ik, st = f % RST, sb = f & 1;
                        if (mbar_test_warp(&bar->ds_full[sb], (f >> 1) & 1)) {
                            const uint64_t qd = desc_rows(r0 + uniform(st) * 2 * RT);
                            const uint32_t src = 128 + uniform(sb) * 64, acc = uniform(ik > 0);
                            tc_fence_after();
                            if (elect_one()) {
                                mma_tn<D>(256 + D, src, qd, acc, 4);   // dK += dS^T Q
                                umma_commit(&bar->dp_empty[sb]);
                                umma_commit(&bar->r_empty[st]);
                                if (ik == nt - 1) umma_commit(&bar->acc_full);
                            }
                            __syncwarp();
                            ++ik;
                            moved = true;
                        }
                    }
                    if (moved) limit.progress();
                    else if (limit.expired(abort, status)) {
                        ok = false;
                        break;
                    }
                }
                n += nt;
            }
            if (elect_one()) umma_commit(&bar->done[1]);
            __syncwarp();
            mbar_drain(&bar->done[1], 0);
        } else {
            // ------------------------------------------------------------ lse and D of each row tile, their loads two tiles
            // ahead of the stores (a tile's loads take about as long as a tile)
            uint32_t n = 0;
            bool ok = true;
            const int c0 = lane / a.G, c1 = (lane + 32) / a.G;                // token of this lane's two rows
            const int h0 = lane % a.G, h1 = (lane + 32) % a.G;
            for (int idx = blockIdx.x; idx < nitems && ok; idx += gridDim.x) {
                const KvItem it = kv_item(w, idx, tok);
                auto fetch = [&](int i, float (&x)[4]) {
                    const int t0 = it.ta + i * tok;
                    const bool in0 = i < it.nt && c0 < tok && t0 + c0 < it.tb, in1 = i < it.nt && c1 < tok && t0 + c1 < it.tb;
                    const long long r0 = in0 ? (long long)(it.s.row0 + t0 + c0) * a.H + it.j * a.G + h0 : 0;
                    const long long r1 = in1 ? (long long)(it.s.row0 + t0 + c1) * a.H + it.j * a.G + h1 : 0;
                    x[0] = in0 ? a.lse[r0] * -1.4426950408889634f : 0.f;
                    x[1] = in1 ? a.lse[r1] * -1.4426950408889634f : 0.f;
                    x[2] = in0 ? w.D[r0] : 0.f;
                    x[3] = in1 ? w.D[r1] : 0.f;
                };
                auto put = [&](int i, const float (&x)[4]) -> bool {
                    const uint32_t f = n + i, st = f % RST;
                    if (f >= RST && !mbar_wait(&bar->st_empty[st], (f / RST - 1) & 1, abort, status)) return false;
                    bar->lse2[st][lane] = x[0];
                    bar->lse2[st][lane + 32] = x[1];
                    bar->dd[st][lane] = x[2];
                    bar->dd[st][lane + 32] = x[3];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->st_full[st]);
                    return true;
                };
                float x[4], y[4];
                fetch(0, x);
                fetch(1, y);
                for (int i = 0; i < it.nt && ok; i += 2) {
                    if (!(ok = put(i, x))) break;
                    fetch(i + 2, x);
                    if (i + 1 < it.nt && !(ok = put(i + 1, y))) break;
                    fetch(i + 3, y);
                }
                n += it.nt;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

}  // namespace

bool bwd_tc_supported(const LocArgs &a, int dtype) { return dtype == HSA_BF16 && a.max_kv > 0 && a.max_q > 0; }

cudaError_t launch_bwd_tc(const BwdArgs &w, const void *Q, const void *K, const void *V, const void *dO, void *dQ,
                          void *dK, void *dV, cudaStream_t st) {
    const LocArgs &a = w.a;
    const int tok = MR / a.G, nblk = (a.max_q + tok - 1) / tok, rtok = RR / a.G;
    CUtensorMap mq, mg, rq, rg, mk, mv;
    const uint64_t d = a.d;
    const uint64_t qd[3] = {d, (uint64_t)a.H, (uint64_t)a.rows}, qs[2] = {d * 2, (uint64_t)a.H * d * 2};
    const uint32_t qb[3] = {64, (uint32_t)a.G, (uint32_t)tok};
    const uint64_t kd[3] = {d, (uint64_t)a.Hkv, (uint64_t)a.B * a.Tcap}, ks[2] = {d * 2, (uint64_t)a.Hkv * d * 2};
    const uint32_t kb[3] = {64, 1, 64};
    cudaError_t e = make_tmap_3d(&mq, Q, qd, qs, qb);
    if (e == cudaSuccess) e = make_tmap_3d(&mg, dO, qd, qs, qb);
    const uint32_t rb[3] = {64, (uint32_t)a.G, (uint32_t)rtok};
    if (e == cudaSuccess) e = make_tmap_3d(&rq, Q, qd, qs, rb);
    if (e == cudaSuccess) e = make_tmap_3d(&rg, dO, qd, qs, rb);
    if (e == cudaSuccess) e = make_tmap_3d(&mk, K, kd, ks, kb);
    if (e == cudaSuccess) e = make_tmap_3d(&mv, V, kd, ks, kb);
    if (e != cudaSuccess) return e;
    const long long nq = (long long)a.B * nblk * a.Hkv, nk = (long long)a.B * (w.nkt * w.nwin + w.nst * w.nfar) * a.Hkv;
    auto go = [&](auto dq, auto dkv, int tile) {
        const size_t s1 = 1024 + (size_t)(2 + (KST + VST) / 2) * tile + sizeof(DqBars);
        const size_t s2 = 1024 + (size_t)(2 + RST) * tile + sizeof(KvBars);   // a row tile of Q and dO: one tile's bytes
        cudaError_t x = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s1);
        if (x == cudaSuccess) x = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s2);
        if (x != cudaSuccess) return x;
        dkv<<<(unsigned)(nk < 148 ? nk : 148), NTK, s2, st>>>(rq, rg, mk, mv, (__nv_bfloat16 *)dK, (__nv_bfloat16 *)dV, w,
                                                             rtok, (int)nk);
        dq<<<(unsigned)(nq < 148 ? nq : 148), NTQ, s1, st>>>(mq, mg, mk, mv, (__nv_bfloat16 *)dQ, w, tok, nblk, (int)nq);
        return cudaGetLastError();
    };
    return a.d == 64 ? go(window_dq_kernel<64>, window_dkv_kernel<64>, Cfg<64>::TILE)
                     : go(window_dq_kernel<128>, window_dkv_kernel<128>, Cfg<128>::TILE);
}

}  // namespace local
}  // namespace hsa
