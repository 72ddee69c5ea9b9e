// window_few.cu -- sliding-window attention with sinks for few query rows (at
// most 16 rows = tokens x group heads per kv head: single tokens, short drafts),
// bf16, contiguous or paged K/V.
//
// Bound: HBM (every visible K and V row is read once per kv head).  The key axis
// of a (sequence, kv head) is split over CTAs.  A producer warp streams tiles of
// 64 keys through a TMA ring; four consumer warps take 16 keys of a tile each:
// S = Q K^T and O += P V with mma.sync (16 rows fill its M; tcgen05 would pad them
// to 128), with a running maximum and sum of their own.  The warps' and then the
// CTAs' states are joined by O = sum 2^(m_i - m) O_i: within a cluster over
// distributed shared memory (one launch, no workspace), or, for more splits than a
// cluster holds, as partials that combine_kernel joins.
//
// 64 sequences of up to 16384 paged tokens, 32 + 8 heads of 128: 450 us, 5.6 TB/s (86% of
// the measured copy rate); 8 sequences, window 4096: 28.7 us, 4.7 TB/s (256 CTAs on 148 SMs:
// the SMs with two set the time).  The tcgen05 kernel, whose tiles hold 128 rows: 862 and 57 us.
#include "decode_mma.cuh"
#include "local.cuh"
#include "sm100.cuh"

namespace hsa {
namespace local {

namespace {

using namespace sm100;
using decode::ldsm_x4;
using decode::ldsm_x4_t;
using decode::mma16816;
using decode::pack_bf16;
using decode::swz;

constexpr int BK = 64;           // keys per tile
constexpr int NW = 4;            // consumer warps, 16 keys of a tile each
constexpr int NT = 32 * (NW + 1);
constexpr int NST = 3;           // ring stages of K and V
constexpr int ROWS = 16;

template <int D> struct Shape {
    static constexpr int NBX = D / 64, BOX = BK * 128, STAGE = 2 * NBX * BOX;
};

struct __align__(8) FewBars {
    uint64_t full[NST], empty[NST];
    int abort;
    float m[NW + 1][ROWS], l[NW + 1][ROWS];   // last: the CTA's
};

// The visible keys in tiles: sinks from 0, then the window from its first key
// (paged: from that key's page).
struct KeyTiles {
    int lo, hi, ns, send, base, nst, nt;
    __device__ __forceinline__ int start(int i) const { return i < nst ? i * BK : base + (i - nst) * BK; }
    __device__ __forceinline__ int end(int i) const { return min(start(i) + BK, i < nst ? send : hi); }
};

__device__ __forceinline__ KeyTiles key_tiles(int pa, int pb, int kv, int window, int sinks, int align) {
    KeyTiles t;
    t.hi = max(0, min(pb + 1, kv));
    t.lo = min(pa >= window ? pa - window + 1 : 0, t.hi);
    t.ns = min(sinks, t.lo);
    t.base = t.lo & ~(align - 1);
    t.send = min(t.ns, t.base);
    if (t.hi == t.lo) t.base = t.hi, t.send = t.ns;
    t.nst = (t.send + BK - 1) / BK;
    t.nt = t.nst + (t.hi - t.base + BK - 1) / BK;
    return t;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// fp32 at the same shared-memory offset in CTA `rank` of the cluster
__device__ __forceinline__ float4 peer_ld4(uint32_t addr, uint32_t rank) {
    uint32_t p;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ float peer_ld(uint32_t addr, uint32_t rank) {
    uint32_t p;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
    return v;
}

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(NT) window_few_kernel(const __grid_constant__ CUtensorMap tmK,
                                                        const __grid_constant__ CUtensorMap tmV,
                                                        const __nv_bfloat16 *__restrict__ Q,
                                                        __nv_bfloat16 *__restrict__ O,
                                                        const __grid_constant__ LocArgs a) {
    typedef Shape<D> C;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    FewBars *bar = reinterpret_cast<FewBars *>(ring + NST * C::STAGE);
    float *sO = reinterpret_cast<float *>(ring);   // after the last tile: [NW][ROWS][D] partial sums
    volatile int *abort = &bar->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    const Seq s = seq_of(a, b);
    const int rows = s.n * a.G;
    if (rows == 0) return;   // the whole cluster returns
    const KeyTiles tl =
        key_tiles(s.pos0, s.pos0 + s.n - 1, s.kv, a.window, a.sinks, a.paged ? 1 << a.page_shift : 1);
    int i0, i1;
    split_range(tl.nt, a.nsplit, split, &i0, &i1);
    if (threadIdx.x == 0) {
        for (int x = 0; x < NST; ++x) {
            mbar_init(&bar->full[x], 1);
            mbar_init(&bar->empty[x], NW);
        }
        bar->abort = 0;
        fence_mbar_init();
    }
    __syncthreads();

    const int psize = a.paged ? min(BK, 1 << a.page_shift) : BK;   // rows per box
    const int g0 = lane >> 2, g1 = g0 + 8, q2 = 2 * (lane & 3);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;

    int issued = 0;   // producer: tiles whose loads are under way or have landed
    if (warp == NW) {
        // ---------------------------------------------------------------- producer
        for (int i = i0; i < i1; ++i) {
            const int n = i - i0, st = n % NST;
            const int u0 = tl.start(i), nbox = (tl.end(i) - u0 + psize - 1) / psize;
            int row = 0x7fffff00;   // a bad page is read past the end, as zeros
            if (lane < nbox) {
                const long long x = kv_row(a, b, u0 + lane * psize);
                if (x >= 0) row = (int)x;
            }
            if (n >= NST && !mbar_wait(&bar->empty[st], (n / NST - 1) & 1, abort, a.status)) break;
            ++issued;
            if (lane == 0) mbar_expect_tx(&bar->full[st], (uint32_t)(nbox * psize) * 128u * 2 * C::NBX);
            __syncwarp();
            if (lane < nbox) {
                uint8_t *dst = ring + st * C::STAGE + lane * psize * 128;
                for (int x = 0; x < C::NBX; ++x) {
                    tma_load_3d(dst + x * C::BOX, &tmK, 64 * x, j, row, &bar->full[st]);
                    tma_load_3d(dst + (C::NBX + x) * C::BOX, &tmV, 64 * x, j, row, &bar->full[st]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- consumers
        uint32_t qa[D / 16][4];
        const __nv_bfloat16 *q0 = nullptr, *q1 = nullptr;
        if (g0 < rows) q0 = Q + ((long long)(s.row0 + g0 / a.G) * a.H + j * a.G + g0 % a.G) * D;
        if (g1 < rows) q1 = Q + ((long long)(s.row0 + g1 / a.G) * a.H + j * a.G + g1 % a.G) * D;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int k0 = 16 * ks + q2;
            qa[ks][0] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + k0) : 0u;
            qa[ks][1] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + k0) : 0u;
            qa[ks][2] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + k0 + 8) : 0u;
            qa[ks][3] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + k0 + 8) : 0u;
        }
        const int p0 = g0 < rows ? s.pos0 + g0 / a.G : -1, p1 = g1 < rows ? s.pos0 + g1 / a.G : -1;
        const int mi = lane >> 3, r8 = lane & 7;   // ldmatrix: this lane addresses row r8 of matrix mi
        const int kw = 16 * warp;                  // this warp's keys of the tile
        for (int i = i0; i < i1; ++i) {
            const int n = i - i0, st = n % NST, u0 = tl.start(i), ue = tl.end(i);
            if (!mbar_wait(&bar->full[st], (n / NST) & 1, abort, a.status)) break;
            if (u0 + kw < ue) {
                const uint32_t sK = smem_u32(ring + st * C::STAGE), sV = sK + C::NBX * C::BOX;
                float sc[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) sc[x][0] = sc[x][1] = sc[x][2] = sc[x][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(swz(sK + (ks / 4) * C::BOX, kw + 8 * (mi >> 1) + r8, 2 * (ks % 4) + (mi & 1)), b0, b1, b2, b3);
                    mma16816(sc[0], qa[ks], b0, b1);
                    mma16816(sc[1], qa[ks], b2, b3);
                }
                // keys that no row sees (the tile's ragged ends): their V rows must not meet a product
                const int ua = u0 + kw;
                const bool edge = ua + 16 > ue || (ua < tl.lo && ua + 16 > tl.ns);
                if (edge) {
                    for (int x = lane; x < 16 * 8 * C::NBX; x += 32) {
                        const int r = x >> 3 & 15, u = ua + r;
                        if (!(u < ue && (u >= tl.lo || u < tl.ns)))
                            *reinterpret_cast<uint4 *>(ring + st * C::STAGE + (C::NBX + (x >> 7)) * C::BOX + (kw + r) * 128 +
                                                       (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int u = ua + 8 * x + q2 + c;
                        const bool in = u < ue;
                        sc[x][c] = in && visible(p0, u, s.kv, a.window, a.sinks) ? sc[x][c] * a.scale_log2 : -INFINITY;
                        sc[x][2 + c] = in && visible(p1, u, s.kv, a.window, a.sinks) ? sc[x][2 + c] * a.scale_log2 : -INFINITY;
                        t0 = fmaxf(t0, sc[x][c]);
                        t1 = fmaxf(t1, sc[x][2 + c]);
                    }
                t0 = fmaxf(t0, __shfl_xor_sync(FULL, t0, 1));
                t0 = fmaxf(t0, __shfl_xor_sync(FULL, t0, 2));
                t1 = fmaxf(t1, __shfl_xor_sync(FULL, t1, 1));
                t1 = fmaxf(t1, __shfl_xor_sync(FULL, t1, 2));
                t0 = fmaxf(t0, m0);
                t1 = fmaxf(t1, m1);
                if (__any_sync(FULL, t0 > m0 || t1 > m1)) {
                    const float f0 = t0 > m0 ? exp2f(m0 - t0) : 1.f, f1 = t1 > m1 ? exp2f(m1 - t1) : 1.f;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        o[x][0] *= f0;
                        o[x][1] *= f0;
                        o[x][2] *= f1;
                        o[x][3] *= f1;
                    }
                    m0 = t0;
                    m1 = t1;
                }
                const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    sc[x][0] = exp2f(sc[x][0] - r0);
                    sc[x][1] = exp2f(sc[x][1] - r0);
                    sc[x][2] = exp2f(sc[x][2] - r1);
                    sc[x][3] = exp2f(sc[x][3] - r1);
                    l0 += sc[x][0] + sc[x][1];
                    l1 += sc[x][2] + sc[x][3];
                }
                // the tensor cores take P as bf16
                const uint32_t pa[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                                        pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
#pragma unroll
                for (int pp = 0; pp < D / 16; ++pp) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_t(swz(sV + (pp / 4) * C::BOX, kw + 8 * (mi & 1) + r8, 2 * (pp % 4) + (mi >> 1)), b0, b1, b2, b3);
                    mma16816(o[2 * pp], pa, b0, b1);
                    mma16816(o[2 * pp + 1], pa, b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->empty[st]);
        }
        l0 += __shfl_xor_sync(FULL, l0, 1);
        l0 += __shfl_xor_sync(FULL, l0, 2);
        l1 += __shfl_xor_sync(FULL, l1, 1);
        l1 += __shfl_xor_sync(FULL, l1, 2);
    }
    __syncthreads();
    if (*abort) {   // loads may still be in flight into the ring: leave it alone until they have landed
        if (warp == NW)
            for (int x = 0; x < NST && x < issued; ++x) mbar_drain(&bar->full[x], ((issued - 1 - x) / NST) & 1);
    } else if (warp < NW) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
            *reinterpret_cast<float2 *>(sO + (warp * ROWS + g0) * D + 8 * x + q2) = make_float2(o[x][0], o[x][1]);
            *reinterpret_cast<float2 *>(sO + (warp * ROWS + g1) * D + 8 * x + q2) = make_float2(o[x][2], o[x][3]);
        }
        if ((lane & 3) == 0) {
            bar->m[warp][g0] = m0;
            bar->m[warp][g1] = m1;
            bar->l[warp][g0] = l0;
            bar->l[warp][g1] = l1;
        }
    }
    __syncthreads();
    // the CTA's state: sum over its warps, into warp 0's rows
    for (int e = threadIdx.x; e < rows * (D / 4); e += NT) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, bar->m[w][r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        if (mx != -INFINITY) {
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = exp2f(bar->m[w][r] - mx);
                const float4 x = *reinterpret_cast<const float4 *>(sO + (w * ROWS + r) * D + c);
                l = fmaf(f, bar->l[w][r], l);
                v.x = fmaf(f, x.x, v.x);
                v.y = fmaf(f, x.y, v.y);
                v.z = fmaf(f, x.z, v.z);
                v.w = fmaf(f, x.w, v.w);
            }
        }
        *reinterpret_cast<float4 *>(sO + r * D + c) = v;
        if (c == 0) {
            bar->m[NW][r] = mx;
            bar->l[NW][r] = l;
        }
    }
    if constexpr (CLUSTER) cluster_sync();
    else __syncthreads();
    const int share = CLUSTER ? (int)cluster_rank() : 0, shares = CLUSTER ? a.nsplit : 1;
    const uint32_t so = smem_u32(sO), sm = smem_u32(bar->m[NW]), sl = smem_u32(bar->l[NW]);
    for (int e = share * NT + threadIdx.x; e < rows * (D / 4); e += NT * shares) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float mx, l;
        float4 v;
        if constexpr (CLUSTER) {
            float ms[8], ls[8];
            float4 x[8];
            mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < a.nsplit) {
                    ms[k] = peer_ld(sm + r * 4, k);
                    ls[k] = peer_ld(sl + r * 4, k);
                    x[k] = peer_ld4(so + (r * D + c) * 4, k);
                    mx = fmaxf(mx, ms[k]);
                }
            v = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < a.nsplit && mx != -INFINITY) {
                    const float f = exp2f(ms[k] - mx);
                    l = fmaf(f, ls[k], l);
                    v.x = fmaf(f, x[k].x, v.x);
                    v.y = fmaf(f, x[k].y, v.y);
                    v.z = fmaf(f, x[k].z, v.z);
                    v.w = fmaf(f, x[k].w, v.w);
                }
        } else {
            mx = bar->m[NW][r];
            l = bar->l[NW][r];
            v = *reinterpret_cast<const float4 *>(sO + r * D + c);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse = l > 0.f ? mx * 0.6931471805599453f + logf(l) : -INFINITY;
        const long long row = (long long)(s.row0 + r / a.G) * a.H + j * a.G + r % a.G;
        if (!CLUSTER && a.nsplit > 1) {
            const long long prow = part_row(a, split, b, r / a.G) + j * a.G + r % a.G;
            *reinterpret_cast<float4 *>(a.opart + prow * D + c) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            if (c == 0) a.lpart[prow] = lse;
        } else {
            *reinterpret_cast<uint2 *>(O + row * D + c) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (c == 0 && a.lse) a.lse[row] = lse;
        }
    }
    if constexpr (CLUSTER) cluster_sync();   // peers may still read this CTA's shared memory
}

// D of the query rows that see few keys, for the backward: D = sum_u P[u] dP[u], P = exp(scale S - lse), dP = dO . V[u],
// in fp32.  dO . O is the same in exact arithmetic, but the bf16 O is off by up to 2^-8 of itself, and over n equal keys that
// part of dQ and dK is about 1 / sqrt(n) of the one that rounding dS leaves: as large with one key, nothing with many.
// A warp takes 16 rows (token, head of the group), keys in eights; 16-byte chunks go straight to the fragments (the
// contraction runs over the elements in any order that both operands share).
//
// DOT_KEYS: the gradients' error against 64 bits with 64 keys or fewer was up to 1.6 times that of rounding the exact
// result once, and is 1.4 times with this kernel (rounding dS and the result).  2 x 4096 tokens, 32 + 8 heads of 128:
// the whole backward takes 232 us with a window of 64, 199 with one of 65 (which leaves the kernel 64 tokens), 182
// with 16.
constexpr int DOT_KEYS = 64;

__device__ __forceinline__ int keys_seen(const LocArgs &a, int p) {
    const int hi = min(p + 1, a.max_kv), lo = min(p >= a.window ? p - a.window + 1 : 0, hi);
    return hi - lo + min(a.sinks, lo);
}

template <int D>
__global__ void __launch_bounds__(128) few_rowdot_kernel(LocArgs a, const __nv_bfloat16 *__restrict__ Q,
                                                         const __nv_bfloat16 *__restrict__ K,
                                                         const __nv_bfloat16 *__restrict__ V,
                                                         const __nv_bfloat16 *__restrict__ dO, float *__restrict__ out,
                                                         int ntok) {
    constexpr int C = D / 32;   // 16-byte chunks of a row per lane
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, j = blockIdx.y, b = blockIdx.z;
    const long long n = (long long)ntok * a.G, e0 = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * 16;
    if (e0 >= n) return;
    int pos[2];
    long long row[2];
    float nl[2];
    uint4 q[2][C], d[2][C];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const long long e = min(e0 + g + 8 * x, n - 1);   // rows behind the last repeat it
        const int t = (int)(e / a.G);
        pos[x] = a.q_pos0 + t;
        row[x] = ((long long)b * a.max_q + t) * a.H + j * a.G + (int)(e % a.G);
    }
    if (!__any_sync(FULL, min(keys_seen(a, pos[0]), keys_seen(a, pos[1])) <= DOT_KEYS)) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        nl[x] = a.lse[row[x]] * -1.4426950408889634f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            q[x][i] = reinterpret_cast<const uint4 *>(Q + row[x] * D)[c + 4 * i];
            d[x][i] = reinterpret_cast<const uint4 *>(dO + row[x] * D)[c + 4 * i];
        }
    }
    const int pa = a.q_pos0 + (int)(e0 / a.G), pb = a.q_pos0 + (int)(min(e0 + 15, n - 1) / a.G);
    const int hi = min(pb + 1, a.max_kv), lo = min(pa >= a.window ? pa - a.window + 1 : 0, hi);
    float sum[2] = {0.f, 0.f};
    for (int part = 0; part < 2; ++part) {   // sinks before the window, then the window
        const int ua = part ? lo : 0, ub = part ? hi : min(a.sinks, lo);
        for (int u0 = ua; u0 < ub; u0 += 8) {
            const long long at = ((kv_row(a, b, min(u0 + g, ub - 1))) * a.Hkv + j) * D;
            uint4 k[C], v[C];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                k[i] = reinterpret_cast<const uint4 *>(K + at)[c + 4 * i];
                v[i] = reinterpret_cast<const uint4 *>(V + at)[c + 4 * i];
            }
            float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C; ++i) {
                mma16816(s, q[0][i].x, q[1][i].x, q[0][i].y, q[1][i].y, k[i].x, k[i].y);
                mma16816(dp, d[0][i].x, d[1][i].x, d[0][i].y, d[1][i].y, v[i].x, v[i].y);
                mma16816(s, q[0][i].z, q[1][i].z, q[0][i].w, q[1][i].w, k[i].z, k[i].w);
                mma16816(dp, d[0][i].z, d[1][i].z, d[0][i].w, d[1][i].w, v[i].z, v[i].w);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int x = y >> 1, u = u0 + 2 * c + (y & 1);
                const float pr = exp2f(fmaf(s[y], a.scale_log2, nl[x])) * dp[y];
                // selected, not multiplied: keys that a row does not see may hold NaN
                sum[x] += u < ub && visible(pos[x], u, a.max_kv, a.window, a.sinks) ? pr : 0.f;
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        sum[x] += __shfl_xor_sync(FULL, sum[x], 1);
        sum[x] += __shfl_xor_sync(FULL, sum[x], 2);
        if (c == 0 && e0 + g + 8 * x < n) out[row[x]] = sum[x];
    }
}

}  // namespace

bool few_supported(const LocArgs &a, int dtype) {
    return dtype == HSA_BF16 && a.max_kv > 0 && a.max_q > 0 && (long long)a.max_q * a.G <= ROWS;
}

cudaError_t launch_few(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t d = a.d;
    const uint64_t kvrows = a.paged ? (uint64_t)a.npages << a.page_shift : (uint64_t)a.B * a.Tcap;
    const uint64_t kd[3] = {d, (uint64_t)a.Hkv, kvrows}, ks[2] = {d * 2, (uint64_t)a.Hkv * d * 2};
    const uint32_t kb[3] = {64, 1, a.paged && a.page_shift < 6 ? 1u << a.page_shift : (uint32_t)BK};
    cudaError_t e = make_tmap_3d(&mk, K, kd, ks, kb);
    if (e == cudaSuccess) e = make_tmap_3d(&mv, V, kd, ks, kb);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kern, int stage, bool cluster) {
        const size_t smem = 1024 + (size_t)NST * stage + sizeof(FewBars);
        cudaError_t x = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (x != cudaSuccess) return x;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.nsplit, a.Hkv, a.B);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = a.nsplit;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = cluster ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, kern, mk, mv, (const __nv_bfloat16 *)Q, (__nv_bfloat16 *)O, a);
    };
    const bool cluster = a.nsplit > 1 && a.nsplit <= FEW_CLUSTER;
    if (a.d == 64)
        return cluster ? go(window_few_kernel<64, true>, Shape<64>::STAGE, true)
                       : go(window_few_kernel<64, false>, Shape<64>::STAGE, false);
    return cluster ? go(window_few_kernel<128, true>, Shape<128>::STAGE, true)
                   : go(window_few_kernel<128, false>, Shape<128>::STAGE, false);
}

bool few_rowdot_all(const LocArgs &a) {
    return a.max_kv > 0 && a.window <= DOT_KEYS && a.sinks <= DOT_KEYS - a.window;
}

cudaError_t launch_few_rowdot(const LocArgs &a, const void *Q, const void *K, const void *V, const void *dO, float *D,
                              cudaStream_t st) {
    // all tokens with a window of few keys, or where queries run past the keys; else the first ones
    const bool all = a.window <= DOT_KEYS || (long long)a.q_pos0 + a.max_q > a.max_kv;
    const int ntok = all ? a.max_q : max(0, min(a.max_q, DOT_KEYS - a.q_pos0));
    if (ntok == 0 || a.max_kv == 0) return cudaSuccess;
    typedef __nv_bfloat16 h;
    const dim3 grid((unsigned)(((long long)ntok * a.G + 63) / 64), a.Hkv, a.B);
    if (a.d == 64)
        few_rowdot_kernel<64><<<grid, 128, 0, st>>>(a, (const h *)Q, (const h *)K, (const h *)V, (const h *)dO, D, ntok);
    else
        few_rowdot_kernel<128><<<grid, 128, 0, st>>>(a, (const h *)Q, (const h *)K, (const h *)V, (const h *)dO, D, ntok);
    return cudaGetLastError();
}

}  // namespace local
}  // namespace hsa
