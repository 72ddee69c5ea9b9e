// window_simt.cu -- sliding-window attention with sinks on the CUDA cores, in
// fp32 throughout: the fp32 problems' kernels, and the ones HSA_FLAG_SIMT asks
// for.  Contiguous or paged K/V.  Also the pieces every path shares: the join
// of key-axis splits, the row sums D of the backward, and the join of the
// backward's partials.
//
// 64 x 64 tiles, 4 x 4 elements a thread (16 or 32 rows where there are few).  Bound:
// latency at small sizes (2 x 777 tokens, 4 heads of 64, window 129: forward 34 us, dQ
// 42 us, dK and dV 59 us on 100 to 200 blocks of two warps per SM sub-partition, which
// wait for shared memory), shared memory at large ones (bf16 inputs, 65536 tokens,
// window 4096, 32 heads of 128: 28 TFLOP/s).
#include "local.cuh"
#include "local_sm100.cuh"

namespace hsa {
namespace local {

namespace {

constexpr int BM = 64;   // rows (token, head) per row tile of dK, dV
constexpr int BN = 64;   // keys per tile
constexpr int NT = 256;  // 16 x 16 threads: RM rows x 4 keys of S each
constexpr int PP = BN + 4;

// R rows of a tensor into shared memory as fp32 (pitch P); row r is read at src(r), or
// zero where that is negative.
template <typename T, int D, int P, int R = 64, typename Src>
__device__ __forceinline__ void load_rows(float *dst, const T *__restrict__ g, Src src) {
    constexpr int V = 16 / sizeof(T);    // elements per 16-byte load
    constexpr int PR = D / V;            // loads per row
    constexpr int N = (R * PR + NT - 1) / NT;
    uint4 u[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {        // all of a thread's loads at once
        const int i = threadIdx.x + n * NT;
        u[n] = make_uint4(0, 0, 0, 0);
        if (i < R * PR) {
            const long long at = src(i / PR);
            if (at >= 0) u[n] = *reinterpret_cast<const uint4 *>(g + at + i % PR * V);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + n * NT;
        if (i >= R * PR) continue;
        const T *t = reinterpret_cast<const T *>(&u[n]);
        float *d = dst + i / PR * P + i % PR * V;
#pragma unroll
        for (int x = 0; x < V; x += 4)
            *reinterpret_cast<float4 *>(d + x) =
                make_float4(to_f32(t[x]), to_f32(t[x + 1]), to_f32(t[x + 2]), to_f32(t[x + 3]));
    }
}

// Packed fp32 pairs (one instruction does two multiply-adds): these loops are bound by issue.
__device__ __forceinline__ ulonglong2 ld_pairs(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }

// s[i][j] = row (ty*RM + i) of A . row (tx + 16 j) of B, over D; even and odd elements are summed apart
template <int D, int PA, int PB, int RM = 4>
__device__ __forceinline__ void dot_tile(const float *A, const float *B, int ty, int tx, float (&s)[RM][4]) {
    uint64_t t[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) t[i][j] = 0;
#pragma unroll 8
    for (int x = 0; x < D; x += 4) {
        ulonglong2 a[RM], b[4];
#pragma unroll
        for (int i = 0; i < RM; ++i) a[i] = ld_pairs(A + (ty * RM + i) * PA + x);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = ld_pairs(B + (tx + 16 * j) * PB + x);
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) t[i][j] = sm100::fma2(a[i].y, b[j].y, sm100::fma2(a[i].x, b[j].x, t[i][j]));
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            sm100::unpair(t[i][j], lo, hi);
            s[i][j] = lo + hi;
        }
}

// acc[i][c] += sum_k P[row ty*RM + i][k] X[k][col]; acc's pair c: columns tx*4 + 64*(c/2) + 2*(c%2), and the next.
// PT: P is stored [k][row] instead (transposed product; RM = 4).
template <int D, int PX, bool PT, int RM = 4>
__device__ __forceinline__ void acc_tile(const float *Pm, const float *X, int ty, int tx, uint64_t (&acc)[RM][D / 32]) {
#pragma unroll 8
    for (int k = 0; k < 64; ++k) {
        float p[RM];
        if constexpr (PT) {
            const float4 v = *reinterpret_cast<const float4 *>(Pm + k * PP + ty * 4);
            p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < RM; ++i) p[i] = Pm[(ty * RM + i) * PP + k];
        }
        uint64_t pp[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) pp[i] = sm100::pair(p[i], p[i]);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const ulonglong2 v = ld_pairs(X + k * PX + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                acc[i][2 * c] = sm100::fma2(pp[i], v.x, acc[i][2 * c]);
                acc[i][2 * c + 1] = sm100::fma2(pp[i], v.y, acc[i][2 * c + 1]);
            }
        }
    }
}

template <typename T> __device__ __forceinline__ void store4(T *p, float a, float b, float c, float d);
template <> __device__ __forceinline__ void store4<float>(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float a, float b, float c, float d) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t *>(&lo);
    u.y = *reinterpret_cast<uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(p) = u;
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, o));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
    return x;
}

// Forward: one pass over the block's key tiles with a running maximum m and
// sum l per row; O is rescaled by exp(m_old - m_new) when the maximum grows.
template <typename T, int D, int RM>
__global__ void __launch_bounds__(NT) simt_fwd_kernel(LocArgs a, const T *__restrict__ Q, const T *__restrict__ K,
                                                      const T *__restrict__ V, T *__restrict__ O) {
    extern __shared__ __align__(16) float sm[];
    constexpr int BM = 16 * RM;   // rows (token, head) of this block
    float *sQ = sm, *sK = sQ + BM * D, *sV = sK + BN * (D + 4), *sP = sV + BN * D;
    const int j = blockIdx.y;
    const int split = blockIdx.x % a.nsplit;
    const int tok = BM / a.G;                       // tokens per block
    int b = blockIdx.z, blk = blockIdx.x / a.nsplit;
    if (a.by_rows && !tile_by_row(a, blk, tok, &b, &blk)) return;
    const Seq s = seq_of(a, b);
    const int t0 = blk * tok, t1 = min(s.n, t0 + tok);
    if (t0 >= s.n) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Tiles tl = tiles_of<BN>(s.pos0 + t0, s.pos0 + t1 - 1, s.kv, a.window, a.sinks);
    int i0, i1;
    split_range(tl.nt, a.nsplit, split, &i0, &i1);

    load_rows<T, D, D, BM>(sQ, Q, [&](int r) -> long long {
        const int t = t0 + r / a.G;
        return r < tok * a.G && t < t1 ? ((long long)(s.row0 + t) * a.H + j * a.G + r % a.G) * D : -1;
    });
    float m[RM], l[RM];
    uint64_t o[RM][D / 32];   // pairs of columns
    int p[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = ty * RM + i;
        m[i] = -INFINITY;
        l[i] = 0.f;
        p[i] = r < tok * a.G && t0 + r / a.G < t1 ? s.pos0 + t0 + r / a.G : -1;   // -1: sees nothing
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[i][c] = 0;
    }
    for (int it = i0; it < i1; ++it) {
        const int u0 = tl.tile(it) * BN;
        __syncthreads();
        auto src = [&](int r) -> long long {
            if (!key_live(tl, u0 + r)) return -1;
            const long long row = kv_row(a, b, u0 + r);
            return row < 0 ? -1 : (row * a.Hkv + j) * D;
        };
        load_rows<T, D, D + 4>(sK, K, src);
        load_rows<T, D, D>(sV, V, src);
        __syncthreads();
        float sc[RM][4];
        dot_tile<D, D, D + 4, RM>(sQ, sK, ty, tx, sc);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int u = u0 + tx + 16 * c;
                sc[i][c] = visible(p[i], u, s.kv, a.window, a.sinks) ? sc[i][c] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, sc[i][c]);
            }
            mx = fmaxf(m[i], max16(mx));
            const float ref = mx == -INFINITY ? 0.f : mx;   // rows without a key so far: every exp is 0
            const float f = exp2f(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = exp2f(sc[i][c] - ref);
                sum += e;
                sP[(ty * RM + i) * PP + tx + 16 * c] = e;
            }
            l[i] = l[i] * f + sum16(sum);
            m[i] = mx;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[i][c] = sm100::fma2(o[i][c], sm100::pair(f, f), 0);
        }
        __syncwarp();   // a warp reads only the P rows that it wrote
        acc_tile<D, D, false, RM>(sP, sV, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int r = ty * RM + i;
        if (r >= tok * a.G || t0 + r / a.G >= t1) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const float lse = l[i] > 0.f ? m[i] * 0.6931471805599453f + logf(l[i]) : -INFINITY;
        const long long row = (long long)(s.row0 + t0 + r / a.G) * a.H + j * a.G + r % a.G;
        const long long prow = part_row(a, split, b, t0 + r / a.G) + j * a.G + r % a.G;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float x, y, z, w;
            sm100::unpair(o[i][2 * c], x, y);
            sm100::unpair(o[i][2 * c + 1], z, w);
            x *= inv, y *= inv, z *= inv, w *= inv;
            if (a.nsplit > 1)
                store4<float>(a.opart + prow * D + tx * 4 + 64 * c, x, y, z, w);
            else
                store4<T>(O + row * D + tx * 4 + 64 * c, x, y, z, w);
        }
        if (tx == 0) {
            if (a.nsplit > 1)
                a.lpart[prow] = lse;
            else if (a.lse)
                a.lse[row] = lse;
        }
    }
}

// Joins the key-axis splits of a row: O = sum_s exp(lse_s - lse) O_s with
// lse = ln sum_s exp(lse_s), in split order.  One warp per (token, head).
// Only the rows of the call's sequences were written; the others are left alone.
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_kernel(LocArgs a, T *__restrict__ O) {
    const int b = blockIdx.y;
    const Seq s = seq_of(a, b);
    const int lane = threadIdx.x & 31;
    const long long e = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (e >= (long long)s.n * a.H) return;
    const long long row = (long long)s.row0 * a.H + e;
    const long long prow = part_row(a, 0, b, 0) + e, stride = part_row(a, 1, 0, 0);
    float mx = -INFINITY;
    for (int i = lane; i < a.nsplit; i += 32) mx = fmaxf(mx, a.lpart[i * stride + prow]);
    mx = warp_max(mx);
    constexpr int N = D / 32;
    float acc[N], l = 0.f;
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] = 0.f;
    if (mx != -INFINITY) {
        for (int i = 0; i < a.nsplit; ++i) {
            const float w = expf(a.lpart[i * stride + prow] - mx);
            l += w;
            const float *src = a.opart + (i * stride + prow) * D + lane * N;
#pragma unroll
            for (int x = 0; x < N; ++x) acc[x] = fmaf(w, src[x], acc[x]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int x = 0; x < N; ++x) O[row * D + lane * N + x] = from_f32<T>(acc[x] * inv);
    if (lane == 0 && a.lse) a.lse[row] = l > 0.f ? mx + logf(l) : -INFINITY;
}

// D[row] = sum_x dO[row][x] O[row][x]: 16-byte loads, the lanes of a row side by side, four rows in flight per lane.
template <typename T, int D>
__global__ void __launch_bounds__(256) rowdot_kernel(const T *__restrict__ O, const T *__restrict__ dO,
                                                     float *__restrict__ out, long long n) {
    constexpr int V = 16 / sizeof(T), LPR = D / V, RPW = 32 / LPR, U = 4;   // lanes per row, rows per warp and load
    const int lane = threadIdx.x & 31;
    const long long r0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW * U + lane / LPR;
    uint4 o[U], g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long r = r0 + u * RPW;
        if (r < n) {
            o[u] = reinterpret_cast<const uint4 *>(O + r * D)[lane % LPR];
            g[u] = reinterpret_cast<const uint4 *>(dO + r * D)[lane % LPR];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long r = r0 + u * RPW;
        float s = 0.f;
        if (r < n) {
            const T *x = reinterpret_cast<const T *>(&o[u]), *y = reinterpret_cast<const T *>(&g[u]);
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(to_f32(x[e]), to_f32(y[e]), s);
        }
#pragma unroll
        for (int w = LPR / 2; w > 0; w >>= 1) s += __shfl_xor_sync(FULL, s, w);
        if (r < n && lane % LPR == 0) out[r] = s;
    }
}

// dQ: the forward's iteration; P from lse, dP = dO V^T, dS = P (dP - D), dQ += dS K.
template <typename T, int D, int RM>
__global__ void __launch_bounds__(NT) simt_dq_kernel(BwdArgs w, const T *__restrict__ Q, const T *__restrict__ K,
                                                     const T *__restrict__ V, const T *__restrict__ dO,
                                                     T *__restrict__ dQ) {
    extern __shared__ __align__(16) float sm[];
    const LocArgs &a = w.a;
    constexpr int BM = 16 * RM;
    float *sQ = sm, *sG = sQ + BM * D, *sK = sG + BM * D, *sV = sK + BN * (D + 4), *sP = sV + BN * (D + 4);
    const int b = blockIdx.z, j = blockIdx.y;
    const int tok = BM / a.G;
    const Seq s = seq_of(a, b);
    const int t0 = blockIdx.x * tok, t1 = min(s.n, t0 + tok);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Tiles tl = tiles_of<BN>(s.pos0 + t0, s.pos0 + t1 - 1, s.kv, a.window, a.sinks);
    auto qsrc = [&](int r) -> long long {
        const int t = t0 + r / a.G;
        return r < tok * a.G && t < t1 ? ((long long)(s.row0 + t) * a.H + j * a.G + r % a.G) * D : -1;
    };
    load_rows<T, D, D, BM>(sQ, Q, qsrc);
    load_rows<T, D, D, BM>(sG, dO, qsrc);
    float lse2[RM], dd[RM];
    uint64_t acc[RM][D / 32];
    int p[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const long long at = qsrc(ty * RM + i);
        p[i] = at >= 0 ? s.pos0 + t0 + (ty * RM + i) / a.G : -1;
        lse2[i] = at >= 0 ? a.lse[at / D] * 1.4426950408889634f : 0.f;
        dd[i] = at >= 0 ? w.D[at / D] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = 0;
    }
    for (int it = 0; it < tl.nt; ++it) {
        const int u0 = tl.tile(it) * BN;
        __syncthreads();
        auto src = [&](int r) -> long long {
            return key_live(tl, u0 + r) ? (kv_row(a, b, u0 + r) * a.Hkv + j) * D : -1;
        };
        load_rows<T, D, D + 4>(sK, K, src);
        load_rows<T, D, D + 4>(sV, V, src);
        __syncthreads();
        float sc[RM][4], dp[RM][4];
        dot_tile<D, D, D + 4, RM>(sQ, sK, ty, tx, sc);
        dot_tile<D, D, D + 4, RM>(sG, sV, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool vis = visible(p[i], u0 + tx + 16 * c, s.kv, a.window, a.sinks);
                const float pr = vis ? exp2f(fmaf(sc[i][c], a.scale_log2, -lse2[i])) : 0.f;
                sP[(ty * RM + i) * PP + tx + 16 * c] = vis ? pr * (dp[i][c] - dd[i]) : 0.f;
            }
        __syncwarp();
        acc_tile<D, D + 4, false, RM>(sP, sK, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const long long at = qsrc(ty * RM + i);
        if (at < 0) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float x, y, z, v;
            sm100::unpair(acc[i][2 * c], x, y);
            sm100::unpair(acc[i][2 * c + 1], z, v);
            store4<T>(dQ + at + tx * 4 + 64 * c, x * a.scale, y * a.scale, z * a.scale, v * a.scale);
        }
    }
}

// dK, dV of one key tile: over the rows of every query token that sees it.
// Work item x: see kv_range.
template <typename T, int D>
__global__ void __launch_bounds__(NT) simt_dkv_kernel(BwdArgs w, const T *__restrict__ Q, const T *__restrict__ K,
                                                      const T *__restrict__ V, const T *__restrict__ dO,
                                                      T *__restrict__ dK, T *__restrict__ dV) {
    extern __shared__ __align__(16) float sm[];
    const LocArgs &a = w.a;
    float *sK = sm, *sV = sK + BN * (D + 4), *sQ = sV + BN * (D + 4), *sG = sQ + BM * (D + 4),
          *sP = sG + BM * (D + 4), *sS = sP + BM * PP;
    const int b = blockIdx.z, j = blockIdx.y;
    const Seq s = seq_of(a, b);
    const KvRange it = kv_range(w, s, blockIdx.x, BN);
    const int u0 = it.kt * BN, ta = it.ta, tb = it.tb;
    const bool part = it.kt < w.npt;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    auto src = [&](int r) -> long long {
        return u0 + r < s.kv ? (kv_row(a, b, u0 + r) * a.Hkv + j) * D : -1;
    };
    const int tok = BM / a.G;
    uint64_t gk[4][D / 32], gv[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) gk[i][c] = gv[i][c] = 0;
    if (ta < tb) {
        load_rows<T, D, D + 4>(sK, K, src);
        load_rows<T, D, D + 4>(sV, V, src);
    }
    for (int t0 = ta; t0 < tb; t0 += tok) {
        const int t1 = min(tb, t0 + tok);
        auto qsrc = [&](int r) -> long long {
            const int t = t0 + r / a.G;
            return r < tok * a.G && t < t1 ? ((long long)(s.row0 + t) * a.H + j * a.G + r % a.G) * D : -1;
        };
        __syncthreads();
        load_rows<T, D, D + 4>(sQ, Q, qsrc);
        load_rows<T, D, D + 4>(sG, dO, qsrc);
        __syncthreads();
        float sc[4][4], dp[4][4];
        dot_tile<D, D + 4, D + 4>(sQ, sK, ty, tx, sc);
        dot_tile<D, D + 4, D + 4>(sG, sV, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            const long long at = qsrc(r);
            const int p = at >= 0 ? s.pos0 + t0 + r / a.G : -1;
            const float lse2 = at >= 0 ? a.lse[at / D] * 1.4426950408889634f : 0.f;
            const float dd = at >= 0 ? w.D[at / D] : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool vis = visible(p, u0 + tx + 16 * c, s.kv, a.window, a.sinks);
                const float pr = vis ? exp2f(fmaf(sc[i][c], a.scale_log2, -lse2)) : 0.f;
                sP[r * PP + tx + 16 * c] = pr;
                sS[r * PP + tx + 16 * c] = vis ? pr * (dp[i][c] - dd) : 0.f;
            }
        }
        __syncthreads();
        // key rows ty*4 + i: sum over the 64 query rows of P[row][key] dO[row][:]
        acc_tile<D, D + 4, true>(sP, sG, ty, tx, gv);
        acc_tile<D, D + 4, true>(sS, sQ, ty, tx, gk);
    }
    const long long psz = (long long)a.B * a.Hkv * w.npt * BN * D;   // one slot of partials
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = u0 + ty * 4 + i;
        if (u >= s.kv) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int col = tx * 4 + 64 * c;
            float k4[4], v4[4];
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                sm100::unpair(gk[i][2 * c + x / 2], k4[x], k4[x + 1]);
                sm100::unpair(gv[i][2 * c + x / 2], v4[x], v4[x + 1]);
                k4[x] *= a.scale;
                k4[x + 1] *= a.scale;
            }
            if (part) {
                const long long at = (((long long)b * a.Hkv + j) * w.npt * BN + u) * D + col;
                float *pk = w.part + it.slot * psz + at, *pv = pk + (w.nwin + w.nfar) * psz;
                store4<float>(pk, k4[0], k4[1], k4[2], k4[3]);
                store4<float>(pv, v4[0], v4[1], v4[2], v4[3]);
            } else {
                const long long at = (((long long)b * a.Tcap + u) * a.Hkv + j) * D + col;
                store4<T>(dK + at, k4[0], k4[1], k4[2], k4[3]);
                store4<T>(dV + at, v4[0], v4[1], v4[2], v4[3]);
            }
        }
    }
}

// dK, dV of the tiles written as partials, summed in slot order (the window's chunks, then
// the far ones of sink tiles) and rounded once.  One thread per four elements.
template <typename T, int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(BwdArgs w, int bk, T *__restrict__ dK, T *__restrict__ dV) {
    const LocArgs &a = w.a;
    const long long psz = (long long)a.B * a.Hkv * w.npt * bk * D;
    const long long e = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= psz) return;
    const int u = (int)(e / D % (w.npt * bk));
    const long long bj = e / D / (w.npt * bk);
    if (u >= a.max_kv) return;
    const float *src = w.part + (blockIdx.y ? (w.nwin + w.nfar) * psz : 0) + e;
    const int slots = w.nwin + (u / bk < w.nst ? w.nfar : 0);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < slots; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(src + i * psz);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    T *dst = (blockIdx.y ? dV : dK) + ((bj / a.Hkv * a.Tcap + u) * a.Hkv + bj % a.Hkv) * D + e % D;
    store4<T>(dst, s.x, s.y, s.z, s.w);
}

template <typename F> cudaError_t with_smem(F f, size_t bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int D, int RM>
cudaError_t fwd_rows(LocArgs a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st) {
    constexpr int BM = 16 * RM;
    const size_t smem = (BM * D + BN * (D + 4) + BN * D + BM * PP) * sizeof(float);
    cudaError_t e = with_smem(simt_fwd_kernel<T, D, RM>, smem);
    if (e != cudaSuccess) return e;
    const int tok = BM / a.G;
    dim3 grid((unsigned)((a.max_q + tok - 1) / tok) * a.nsplit, a.Hkv, a.B);
    // max_q bounds the tokens of every paged sequence and may be far above most (all rows, if the caller knows no
    // better): 65535 single tokens would get 2.7e8 blocks per kv head with it, minutes of empty ones.  Beyond 2^20
    // blocks (about 5 ms of them) the tiles are numbered over the rows, a search in q_start per block.
    if (a.paged && a.nsplit == 1 && (double)grid.x * a.Hkv * a.B > 1 << 20) {
        a.by_rows = 1;
        grid = dim3((unsigned)(a.rows / tok + a.B), a.Hkv, 1);
    }
    simt_fwd_kernel<T, D, RM><<<grid, NT, smem, st>>>(a, (const T *)Q, (const T *)K, (const T *)V, (T *)O);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t fwd(const LocArgs &a, const void *Q, const void *K, const void *V, void *O, cudaStream_t st) {
    const int rows = simt_rows(a);
    return rows == 16   ? fwd_rows<T, D, 1>(a, Q, K, V, O, st)
           : rows == 32 ? fwd_rows<T, D, 2>(a, Q, K, V, O, st)
                        : fwd_rows<T, D, 4>(a, Q, K, V, O, st);
}

template <typename T, int D, int RM>
cudaError_t dq_rows(const BwdArgs &w, const void *Q, const void *K, const void *V, const void *dO, void *dQ,
                    cudaStream_t st) {
    constexpr int BM = 16 * RM;
    const size_t smem = (2 * BM * D + 2 * BN * (D + 4) + BM * PP) * sizeof(float);
    cudaError_t e = with_smem(simt_dq_kernel<T, D, RM>, smem);
    if (e != cudaSuccess) return e;
    const int tok = BM / w.a.G;
    simt_dq_kernel<T, D, RM><<<dim3((w.a.max_q + tok - 1) / tok, w.a.Hkv, w.a.B), NT, smem, st>>>(
        w, (const T *)Q, (const T *)K, (const T *)V, (const T *)dO, (T *)dQ);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const BwdArgs &w, const void *Q, const void *K, const void *V, const void *dO, void *dQ, void *dK,
                void *dV, cudaStream_t st) {
    const size_t smem = (4 * BN * (D + 4) + 2 * BM * PP) * sizeof(float);
    cudaError_t e = with_smem(simt_dkv_kernel<T, D>, smem);
    if (e == cudaSuccess && w.a.max_q > 0)
        e = simt_rows(w.a) < 64 ? dq_rows<T, D, 2>(w, Q, K, V, dO, dQ, st) : dq_rows<T, D, 4>(w, Q, K, V, dO, dQ, st);
    if (e != cudaSuccess) return e;
    if (w.nkt > 0)
        simt_dkv_kernel<T, D><<<dim3(w.nkt * w.nwin + w.nst * w.nfar, w.a.Hkv, w.a.B), NT, smem, st>>>(
            w, (const T *)Q, (const T *)K, (const T *)V, (const T *)dO, (T *)dK, (T *)dV);
    return cudaGetLastError();
}

#define BY_TYPE(call_f64, call_f128, call_b64, call_b128) \
    (dtype == HSA_F32 ? (d == 64 ? call_f64 : call_f128) : (d == 64 ? call_b64 : call_b128))

}  // namespace

int simt_rows(const LocArgs &a) {
    // few rows in all: 16; few blocks: 32, so that more SMs and more warps per SM have some (2 x 777 tokens of 4
    // heads, window 129: 34 us; 40 with 64 rows and the keys in two splits); else 64, which reads the keys half as often
    if ((long long)a.max_q * a.G <= 16) return 16;
    const int tok = 64 / a.G;
    return (long long)((a.max_q + tok - 1) / tok) * a.Hkv * a.B < 2 * 148 ? 32 : 64;
}

cudaError_t launch_simt(const LocArgs &a, int dtype, const void *Q, const void *K, const void *V, void *O,
                        cudaStream_t st) {
    const int d = a.d;
    return BY_TYPE((fwd<float, 64>(a, Q, K, V, O, st)), (fwd<float, 128>(a, Q, K, V, O, st)),
                   (fwd<__nv_bfloat16, 64>(a, Q, K, V, O, st)), (fwd<__nv_bfloat16, 128>(a, Q, K, V, O, st)));
}

cudaError_t launch_combine(const LocArgs &a, int dtype, void *O, cudaStream_t st) {
    const int d = a.d;
    const dim3 grid((unsigned)(((long long)a.max_q * a.H + 7) / 8), a.B);
    if (dtype == HSA_F32) {
        if (d == 64) combine_kernel<float, 64><<<grid, 256, 0, st>>>(a, (float *)O);
        else combine_kernel<float, 128><<<grid, 256, 0, st>>>(a, (float *)O);
    } else {
        if (d == 64) combine_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(a, (__nv_bfloat16 *)O);
        else combine_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(a, (__nv_bfloat16 *)O);
    }
    return cudaGetLastError();
}

cudaError_t launch_rowdot(const LocArgs &a, int dtype, const void *O, const void *dO, float *D, cudaStream_t st) {
    const long long n = (long long)a.rows * a.H;
    if (n == 0) return cudaSuccess;
    const int per = 8 * 4 * 32 / (a.d / (dtype == HSA_F32 ? 4 : 8));   // rows per block
    const unsigned g = (unsigned)((n + per - 1) / per);
    if (dtype == HSA_F32) {
        if (a.d == 64) rowdot_kernel<float, 64><<<g, 256, 0, st>>>((const float *)O, (const float *)dO, D, n);
        else rowdot_kernel<float, 128><<<g, 256, 0, st>>>((const float *)O, (const float *)dO, D, n);
    } else {
        typedef __nv_bfloat16 h;
        if (a.d == 64) rowdot_kernel<h, 64><<<g, 256, 0, st>>>((const h *)O, (const h *)dO, D, n);
        else rowdot_kernel<h, 128><<<g, 256, 0, st>>>((const h *)O, (const h *)dO, D, n);
    }
    return cudaGetLastError();
}

cudaError_t launch_bwd_simt(const BwdArgs &w, int dtype, const void *Q, const void *K, const void *V, const void *dO,
                            void *dQ, void *dK, void *dV, cudaStream_t st) {
    const int d = w.a.d;
    return BY_TYPE((bwd<float, 64>(w, Q, K, V, dO, dQ, dK, dV, st)), (bwd<float, 128>(w, Q, K, V, dO, dQ, dK, dV, st)),
                   (bwd<__nv_bfloat16, 64>(w, Q, K, V, dO, dQ, dK, dV, st)),
                   (bwd<__nv_bfloat16, 128>(w, Q, K, V, dO, dQ, dK, dV, st)));
}

cudaError_t launch_bwd_join(const BwdArgs &w, int bk, int dtype, void *dK, void *dV, cudaStream_t st) {
    if (w.npt == 0) return cudaSuccess;
    const long long psz = (long long)w.a.B * w.a.Hkv * w.npt * bk * w.a.d;
    const dim3 grid((unsigned)((psz / 4 + 255) / 256), 2);
    if (dtype == HSA_F32) {
        if (w.a.d == 64) bwd_join_kernel<float, 64><<<grid, 256, 0, st>>>(w, bk, (float *)dK, (float *)dV);
        else bwd_join_kernel<float, 128><<<grid, 256, 0, st>>>(w, bk, (float *)dK, (float *)dV);
    } else {
        typedef __nv_bfloat16 h;
        if (w.a.d == 64) bwd_join_kernel<h, 64><<<grid, 256, 0, st>>>(w, bk, (h *)dK, (h *)dV);
        else bwd_join_kernel<h, 128><<<grid, 256, 0, st>>>(w, bk, (h *)dK, (h *)dV);
    }
    return cudaGetLastError();
}

}  // namespace local
}  // namespace hsa
