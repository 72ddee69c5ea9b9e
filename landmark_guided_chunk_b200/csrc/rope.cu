// rope.cu -- rotary positions of query and key heads, and the append of new
// tokens to a paged cache (the same rotation on the way into the pages).
//
// For the pair (x1, x2) with index i at position p, with a = p f_i:
//   y1 = mult (x1 cos a - x2 sin a),  y2 = mult (x2 cos a + x1 sin a)
// f_i / 2 pi is held in fp64, the turns p f_i / 2 pi are reduced to (-1/2, 1/2]
// in fp64 and only then rounded to fp32: at position 2^24 an fp32 angle would be
// off by a radian.  A block takes TB tokens; their sines are computed once, into
// shared memory, and used by all heads.
//
// Bound: HBM (each element read once and written once; 3 flops per element).
#include "local.cuh"

namespace hsa {
namespace local {

namespace {

constexpr int NT = 256;
constexpr int MAXTB = 4;
constexpr int NB = 4;   // units in flight per thread

struct IoArgs {
    const void *q, *k, *v;
    void *qo, *ko, *vo;
    int hq, hk, hv;          // heads of each tensor that are processed (0: none)
    int d;
    long long tokens;        // tokens in all (append: rows of the row tensors)
    int T, pos0;             // rotation alone: tokens per sequence, position of its token 0
    const int32_t *pos;      // rotation alone: explicit positions
};

template <typename T, int V> struct Vec;
template <> struct Vec<float, 4> { typedef float4 type; };
template <> struct Vec<__nv_bfloat16, 8> { typedef uint4 type; };
template <> struct Vec<float, 1> { typedef float type; };
template <> struct Vec<__nv_bfloat16, 1> { typedef __nv_bfloat16 type; };

// The sequence that owns row r: the last b with q_start[b] <= r, or -1.
__device__ int find_seq(const LocArgs &a, int r) {
    int lo = 0, hi = a.B;   // q_start is non-decreasing over [0, B]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid + 1] <= r) lo = mid + 1;
        else hi = mid;
    }
    return lo < a.B && a.q_start[lo] <= r ? lo : -1;
}

// V: elements per vector.  A unit is two vectors of one head: the two halves of
// V pairs, or 2 V neighbours to copy.
template <typename T, int V, int TB, bool APPEND>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ RopeArgs r, const __grid_constant__ IoArgs io,
                                                  const __grid_constant__ LocArgs a) {
    typedef typename Vec<T, V>::type W;
    __shared__ float2 cs[TB][64];
    __shared__ int spos[TB];
    __shared__ long long srow[TB];   // token's row of K and V at the destination (-1: not written)
    __shared__ int slive[TB];
    const long long tok0 = (long long)blockIdx.x * TB;
    if (threadIdx.x < TB) {
        const long long t = tok0 + threadIdx.x;
        int live = t < io.tokens, p = 0;
        long long row = t;
        if (live) {
            if constexpr (APPEND) {
                const int b = find_seq(a, (int)t);
                live = b >= 0;
                if (live) {
                    const int r0 = a.q_start[b], n = a.q_start[b + 1] - r0, kv = a.kv_len[b];
                    p = kv - n + (int)t - r0;
                    // a length outside its bounds writes nothing
                    const bool ok = r0 >= 0 && n <= a.max_q && kv <= a.max_kv && p >= 0 && p < a.max_kv;
                    if (!ok) atomicOr(a.status, DEV_BAD_INDEX);
                    row = ok ? kv_row(a, b, p) : -1;
                    live = ok;
                }
            } else {
                p = io.pos ? io.pos[t] : io.pos0 + (int)(t % io.T);
            }
        }
        spos[threadIdx.x] = p;
        srow[threadIdx.x] = row;
        slive[threadIdx.x] = live;
    }
    __syncthreads();
    const int np = r.rot >> 1;
    for (int i = threadIdx.x; i < TB * np; i += NT) {
        const int t = i / np, x = i % np;
        const double turns = (double)spos[t] * r.f[x];
        const float fr = (float)(turns - rint(turns));
        float sn, cn;
        sincospif(2.f * fr, &sn, &cn);
        cs[t][x] = make_float2(cn * r.mult, sn * r.mult * r.sgn);
    }
    __syncthreads();
    const int per_head = io.d / (2 * V), heads = io.hq + io.hk + io.hv;
    const int units = TB * heads * per_head;
    const int nrot = r.rot / (2 * V);   // rotated units per head
    for (int base = threadIdx.x; base < units; base += NT * NB) {
        W x1[NB], x2[NB];
        T *dst[NB];
        int off2[NB], pair[NB];         // pair: first pair index, or -1 for a copy
        int tk[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int u = base + n * NT;
            dst[n] = nullptr;
            if (u >= units) continue;
            const int c = u % per_head, hh = u / per_head % heads, t = u / per_head / heads;
            if (!slive[t]) continue;
            const T *src;
            T *out;
            bool rot = c < nrot;
            if (hh < io.hq) {
                const long long e = ((tok0 + t) * io.hq + hh) * io.d;
                src = (const T *)io.q + e;
                out = (T *)io.qo + e;
            } else {
                const bool isv = hh >= io.hq + io.hk;
                const int h = hh - io.hq - (isv ? io.hk : 0);
                const long long e = ((tok0 + t) * io.hk + h) * io.d;
                src = (const T *)(isv ? io.v : io.k) + e;
                if (srow[t] < 0) continue;
                out = (T *)(isv ? io.vo : io.ko) + (srow[t] * io.hk + h) * io.d;
                rot = rot && !isv;
            }
            const int o1 = rot && !r.interleaved ? c * V : c * 2 * V;
            off2[n] = rot && !r.interleaved ? np : V;
            pair[n] = rot ? c * V : -1;
            tk[n] = t;
            x1[n] = *reinterpret_cast<const W *>(src + o1);
            x2[n] = *reinterpret_cast<const W *>(src + o1 + off2[n]);
            dst[n] = out + o1;
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (!dst[n]) continue;
            if (pair[n] >= 0) {
                T e[2 * V];
                *reinterpret_cast<W *>(e) = x1[n];
                *reinterpret_cast<W *>(e + V) = x2[n];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 f = cs[tk[n]][pair[n] + i];
                    const float u = to_f32(r.interleaved ? e[2 * i] : e[i]);
                    const float v = to_f32(r.interleaved ? e[2 * i + 1] : e[V + i]);
                    const T y1 = from_f32<T>(u * f.x - v * f.y), y2 = from_f32<T>(v * f.x + u * f.y);
                    if (r.interleaved) {
                        e[2 * i] = y1;
                        e[2 * i + 1] = y2;
                    } else {
                        e[i] = y1;
                        e[V + i] = y2;
                    }
                }
                x1[n] = *reinterpret_cast<W *>(e);
                x2[n] = *reinterpret_cast<W *>(e + V);
            }
            *reinterpret_cast<W *>(dst[n]) = x1[n];
            *reinterpret_cast<W *>(dst[n] + off2[n]) = x2[n];
        }
    }
}

template <typename T, int V, bool APPEND>
cudaError_t go(const RopeArgs &r, const IoArgs &io, const LocArgs &a, cudaStream_t st) {
    // few tokens: one per block, so that they spread over the SMs
    if (io.tokens <= 2048)
        rope_kernel<T, V, 1, APPEND><<<(unsigned)io.tokens, NT, 0, st>>>(r, io, a);
    else
        rope_kernel<T, V, MAXTB, APPEND><<<(unsigned)((io.tokens + MAXTB - 1) / MAXTB), NT, 0, st>>>(r, io, a);
    return cudaGetLastError();
}

template <bool APPEND>
cudaError_t by_type(const RopeArgs &r, int dtype, const IoArgs &io, const LocArgs &a, cudaStream_t st) {
    if (io.tokens == 0 || io.hq + io.hk + io.hv == 0) return cudaSuccess;
    // whole 16-byte vectors where the rotated part is made of them, else single elements
    if (dtype == HSA_F32)
        return r.rot % 8 == 0 ? go<float, 4, APPEND>(r, io, a, st) : go<float, 1, APPEND>(r, io, a, st);
    return r.rot % 16 == 0 ? go<__nv_bfloat16, 8, APPEND>(r, io, a, st) : go<__nv_bfloat16, 1, APPEND>(r, io, a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &r, int dtype, int B, int T, int H, int Hkv, int d, int pos0,
                        const int32_t *pos, const void *Q, const void *K, void *Qr, void *Kr, cudaStream_t st) {
    IoArgs io{};
    io.q = Q;
    io.k = K;
    io.qo = Qr;
    io.ko = Kr;
    io.hq = Q ? H : 0;
    io.hk = K ? Hkv : 0;
    io.d = d;
    io.tokens = (long long)B * T;
    io.T = T;
    io.pos0 = pos0;
    io.pos = pos;
    return by_type<false>(r, dtype, io, LocArgs{}, st);
}

cudaError_t launch_append(const RopeArgs *r, const LocArgs &a, int dtype, const void *k, const void *v, const void *Q,
                          void *Qr, void *Kp, void *Vp, cudaStream_t st) {
    IoArgs io{};
    io.q = Q;
    io.k = k;
    io.v = v;
    io.qo = Qr;
    io.ko = Kp;
    io.vo = Vp;
    io.hq = Q ? a.H : 0;
    io.hk = io.hv = a.Hkv;
    io.d = a.d;
    io.tokens = a.rows;
    RopeArgs none{};
    return by_type<true>(r ? *r : none, dtype, io, a, st);
}

}  // namespace local
}  // namespace hsa
