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
// 65536 tokens of 32 + 8 heads of 128, bf16: 222 us, where torch's copy of the
// same bytes takes 215.  One unit per thread and turn: two or four in flight per
// thread cost the registers of a block per SM (245 and 275 us).
#include "local.cuh"

namespace hsa {
namespace local {

namespace {

constexpr int NT = 256;

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
// V pairs, or 2 V neighbours to copy.  A thread's first unit is on its way
// before the block looks up where its tokens sit (for the append, a search and
// two dependent loads) and takes their sines.
template <typename T, int V, int TB, bool APPEND>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ RopeArgs r, const __grid_constant__ IoArgs io,
                                                  const __grid_constant__ LocArgs a) {
    typedef typename Vec<T, V>::type W;
    __shared__ float2 cs[TB][64];
    __shared__ int spos[TB];
    __shared__ long long srow[TB];   // token's row of K and V at the destination (-1: not written)
    __shared__ int slive[TB];
    const long long tok0 = (long long)blockIdx.x * TB;
    const int ntok = (int)min((long long)TB, io.tokens - tok0);
    const int ph_log = 31 - __clz(io.d / (2 * V)), heads = io.hq + io.hk + io.hv;   // units per head: a power of two
    const int units = ntok * heads << ph_log;
    const int np = r.rot >> 1, nrot = r.rot / (2 * V);   // pairs, rotated units per head
    const unsigned magic = 0xffffffffu / (unsigned)heads + 1u;   // row / heads for rows below 2^16 (heads > 1)

    struct Unit {
        W x1, x2;
        int t, o1, off2, pair, h, kind;   // kind: 0 Q, 1 K, 2 V, -1 none; pair: first pair index, -1 to copy
    } u;
    auto load = [&](int i) {
        u.kind = -1;
        if (i >= units) return;
        const int c = i & ((1 << ph_log) - 1), row = i >> ph_log;
        u.t = heads == 1 ? row : (int)__umulhi((unsigned)row, magic);
        int hh = row - u.t * heads;
        const T *src;
        if (hh < io.hq) {
            u.kind = 0;
            src = (const T *)io.q + ((tok0 + u.t) * io.hq + hh) * io.d;
        } else {
            hh -= io.hq;
            u.kind = hh < io.hk ? 1 : 2;
            if (u.kind == 2) hh -= io.hk;
            src = (const T *)(u.kind == 2 ? io.v : io.k) + ((tok0 + u.t) * io.hk + hh) * io.d;
        }
        u.h = hh;
        const bool rot = c < nrot && u.kind != 2;
        u.o1 = rot && !r.interleaved ? c * V : c * 2 * V;
        u.off2 = rot && !r.interleaved ? np : V;
        u.pair = rot ? c * V : -1;
        u.x1 = *reinterpret_cast<const W *>(src + u.o1);
        u.x2 = *reinterpret_cast<const W *>(src + u.o1 + u.off2);
    };
    load(threadIdx.x);
    if (threadIdx.x < ntok) {
        const long long t = tok0 + threadIdx.x;
        int live = 1, p = 0;
        long long row = t;
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
        spos[threadIdx.x] = p;
        srow[threadIdx.x] = row;
        slive[threadIdx.x] = live;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ntok * np; i += NT) {
        const int t = i / np, x = i % np;
        const double turns = (double)spos[t] * r.f[x];
        const float fr = (float)(turns - rint(turns));
        float sn, cn;
        sincospif(2.f * fr, &sn, &cn);
        cs[t][x] = make_float2(cn * r.mult, sn * r.mult * r.sgn);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < units; i += NT) {
        if (i != (int)threadIdx.x) load(i);
        if (u.kind < 0 || !slive[u.t]) continue;
        T *dst;
        if (u.kind == 0) {
            dst = (T *)io.qo + ((tok0 + u.t) * io.hq + u.h) * io.d + u.o1;
        } else {
            const long long row = srow[u.t];
            if (row < 0) continue;
            dst = (T *)(u.kind == 2 ? io.vo : io.ko) + (row * io.hk + u.h) * io.d + u.o1;
        }
        if (u.pair >= 0) {
            T e[2 * V];
            *reinterpret_cast<W *>(e) = u.x1;
            *reinterpret_cast<W *>(e + V) = u.x2;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float2 f = cs[u.t][u.pair + k];
                const float x = to_f32(r.interleaved ? e[2 * k] : e[k]);
                const float y = to_f32(r.interleaved ? e[2 * k + 1] : e[V + k]);
                const T y1 = from_f32<T>(x * f.x - y * f.y), y2 = from_f32<T>(y * f.x + x * f.y);
                if (r.interleaved) {
                    e[2 * k] = y1;
                    e[2 * k + 1] = y2;
                } else {
                    e[k] = y1;
                    e[V + k] = y2;
                }
            }
            u.x1 = *reinterpret_cast<W *>(e);
            u.x2 = *reinterpret_cast<W *>(e + V);
        }
        *reinterpret_cast<W *>(dst) = u.x1;
        *reinterpret_cast<W *>(dst + u.off2) = u.x2;
    }
}

template <typename T, int V, bool APPEND>
cudaError_t go(const RopeArgs &r, const IoArgs &io, const LocArgs &a, cudaStream_t st) {
    // few tokens: one per block, so that they spread over the SMs; many: several per block
    auto run = [&](auto kern, int tb) {
        kern<<<(unsigned)((io.tokens + tb - 1) / tb), NT, 0, st>>>(r, io, a);
        return cudaGetLastError();
    };
    return io.tokens <= 2048 ? run(rope_kernel<T, V, 1, APPEND>, 1) : run(rope_kernel<T, V, 4, APPEND>, 4);
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
