// Norms of queries and keys and their rotation by position: forward.
//
// Each feature is read once and written once and HBM is what bounds a long call. A warp takes a token (or a part of its
// heads, where tokens are few): its angles once, then its heads, as many side by side as 32 lanes of two 16-byte pieces hold,
// U such groups in flight. Warps have few tokens each, so that those of an SM are at different places: with one round of CTAs all
// of them load, and then all compute (243 us where many rounds took 182, at B8 T8192, 32 heads of 128). A token's rows may
// lie anywhere: heads before tokens on one side and after them on the other.
//
// Measured at that size (the copy rate is 6.79 TB/s): 164 us, 6.5 TB/s; without a norm 157 us, 6.8; heads of 64, 166 us; in 32
// bits with half the batch 172 us; one token for each of 64 rows 3.4 us, a launch's latency. A norm's instructions are what
// keeps it from the copy rate: 63% of all issue slots. Rings of asynchronous copies, angles shared by a CTA's heads, larger CTAs:
// slower. Lanes behind the rotated part go a way of their own (Turn); sines held in registers over a token's heads in 32 bits:
// 192 instead of 179 us, with spills.
#include "nr_internal.h"

namespace dplr {
namespace nr {
namespace {

template <class XT> struct Shape { static constexpr int U = sizeof(XT) == 2 ? 2 : 1, CTAS = sizeof(XT) == 2 ? 8 : 10; };  // groups in flight, CTAs a SM
constexpr int kRounds = 32;                                 // of CTAs, at most

template <class XT, int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, (Shape<XT>::CTAS)) nr_forward_kernel(const __grid_constant__ Args a, int split, int per) {
    constexpr int E = Piece<XT>::E, L = D / (2 * E), SIDE = 32 / L, U = Shape<XT>::U;
    __shared__ __align__(16) Angles table[kWarps];
    __shared__ __align__(16) float weight[2][NORM ? D : 1];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane % L, mine = lane / L;
    const int H = a.Hq + a.Hk;
    int f0, f1;
    places<E>(j, a.rot, INTER, f0, f1);
    if (NORM) {
        if (w < 2) fill_weights<E, L>(weight[w], w ? a.wk : a.wq, j, f0, f1);
        __syncthreads();
    }
    const int to_f1 = f1 - f0;
    const bool turned = 2 * E * j < a.rot;                      // this lane's features are rotated
    const long long items = (long long)a.B * a.T * split, step = (long long)gridDim.x * kWarps;
    for (long long it = (long long)blockIdx.x * kWarps + w; it < items; it += step) {
        const unsigned tok = split == 1 ? (unsigned)it : (unsigned)(it / split);
        const int part = split == 1 ? 0 : (int)(it - (long long)tok * split);
        const int b = tok / a.T, t = tok - b * a.T;
        const int pos = position(a, b, t);
        if (pos < 0) continue;                                  // a row without a token
        const XT* q = static_cast<const XT*>(a.q.p) + b * a.q.sb + t * a.q.st + f0;
        const XT* k = static_cast<const XT*>(a.k.p) + b * a.k.sb + t * a.k.st + f0;
        XT* oq = static_cast<XT*>(const_cast<void*>(a.oq.p)) + b * a.oq.sb + t * a.oq.st + f0;
        XT* ok = static_cast<XT*>(const_cast<void*>(a.ok.p)) + b * a.ok.sb + t * a.ok.st + f0;
        const int first = part * per, end = min(H, first + per);
        for (int h0 = first; h0 < end; h0 += U * SIDE) {
            uint4 r[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * SIDE + mine;
                r[u][0] = r[u][1] = make_uint4(0, 0, 0, 0);
                if (h < end) {
                    const XT* p = h < a.Hq ? q + h * a.q.sh : k + (h - a.Hq) * a.k.sh;
                    r[u][0] = *reinterpret_cast<const uint4*>(p);
                    r[u][1] = *reinterpret_cast<const uint4*>(p + to_f1);
                }
            }
            if (h0 == first) {                                  // while the first heads are on their way
                __syncwarp();
#pragma unroll 1
                for (int i = lane; i < a.rot / 2; i += 32) angle<E, L>(a, pos, i, table[w]);
                __syncwarp();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * SIDE + mine;
                if (h0 + u * SIDE >= end) break;                // the whole warp
                float2 x[E], y[E];
                unpack<XT>(r[u][0], x);
                unpack<XT>(r[u][1], x + E / 2);
                float scale = h < a.Hq ? a.q_scale : 1.f;
                if (NORM) {
                    scale *= rsqrtf(fmaf(head_dot<E, L>(x, x), a.share, a.eps));
                    const float* wt = weight[h < a.Hq ? 0 : 1];
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = mul2(x[e], weight_of<E, L>(wt, j, e));
                }
                if (turned) {
                    Turn<E, L, INTER> by;
                    by.load(table[w], j);
                    by.template apply<false>(x, y);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = x[e];
                }
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = mul2(both(scale), y[e]);
                if (h < end) {
                    XT* p = h < a.Hq ? oq + h * a.oq.sh : ok + (h - a.Hq) * a.ok.sh;
                    *reinterpret_cast<uint4*>(p) = pack<XT>(y);
                    *reinterpret_cast<uint4*>(p + to_f1) = pack<XT>(y + E / 2);
                }
            }
        }
    }
}

template <class XT, int D> cudaError_t launch_one(const Args& a, cudaStream_t s) {
    constexpr int SIDE = 32 / (D / (2 * Piece<XT>::E));
    const long long tokens = (long long)a.B * a.T;
    const int H = a.Hq + a.Hk, groups = (H + SIDE - 1) / SIDE;
    // Heads of a token are shared out over several warps only where there would otherwise be fewer than 16 warps an SM: each
    // part forms the token's angles again.
    const long long want = 16LL * 152;
    int split = tokens >= want ? 1 : (int)((want + tokens - 1) / tokens);
    if (split > groups) split = groups;
    const int per = (groups + split - 1) / split * SIDE;
    split = (H + per - 1) / per;
    const long long ctas = (tokens * split + kWarps - 1) / kWarps, most = 152LL * Shape<XT>::CTAS * kRounds;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    const auto f = a.norm == kNone ? (a.interleaved ? nr_forward_kernel<XT, D, false, true> : nr_forward_kernel<XT, D, false, false>)
                                   : (a.interleaved ? nr_forward_kernel<XT, D, true, true> : nr_forward_kernel<XT, D, true, false>);
    f<<<grid, kThreads, 0, s>>>(a, split, per);
    return cudaGetLastError();
}

template <class XT> cudaError_t by_size(const Args& a, int d, cudaStream_t s) {
    switch (d) {
        case 32: return launch_one<XT, 32>(a, s);
        case 64: return launch_one<XT, 64>(a, s);
        case 128: return launch_one<XT, 128>(a, s);
        case 256: return launch_one<XT, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_forward(const Args& a, bool bf16, int d, cudaStream_t s) {
    return bf16 ? by_size<__nv_bfloat16>(a, d, s) : by_size<float>(a, d, s);
}

}  // namespace nr
}  // namespace dplr
