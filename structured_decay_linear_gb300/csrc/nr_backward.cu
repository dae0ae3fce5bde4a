// Norms of queries and keys and their rotation by position: gradients.
//
// As the forward (nr_forward.cu): the gradient is turned back by the token's angles and goes through the norm, whose r is
// formed again from x. x and dy are read once, dx is written once. CTAs serve either queries or keys, in proportion to their
// heads, so that a lane's features belong to one weight; weight gradients are summed in registers over all of a CTA's
// tokens, then over groups of CTAs by the last of each, and over groups by the last one, each in a fixed order: the same
// bits on every run. That many CTAs as an SM holds at once (6, for the sums' registers): more would each add sums.
//
// Measured (16 query and 4 key heads of 128, 16 bits, B4 T4096): 57 us with weights, 4.4 TB/s of q, k and the gradients;
// with the forward in front 89 us, and without weights, where 8 CTAs an SM and many rounds of them are free, 75 us. With 32-bit
// gradients coming in 62 us (5.4 TB/s), all in 32 bits 90 us (5.6). Less than half of the issue slots are used and warps wait for
// memory most. The next heads' features asked for before these are done: 6 us more (registers); 5 CTAs an SM: 3 us more.
#include "nr_internal.h"

namespace dplr {
namespace nr {
namespace {

// A piece's gradients: as wide as its inputs, or 32-bit ones of 16-bit inputs.
template <class GT, int E> struct Grads {
    static constexpr int N = E * (int)sizeof(GT) / 16;
    uint4 r[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const GT* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = *reinterpret_cast<const uint4*>(p + 16 / (int)sizeof(GT) * i);
    }
    __device__ __forceinline__ void values(float2* v) const {
#pragma unroll
        for (int i = 0; i < N; ++i) unpack<GT>(r[i], v + E / 2 / N * i);
    }
};

constexpr int kRounds = 16;                                 // of CTAs, at most, where there are no weight gradients

// Sums `n` rows of D, `row` their first; by all threads, the result to `out`.
template <int D> __device__ __forceinline__ void sum_rows(const float* row, int n, float* out) {
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float v = 0.f;
#pragma unroll 8
        for (int r = 0; r < n; ++r) v += __ldcg(row + (long long)r * D + i);
        __stcg(out + i, v);
    }
}

// Whether this CTA is the last of `n` to come here; all of its threads' writes before, and what the others wrote, are then seen.
__device__ __forceinline__ bool last_of(unsigned* count, unsigned n, bool* shared) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        *shared = atomicAdd(count, 1u) + 1u == n;
        if (*shared) *count = 0;                                // for the next launch
    }
    __syncthreads();
    __threadfence();
    return *shared;
}

// SUMS: weight gradients are asked for.
template <class XT, class GT, int D, bool NORM, bool SUMS, bool INTER>
__global__ void __launch_bounds__(kThreads, SUMS ? 6 : 8) nr_backward_kernel(const __grid_constant__ Args a, int q_ctas) {
    constexpr int E = Piece<XT>::E, L = D / (2 * E), SIDE = 32 / L;
    __shared__ __align__(16) Angles table[kWarps];
    __shared__ __align__(16) float weight[NORM ? D : 1];
    const bool is_q = (int)blockIdx.x < q_ctas;
    const int cta = is_q ? blockIdx.x : blockIdx.x - q_ctas, ctas = is_q ? q_ctas : gridDim.x - q_ctas;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane % L, mine = lane / L;
    const int H = is_q ? a.Hq : a.Hk;
    int f0, f1;
    places<E>(j, a.rot, INTER, f0, f1);
    const int to_f1 = f1 - f0;
    const bool turned = 2 * E * j < a.rot;                      // this lane's features are rotated
    if (NORM) {
        if (w == 0) fill_weights<E, L>(weight, is_q ? a.wq : a.wk, j, f0, f1);
        __syncthreads();
    }
    const float out_scale = is_q ? a.q_scale : 1.f;
    float2 acc[SUMS ? E : 1] = {};
    const long long tokens = (long long)a.B * a.T;
    for (long long tok = (long long)cta * kWarps + w; tok < tokens; tok += (long long)ctas * kWarps) {
        const int b = (int)(tok / a.T), t = (int)(tok - (long long)b * a.T);
        const int pos = position(a, b, t);
        const Rows &X = is_q ? a.q : a.k, &G = is_q ? a.gq : a.gk, &O = is_q ? a.oq : a.ok;
        XT* op = static_cast<XT*>(const_cast<void*>(O.p)) + b * O.sb + t * O.st + mine * O.sh + f0;
        if (pos < 0) {                                          // a row without a token: what is not used has no gradient
            for (int h = mine; h < H; h += SIDE, op += SIDE * O.sh) {
                *reinterpret_cast<uint4*>(op) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(op + to_f1) = make_uint4(0, 0, 0, 0);
            }
            continue;
        }
        const XT* xp = static_cast<const XT*>(X.p) + b * X.sb + t * X.st + mine * X.sh + f0;
        const GT* gp = static_cast<const GT*>(G.p) + b * G.sb + t * G.st + mine * G.sh + f0;
        for (int h = mine; h - mine < H; h += SIDE, xp += SIDE * X.sh, gp += SIDE * G.sh, op += SIDE * O.sh) {
            Grads<GT, E> g0, g1;
            uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
            g0.zero(); g1.zero();
            if (h < H) {
                g0.load(gp);
                g1.load(gp + to_f1);
                if (NORM) {
                    r0 = *reinterpret_cast<const uint4*>(xp);
                    r1 = *reinterpret_cast<const uint4*>(xp + to_f1);
                }
            }
            if (h == mine) {                                    // while the first heads are on their way
                __syncwarp();
#pragma unroll 1
                for (int i = lane; i < a.rot / 2; i += 32) angle<E, L>(a, pos, i, table[w]);
                __syncwarp();
            }
            float2 dy[E], z[E];
            g0.values(dy);
            g1.values(dy + E / 2);
            if (turned) {
                Turn<E, L, INTER> by;
                by.load(table[w], j);
                by.template apply<true>(dy, z);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) z[e] = dy[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) z[e] = mul2(both(out_scale), z[e]);
            if (NORM) {
                float2 x[E];
                unpack<XT>(r0, x);
                unpack<XT>(r1, x + E / 2);
                const float sum = head_dot<E, L>(x, x);
                const float inv = h < H ? rsqrtf(fmaf(sum, a.share, a.eps)) : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (SUMS) acc[e] = fma2(mul2(z[e], both(inv)), x[e], acc[e]);
                    z[e] = mul2(z[e], weight_of<E, L>(weight, j, e));
                }
                const float dot = -head_dot<E, L>(z, x) * a.share * inv * inv;
#pragma unroll
                for (int e = 0; e < E; ++e) z[e] = mul2(both(inv), fma2(x[e], both(dot), z[e]));
            }
            if (h < H) {
                *reinterpret_cast<uint4*>(op) = pack<XT>(z);
                *reinterpret_cast<uint4*>(op + to_f1) = pack<XT>(z + E / 2);
            }
        }
    }
    if constexpr (SUMS) {
        __shared__ float sums[kWarps][D];
        __shared__ bool last;
        // this CTA's sums: the warp's heads side by side, then the warps
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (L < 32) {
#pragma unroll
                for (int off = L; off < 32; off <<= 1) {
                    acc[e].x += __shfl_xor_sync(0xffffffffu, acc[e].x, off);
                    acc[e].y += __shfl_xor_sync(0xffffffffu, acc[e].y, off);
                }
            }
            const int f = (e < E / 2 ? f0 : f1 - E) + 2 * e;
            if (mine == 0) { sums[w][f] = acc[e].x; sums[w][f + 1] = acc[e].y; }
        }
        __syncthreads();
        float* rows = a.part + (is_q ? 0LL : (long long)kGradCtas * D);
        for (int i = threadIdx.x; i < D; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) v += sums[x][i];
            __stcg(rows + (long long)cta * D + i, v);
        }
        const int group = cta / kGradGroup, groups = (ctas + kGradGroup - 1) / kGradGroup;
        const int first = group * kGradGroup, n = min(kGradGroup, ctas - first);
        unsigned* counts = a.done + (is_q ? 0 : 1 + kGradGroups);
        float* group_rows = a.part + 2LL * kGradCtas * D + (is_q ? 0LL : (long long)kGradGroups * D);
        float* out = is_q ? a.dwq : a.dwk;
        if (!last_of(counts + 1 + group, n, &last)) return;
        sum_rows<D>(rows + (long long)first * D, n, group_rows + (long long)group * D);
        if (!last_of(counts, groups, &last)) return;
        if (out) sum_rows<D>(group_rows, groups, out);
    }
}

template <class XT, class GT, int D> cudaError_t launch_one(const Args& a, cudaStream_t s) {
    constexpr int SIDE = 32 / (D / (2 * Piece<XT>::E));
    const bool sums = a.dwq || a.dwk;
    const long long tokens = (long long)a.B * a.T, need = (tokens + kWarps - 1) / kWarps;
    const int gq = (a.Hq + SIDE - 1) / SIDE, gk = (a.Hk + SIDE - 1) / SIDE;
    const long long most = sums ? kGradCtas : 152LL * 8 * kRounds;
    long long q = most * gq / (gq + gk), k = a.Hk ? most - q : 0;
    if (q < 1) q = 1;
    if (a.Hk && k < 1) k = 1;
    if (q > most - k) q = most - k;
    if (q > need) q = need;
    if (k > need) k = need;
    void (*f)(Args, int);
    if (a.norm == kNone) f = a.interleaved ? nr_backward_kernel<XT, GT, D, false, false, true> : nr_backward_kernel<XT, GT, D, false, false, false>;
    else if (sums) f = a.interleaved ? nr_backward_kernel<XT, GT, D, true, true, true> : nr_backward_kernel<XT, GT, D, true, true, false>;
    else f = a.interleaved ? nr_backward_kernel<XT, GT, D, true, false, true> : nr_backward_kernel<XT, GT, D, true, false, false>;
    f<<<(unsigned)(q + k), kThreads, 0, s>>>(a, (int)q);
    return cudaGetLastError();
}

template <class XT, class GT> cudaError_t by_size(const Args& a, int d, cudaStream_t s) {
    switch (d) {
        case 32: return launch_one<XT, GT, 32>(a, s);
        case 64: return launch_one<XT, GT, 64>(a, s);
        case 128: return launch_one<XT, GT, 128>(a, s);
        case 256: return launch_one<XT, GT, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_backward(const Args& a, bool bf16, bool grad_bf16, int d, cudaStream_t s) {
    if (!bf16) return by_size<float, float>(a, d, s);
    return grad_bf16 ? by_size<__nv_bfloat16, __nv_bfloat16>(a, d, s) : by_size<__nv_bfloat16, float>(a, d, s);
}

}  // namespace nr
}  // namespace dplr
