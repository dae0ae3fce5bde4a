// Norms of the heads of queries and keys and rotary positions: what the translation units share (not part of the ABI).
//
// Per token and head, with x the head's d features:
//
//   n = x r w,   r = (sum x^2 / d + eps)^-1/2  or  (sum x^2 + eps)^-1/2  (or n = x)
//   (u, v) of pair i among the first `rot` features  ->  c (u cos - v sin, v cos + u sin) at angle pos f_i;  the rest as it is
//   and everything times q_scale for queries
//
// and backwards, with z the scaled gradient turned back and o = z w:
//
//   dx = r (o - x r^2 (o . x) / d)  (L2: without / d),   dw = sum over tokens and heads of z x r
//
// Angles: a frequency is a 64-bit fraction of a turn, so position times frequency in 64-bit integers is exact modulo whole
// turns at every position. It is rounded to 32 bits and its quarter turns are taken off in integers; the rest, up to an eighth of a
// turn, is off by at most 2^-28 turns as a 32-bit float (the whole phase would be off by 2^-26).
#pragma once

#include "hd_internal.h"
#include "packed.cuh"
#include "sm100_ops.cuh"

namespace dplr {
namespace nr {

constexpr int kNone = DPLR_NR_NONE, kRms = DPLR_NR_RMS, kL2 = DPLR_NR_L2;
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kMaxRot = 256;

struct Rows { const void* p; long long sb, sh, st; };   // element strides

struct Args {
    Rows q, k;                     // forward: inputs
    Rows oq, ok;                   // forward: outputs; backward: gradients of the inputs
    Rows gq, gk;                   // backward: gradients of the outputs
    const int* pos; long long psb, pst; int first;   // without pos: first + token
    const unsigned long long* turns;   // [rot / 2]
    const float* wq; const float* wk;  // [d], nullable
    int B, T, Hq, Hk, rot, interleaved, norm;
    float eps, share;              // share: 1 / d or 1
    float q_scale, rot_scale;
    float* dwq; float* dwk;        // backward, nullable: [d]
    float* part;                   // [2][kGradCtas][d] sums of CTAs, then [2][kGradGroups][d] of groups of CTAs
    unsigned* done;                // [2][1 + kGradGroups] counters, zero between launches
};

// Weight gradients: the sums of most CTAs of a side are added up kGradGroup at a time, then those sums.
constexpr int kGradGroup = 24, kGradGroups = 38, kGradCtas = kGradGroup * kGradGroups;

cudaError_t launch_forward(const Args& a, bool bf16, int d, cudaStream_t s);
cudaError_t launch_backward(const Args& a, bool bf16, bool grad_bf16, int d, cudaStream_t s);

// ---------------------------------------------------------------------------------------------------------------
// A head's features over the lanes. A lane holds two 16-byte pieces of E features, as E pairs v[0 .. E): v[0 .. E/2) are piece
// 0. So that both members of a rotated pair are in one lane, pieces 0 and 1 of lane j are features E j.. and rot / 2 + E j.. of
// the rotated part, or its neighbours 2 E j.. where pairs are neighbours, and 2 E j.. of the rest. Pair E j + e is then the
// e-th pair of lane j in both layouts.
// ---------------------------------------------------------------------------------------------------------------
template <class XT> struct Piece {
    static constexpr int E = 16 / (int)sizeof(XT);
};

template <class XT> __device__ __forceinline__ void unpack(const uint4& r, float2* v);
template <> __device__ __forceinline__ void unpack<float>(const uint4& r, float2* v) {
    v[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    v[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& r, float2* v) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
template <class XT> __device__ __forceinline__ uint4 pack(const float2* v);
template <> __device__ __forceinline__ uint4 pack<float>(const float2* v) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
}
template <> __device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float2* v) {
    return make_uint4(sm100::pack_bf16(v[0].x, v[0].y), sm100::pack_bf16(v[1].x, v[1].y), sm100::pack_bf16(v[2].x, v[2].y),
                      sm100::pack_bf16(v[3].x, v[3].y));
}

// First features of lane j's two pieces.
template <int E> __device__ __forceinline__ void places(int j, int rot, int interleaved, int& f0, int& f1) {
    const int turned = rot / (2 * E);
    if (j < turned && !interleaved) { f0 = E * j; f1 = rot / 2 + E * j; }
    else { f0 = 2 * E * j; f1 = f0 + E; }
}

// A token's cosines and sines, times rot_scale, in the order in which lanes read them: lane j's pairs E j .. in pieces of four,
// the j-th of the first pieces, then of the second ones, so that lanes side by side read side by side.
struct Angles { float c[kMaxRot / 2], s[kMaxRot / 2]; };
template <int E, int L> __device__ __forceinline__ int place_of(int pair) {
    const int j = pair / E, e = pair % E;
    return ((e / 4) * L + j) * 4 + e % 4;
}
template <int E, int L> __device__ __forceinline__ void angle(const Args& a, int pos, int pair, Angles& row) {
    const unsigned long long phase = (unsigned long long)(unsigned)pos * a.turns[pair];
    const unsigned turn = (unsigned)((phase + 0x80000000u) >> 32);           // in units of 2^-32
    const unsigned quarters = (turn + 0x20000000u) >> 30;                    // the nearest number of quarter turns, modulo 4
    float s, c;
    sincospif((float)(int)(turn - (quarters << 30)) * 0x1p-31f, &s, &c);     // what is left of it, up to an eighth of a turn
    const float cosine = quarters & 1 ? s : c, sine = quarters & 1 ? c : s;
    row.c[place_of<E, L>(pair)] = ((quarters + 1) & 2 ? -cosine : cosine) * a.rot_scale;
    row.s[place_of<E, L>(pair)] = (quarters & 2 ? -sine : sine) * a.rot_scale;
}

// The rotation of a lane's pairs: v[e] becomes v[e] p[e] + (the other members) q[e], the other members being v's other piece, or
// with neighbours v[e]'s two numbers changed over. Lanes behind the rotated part keep theirs: a factor of 0 would make NaN of a
// partner that is not finite.
template <int E, int L, bool INTER> struct Turn {
    float c[E], s[E];
    __device__ __forceinline__ void load(const Angles& row, int j) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 cs = *reinterpret_cast<const float4*>(row.c + (e * L + 4 * j));
            const float4 sn = *reinterpret_cast<const float4*>(row.s + (e * L + 4 * j));
            c[e] = cs.x; c[e + 1] = cs.y; c[e + 2] = cs.z; c[e + 3] = cs.w;
            s[e] = sn.x; s[e + 1] = sn.y; s[e + 2] = sn.z; s[e + 3] = sn.w;
        }
    }
    static __device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }
    static __device__ __forceinline__ float2 over(float2 v) { return make_float2(v.y, v.x); }
    __device__ __forceinline__ float2 p(int e) const {
        return INTER ? both(c[e]) : make_float2(c[2 * e % E], c[2 * e % E + 1]);
    }
    __device__ __forceinline__ float2 q(int e) const {
        if (INTER) return make_float2(-s[e], s[e]);
        const float2 v = make_float2(s[2 * e % E], s[2 * e % E + 1]);
        return e < E / 2 ? minus(v) : v;
    }
    static __device__ __forceinline__ float2 other(const float2 (&v)[E], int e) { return INTER ? over(v[e]) : v[(e + E / 2) % E]; }
    // BACK: by minus the angles.
    template <bool BACK> __device__ __forceinline__ void apply(const float2 (&v)[E], float2 (&to)[E]) const {
#pragma unroll
        for (int e = 0; e < E; ++e) to[e] = fma2(v[e], p(e), mul2(other(v, e), BACK ? minus(q(e)) : q(e)));
    }
};

// Where feature f of a head stands in a row of weights, so that lanes side by side read side by side: pieces of four features,
// the first ones of all lanes' features, then the second ones.
template <int E, int L> __device__ __forceinline__ int weight_place(int j, int i) { return ((i / 4) * L + j) * 4 + i % 4; }
// Fills a row: the 2 E features of lane j, whose pieces start at f0 and f1. By the threads of one or more whole heads' lanes.
template <int E, int L> __device__ __forceinline__ void fill_weights(float* row, const float* w, int j, int f0, int f1) {
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) row[weight_place<E, L>(j, i)] = w ? w[i < E ? f0 + i : f1 + i - E] : 1.f;
}
// The e-th pair of lane j's weights.
template <int E, int L> __device__ __forceinline__ float2 weight_of(const float* row, int j, int e) {
    return *reinterpret_cast<const float2*>(row + weight_place<E, L>(j, 2 * e));
}

// Sum of the products of two lanes' features over the L lanes of a head (a power of two; heads side by side in a warp).
template <int E, int L> __device__ __forceinline__ float head_dot(const float2 (&x)[E], const float2 (&y)[E]) {
    float2 t = mul2(x[0], y[0]), u = mul2(x[1], y[1]);          // two sums, so that half as many additions wait for one another
#pragma unroll
    for (int e = 2; e < E; e += 2) {
        t = fma2(x[e], y[e], t);
        u = fma2(x[e + 1], y[e + 1], u);
    }
    t = add2(t, u);
    float v = t.x + t.y;
#pragma unroll
    for (int off = 1; off < L; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ int position(const Args& a, int b, int t) {
    return a.pos ? a.pos[b * a.psb + t * a.pst] : a.first + t;
}

}  // namespace nr
}  // namespace dplr
