// Elementwise gated linear recurrence: what its translation units share (not part of the ABI).
//
// Per batch entry and channel, with the gate g_t and the input x_t of a token:
//
//   a_t = exp(g_t)  or  sigmoid(g_t),      s_t = 1,  1 - a_t  or  sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + s_t x_t,           y_t = h_t
//
// Backwards, with D_t the gradient of h_t and E_t = a_t D_t what of it reaches h_{t-1}:
//
//   D_t = dy_t + E_{t+1},  E_{T+1} = dh_T,  dh_0 = E_1,      E_t = a_t E_{t+1} + a_t dy_t
//   dx_t = s_t D_t,        dg_t = (D_t (h_{t-1} + s'(a_t) x_t)) da/dg
//
// so both directions are first-order recurrences with the same factors a_t, forward in h and backward in E.
//
// Composition is associative, (A2, b2) after (A1, b1) being (A2 A1, A2 b1 + b2): a tile of tokens is one map h -> A h + b per
// channel, and tiles are chained by one launch (gr_chain.cuh).
#pragma once

#include <cuda_bf16.h>

#include "dplr_internal.h"
#include "packed.cuh"
#include "sm100_ops.cuh"

namespace dplr {
namespace gr {

constexpr int kCols = 32;           // channels of a tile
constexpr int kRuns = 64 / kCols;   // runs of tokens side by side in a warp, two channels a lane
constexpr int kWarps = 8;
constexpr int kCtas = 2;            // a SM
constexpr int kThreads = 32 * kWarps;
constexpr int kStateStep = 64;     // tokens between two kept states (DPLR_GR_STATE_STEP)
static_assert(kStateStep == DPLR_GR_STATE_STEP, "the ABI's step");

// A workspace starts with this; all of it is zero before its first use.
struct Header {
    int status;                    // the ABI's status word
    int pad[15];
    unsigned ticket;               // tiles handed out in this launch
    unsigned done;                 // CTAs that have finished
    unsigned long long epoch;      // launches that have finished: records of other launches are told by it
};
constexpr size_t kHeader = 256;

// A tile's map, or its last state, of one channel, as its successors read it. 16 bytes, written and read as one access.
struct __align__(16) Record {
    float A, b;                    // kMap: h -> A h + b;  kState: the state b
    unsigned long long tag;        // 4 * (epoch + 1) + kind
};
constexpr unsigned kMap = 1, kState = 2;

constexpr int kBoxRows = 256;      // most tokens of a TMA box

// The walk over earlier tiles' records (gr_chain.cuh): tiles looked at together, and batches of them.
constexpr int kBatch = 4, kBatches = 4;

struct Dims {
    int B, T, D;
    int G;                         // groups of kCols channels
    int NT;                        // tiles of a sequence
};

struct Arg {                       // what the chained kernels share
    Dims d;
    Header* head;
    Record* rec;                   // [B][G][NT][kCols]
    int far;                       // tiles back to one that another round of CTAs has computed
    long long wait_cycles;
};

struct Out { void* p; long long sb, st; };     // rows, element strides

struct ForwardArgs {
    Arg c;
    const float* h0;               // [B][D], nullable
    float* hT;                     // [B][D], nullable
    float* states;                 // [B][ceil(T / kStateStep)][D], nullable: the state in front of every kStateStep tokens
    // a ragged batch (B = 1, T rows): the pool of states and the plan's tables
    float* pool;                   // [n_slots][D]
    const int* starts;             // [R + 1] requests' first rows; the last: rows that hold tokens
    int R;
    const int* slot;               // [T]
    const int* pos;                // [T]
    int n_slots;
    Out y;                         // without data: the states alone
};

struct BackwardArgs {
    Arg c;
    const float* dhT;              // [B][D], nullable
    const float* states;           // as above
    float* dh0;                    // [B][D], nullable
};

struct Types { bool xbf16, gbf16; int gate, input; };

inline int box_rows(int tile) { return tile < kBoxRows ? tile : kBoxRows; }

// Tokens of a tile: as many as its CTA's registers hold, 16 a lane forward and 12 backward, and in 32 bits 8, for the stages.
constexpr int forward_tile(bool xbf16) { return (xbf16 ? 16 : 8) * kWarps * kRuns; }
constexpr int backward_tile(bool xbf16) { return (xbf16 ? 12 : 8) * kWarps * kRuns; }
static_assert(backward_tile(true) % kStateStep == 0 && backward_tile(false) % kStateStep == 0, "a tile starts at a kept state");


cudaError_t launch_forward(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y,
                           const ForwardArgs& a, cudaStream_t s);
// The dense forward with warps of several roles (gr_roles.cu), and where it is taken.
bool use_roles(const Types& t, const Dims& d);
cudaError_t launch_roles(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y,
                         const ForwardArgs& a, cudaStream_t s);
cudaError_t launch_packed(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y,
                          const ForwardArgs& a, cudaStream_t s);
cudaError_t launch_backward(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& dy,
                            const CUtensorMap& dx, const CUtensorMap& dg, const BackwardArgs& a, cudaStream_t s);

struct StepArgs {
    const void* x; const void* g; void* y;
    long long xs, gs, ys;          // row strides, elements
    float* pool; const int* slots; int n_slots, N, D;
    int* status;
};
cudaError_t launch_step(const Types& t, const StepArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------------------------------------------
// One token's a, m = 1 - a and s, two channels at a time (Blackwell multiplies and adds pairs of fp32 numbers in one
// instruction, and instructions issued are what a kernel of few bytes a channel runs out of first).
//
// Exponentials are 2^(g log2 e) of the hardware: off by 2 units of 2^-23 and by |g| 2^-23.7, from the product's rounding and the
// constant's. In what enters a state, a h, that is at most 2^-25 of h beyond the two units for gates below 0 (|g| e^g is at most
// 1 / e); gates above 0 have the factor |g|. m is formed without a difference of nearly equal numbers: a gate that forgets a
// thousandth a token would lose ten of its 24 bits.
// ---------------------------------------------------------------------------------------------------------------
constexpr int kLog = DPLR_GR_LOG, kSigmoid = DPLR_GR_SIGMOID;
constexpr int kPlain = DPLR_GR_PLAIN, kComplement = DPLR_GR_COMPLEMENT, kUnit = DPLR_GR_UNIT;

__device__ __forceinline__ float exp2_hw(float v) { float r; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v)); return r; }
__device__ __forceinline__ float recip_hw(float v) { float r; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v)); return r; }
__device__ __forceinline__ float sqrt_hw(float v) { float r; asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v)); return r; }
__device__ __forceinline__ float min_nan(float a, float b) { float r; asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b)); return r; }

constexpr float kLog2e = 1.4426950408889634f;

// a, and where WANT_M m, or with INPUT kUnit s in its place.
template <int GATE, int INPUT, bool WANT_M> __device__ __forceinline__ void decay(float2 g, float2& a, float2& m) {
    if (GATE == kLog) {
        const float2 t = mul2(g, both(kLog2e));
        a = make_float2(exp2_hw(t.x), exp2_hw(t.y));
        if (!WANT_M) return;
        // 1 - e^g by its series up to g^6 for |g| < 1/4, where the next term is below 5e-8 of it; beyond, gates above 0 among them,
        // the difference loses two bits
        float2 p = fma2(g, both(-1.f / 720.f), both(-1.f / 120.f));
        p = fma2(g, p, both(-1.f / 24.f));
        p = fma2(g, p, both(-1.f / 6.f));
        p = fma2(g, p, both(-0.5f));
        p = fma2(g, p, both(-1.f));
        p = mul2(g, p);
        m = make_float2(fabsf(g.x) < 0.25f ? p.x : 1.f - a.x, fabsf(g.y) < 0.25f ? p.y : 1.f - a.y);
        if (INPUT == kUnit) {
            const float2 s2 = mul2(m, add2(a, both(1.f)));
            m = make_float2(sqrt_hw(s2.x), sqrt_hw(s2.y));
        }
    } else {
        // a = 1 / (1 + e), m = e / (1 + e) with e = e^-g, kept at 2^126 and below; there a is made zero by a difference that no
        // a above 2^-102 notices. s = sqrt(e) sqrt((1 + a) / (1 + e)), since e itself may be too small for a number.
        const float2 t = mul2(g, both(INPUT == kUnit ? -0.5f * kLog2e : -kLog2e));
        constexpr float most = INPUT == kUnit ? 63.f : 126.f;
        const float2 x = make_float2(exp2_hw(min_nan(t.x, most)), exp2_hw(min_nan(t.y, most)));
        const float2 e = INPUT == kUnit ? mul2(x, x) : x;
        const float2 d = add2(e, both(1.f));
        const float2 r = make_float2(recip_hw(d.x), recip_hw(d.y));
        a = add2(r, both(-0x1p-126f));
        if (!WANT_M) return;
        if (INPUT == kUnit) {
            const float2 q = fma2(r, a, r);
            m = mul2(x, make_float2(sqrt_hw(q.x), sqrt_hw(q.y)));
        } else {
            m = mul2(e, r);
        }
    }
}

// s x, from decay's m
template <int INPUT> __device__ __forceinline__ float2 entering(float2 m, float2 x) { return INPUT == kPlain ? x : mul2(m, x); }

// Tokens behind a sequence's last one are made to leave the state alone: x = 0 and a gate of a = 1. TMA fills them with
// zeros, which is that gate in logarithms.
template <int GATE> __device__ __forceinline__ float open_gate() { return GATE == kLog ? 0.f : __int_as_float(0x7f800000); }

// ---- two channels of a row
template <class E> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 load(const void* row, int lane) {
        const uint32_t v = static_cast<const uint32_t*>(row)[lane];
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ void store(void* row, int lane, float2 v) {
        static_cast<uint32_t*>(row)[lane] = sm100::pack_bf16(v.x, v.y);
    }
    static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Pair<float> {
    static __device__ __forceinline__ float2 load(const void* row, int lane) { return static_cast<const float2*>(row)[lane]; }
    static __device__ __forceinline__ void store(void* row, int lane, float2 v) { static_cast<float2*>(row)[lane] = v; }
    static __device__ __forceinline__ float one(float v) { return v; }
};

// Where a lane writes its two channels, token by token. Rows start on 16 bytes, so a pair is aligned.
template <class E> struct Writer {
    E* p;
    long long st;
    bool two, one;                 // both channels are there, or the first alone
    __device__ __forceinline__ Writer(const Out& o, long long b, long long t, int c0, int D)
        : p(static_cast<E*>(o.p) + b * o.sb + t * o.st + c0), st(o.st), two(o.p && c0 + 1 < D), one(o.p && c0 + 1 == D) {}
    __device__ __forceinline__ void write(int i, bool in, float2 v) const {
        E* q = p + i * st;
        if (in && two) Pair<E>::store(q, 0, v);
        if (in && one) *q = Pair<E>::one(v.x);
    }
};

}  // namespace gr
}  // namespace dplr
