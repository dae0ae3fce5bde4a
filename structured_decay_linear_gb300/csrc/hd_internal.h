// Linear attention with one decay per head: what its translation units share (not part of the ABI).
//
// Everything, gradients included, is one operator on three row sequences x, y (DX features) and z (DZ features):
//
//   forward in time    o_t = R_t^T x_t,  R_t = e^{g_t} R_{t-1} + y_t z_t^T
//   backward in time   o_t = R_t^T x_t,  R_t = e^{g_{t+1}} R_{t+1} + y_t z_t^T
//
// The prompt is (x, y, z) = (q, k, v) forward. With dS_t the gradient of the state after token t, dq_t = S_t dO_t is
// (dO, v, k) forward (its state is S^T), dk_t = dS_t v_t is (v, dO, q) backward (state dS^T) and dv_t = dS_t^T k_t is
// (k, q, dO) backward (state dS), because dS_t = e^{g_{t+1}} dS_{t+1} + q_t dO_t^T.
//
// A sequence is cut into segments. Segment i starts (forward) from the boundary state i and ends at boundary i + 1;
// backward it starts from boundary i + 1. "States" passes form each segment's own contribution, a scan turns these
// into the boundary states, and "outputs" passes compute every segment from its boundary state.
#pragma once

#include <initializer_list>

#include "dplr_internal.h"

namespace dplr {
namespace hd {

constexpr int kChunk = 128;           // tokens that the tensor-core kernels compute together
constexpr float kMinGate = -128.f;    // log-gates below this act like it: e^-128 is zero in fp32

// Sums of gates are formed in fixed point, 40 fractional bits of 64: with 32, gates of some 1e-10 became zero or twice what
// they are, and a state that 2^21 such tokens had passed was off by 1.7e-4 (2^22: 3.3e-4). A chunk's sum stays below 2^15
// (a token's below 185), and a sum over chunks is kept above -kForgotten, at which its exponential has long been zero.
constexpr float kGateUnits = 1099511627776.f, kGateUnit = 9.094947017729282e-13f;     // 2^40 and 2^-40
constexpr long long kForgotten = 1LL << 52;                                           // 4096

// Whether an output starts where an input or another output does: a result fed back into the object that holds it, which
// the kernels would overwrite while others still read it.
inline bool taken(std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs) {
    for (auto o = outputs.begin(); o != outputs.end(); ++o) {
        if (!*o) continue;
        for (const void* p : inputs)
            if (p == *o) return true;
        for (auto p = outputs.begin(); p != o; ++p)
            if (*p == *o) return true;
    }
    return false;
}

// Kernels of one call are launched so that the next begins while the one before still runs (programmatic dependent launch):
// it sets itself up and reads the caller's inputs, and calls wait_for_kernel_before() in front of the first access to
// anything that an earlier kernel of the call writes or reads for the last time. The first kernel of a call is an ordinary
// launch. (Between two kernels of a call there were 5 us.)
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_kernel(void (*f)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, bool follows, A&&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&c, f, static_cast<P>(args)...);
}

// One row sequence: element (b, h, t, i) at p + b sb + (h / div) sh + t st + i.
struct View {
    const void* p;
    long long sb, sh, st;
    int div;
};

// Which (batch, head, segment) a CTA works on.
struct Geometry {
    int H;
    int T;                  // tokens of a sequence (dense)
    int nseg, L;            // dense: segments of a sequence, tokens of a segment
    const int* blocks;      // packed: [.][4] request, first row, rows, index in the request; null: dense
    const int* block_starts;   // [R + 1]
    int R;
    const int* slots;
    const int* context;
    int n_slots;
};

struct Segment {
    int b, h, t0, n;
    bool alone;             // the sequence has one segment: its boundary states are the caller's
    bool first, last;
    bool fresh;             // packed: the request starts from zero
    long long ext;          // index of the sequence's state in the caller's arrays
    long long entry;        // index of boundary state "segment start" in the boundary array; the next is entry + step
    long long step;
};

__host__ __device__ inline long long units(const Geometry& g, int B, int max_blocks) {
    return g.blocks ? (long long)max_blocks * g.H : (long long)B * g.H * g.nseg;
}

// False: nothing to do: a block behind the last (s is as it was), or one of a request whose slot has been changed to one out of
// range since the tables were made (s.n is its tokens). KEEP: that one stays, without tokens and without a state to leave.
template <bool KEEP = false>
__device__ __forceinline__ bool locate(const Geometry& g, int unit, Segment& s) {
    if (g.blocks) {
        const int blk = unit / g.H;
        s.h = unit % g.H;
        const int4 e = *reinterpret_cast<const int4*>(g.blocks + 4 * (long long)blk);
        if (e.x < 0) return false;
        const int nb = g.block_starts[e.x + 1] - g.block_starts[e.x];
        s.b = 0; s.t0 = e.y; s.n = e.z;
        s.alone = nb == 1; s.first = e.w == 0; s.last = e.w == nb - 1;
        s.fresh = g.context[e.x] == 0;
        const int slot = g.slots[e.x];
        const bool in = slot >= 0 && slot < g.n_slots;
        if (KEEP) {
            s.n = in ? e.z : 0;
            s.last = in && e.w == nb - 1;
        }
        s.ext = (long long)(in ? slot : 0) * g.H + s.h;
        s.entry = (long long)blk * g.H + s.h;
        s.step = g.H;
        return KEEP || in;
    }
    const int bh = unit / g.nseg, seg = unit % g.nseg;
    s.b = bh / g.H; s.h = bh % g.H;
    s.t0 = seg * g.L;
    s.n = min(g.L, g.T - s.t0);
    s.alone = g.nseg == 1; s.first = seg == 0; s.last = seg == g.nseg - 1;
    s.fresh = false;
    s.ext = bh;
    s.entry = (long long)bh * (g.nseg + 1) + seg;
    s.step = 1;
    return true;
}

// One pass over the segments. Its state is [DX][DZ]; the caller's states (ext) and the boundary states (bound) are arrays of
// such matrices, or `turned` of their transposes [DZ][DX].
struct Pass {
    View x, y, z;
    const float* g; long long gb, gh, gt;   // log-gates (0 strides: one per head)
    int reverse;
    int DX, DZ;
    int ext_turned, bound_turned;
    const float* ext_in;     // the caller's initial (backward in time: final) states, nullable
    float* ext_out;          // outputs pass: where the last segment leaves its state, nullable
    float* bound;            // boundary states (null: every sequence has one segment)
    float* gsum;             // states pass: sum of the segment's gates, at the segment's entry
    // outputs
    void* o; long long ob, oh, ot; int o_f32;
    // dots: per token sum_j o_j w_j with w like z, at dots[zb * B * H * T + (b * H + h) * T + t]; null: none
    View w; float* dots;
    int states_only;         // 1: states pass without the segment whose contribution no boundary needs; 2: with it
};

struct Launch {
    Geometry geo;
    int B, bf16;
    int max_blocks;          // packed
    int npass;
    Pass pass[3];
    int* status;             // the workspace's status word; the word 16 behind it counts a ragged batch's units
    long long wait_cycles;
    int follows;             // another kernel of the call goes before
    const int* order;        // packed, outputs on the tensor cores: the blocks, longest first; null: as they come
};

cudaError_t launch_decode(const View& q, const View& k, const View& v, const float* g, long long gb, long long gh,
                          float* S, const int* slots, int nslots, int B, int H, int dk, int dv, bool bf16, void* o,
                          long long ob, long long oh, int* status, cudaStream_t s);

// CUDA-core kernels (any type and size), 64-column (or 32) blocks of the state per CTA.
int fp32_zblock(int DZ);
cudaError_t launch_fp32(const Launch& a, cudaStream_t s);

// Tensor-core kernels: bf16, head sizes 64 and 128; one CTA per segment of one (batch, head).
bool tc_supported(bool bf16, int dk, int dv);
cudaError_t launch_tc(const Launch& a, cudaStream_t s);

// A ragged batch's blocks in falling order of their chunks, and its unit counter set to zero.
cudaError_t launch_order(const Geometry& g, int max_blocks, int* order, int* counter, cudaStream_t s);

// Turns segments' own contributions into boundary states, in place. Forward: the contribution of segment i lies at
// boundary i + 1, and boundary 0 is ext (or zero); backward: that of segment i at boundary i, boundary nseg is ext.
// Both arrays may be given (the gradient's two scans in one launch). `upto_end`: forward goes on to boundary nseg.
struct Scan {
    Geometry geo;
    int B, R, dk, dv;
    float* fwd; const float* fwd_ext; int upto_end;
    float* bwd; const float* bwd_ext;
    int turned;              // the boundary states are [dv][dk], the ext states [dk][dv]
    const float* gsum;
};
cudaError_t launch_scan(const Scan& a, cudaStream_t s);      // (follows the states pass)

// ddecay from the per-token dots and the boundary states: with a_t = q_t . dq_t - k_t . dk_t and e the end of t's segment,
//   ddecay_t = sum_{s=t..e} a_s + <S_e, dS_e>
// (the contributions of pairs of tokens on the same side of t cancel in the sum; segments keep what cancels short).
struct GateGrad {
    int B, H, T, nseg, L, dk, dv;
    const float* dq_dots; int nq;          // [nq][B*H*T]: partial sums over column blocks
    const float* dk_dots; int nk;
    const float* fwd; const float* bwd;    // boundary states; null: one segment
    int last_end;                          // whether <S_T, dS_T> counts (dST given)
    const float* S_T; const float* dST;    // one segment with last_end: the two states
    float* dg_token;                       // [B,H,T], null with per_head
    double* seg_sum;                       // [B*H*nseg] with per_head
    float* dg_head;                        // [H] with per_head
};
cudaError_t launch_gate_grad(const GateGrad& a, cudaStream_t s);

// Gradients of shared query/key heads: out[b, hq, t] = sum over hq's value heads of part [B,H,T,D] (fp32), in head order.
struct GroupSum {
    int B, H, Hq, T, D, bf16;
    struct One {
        const float* part;
        void* out; long long ob, oh, ot;
    } one[2];                // dq and dk
};
cudaError_t launch_group_sum(const GroupSum& a, cudaStream_t s);

}  // namespace hd
}  // namespace dplr
