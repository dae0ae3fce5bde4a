// Forward of the elementwise gated recurrence, dense and ragged: one pass over the data.
//
// A persistent CTA draws tiles of kCols channels x TT tokens. TMA brings the tile's x and g into one of S stages of shared
// memory ahead of time. Eight warps take 2 L tokens each, a lane two channels of one half of them: a local scan gives each
// half's map and leaves a and s x in registers; once the state in front of the tile is known (gr_chain.cuh) the tokens are
// gone through again. x, g are read once and y is written once: HBM is what bounds a call with many channels. Two CTAs an SM
// let one compute while the other waits for its predecessors.
//
// Measured at D 2048, 16-bit inputs (bytes of x, g and y; the copy rate is 6.79 TB/s): B8 T8192 with 16-bit log-gates 122 us,
// 6.6 TB/s; with sigmoid gates and the complement 127 us, 6.3; with 32-bit gates and the unit form 156 us, 6.9. One sequence
// of 131072 tokens takes 309 us, 5.2 TB/s: its 64 groups of channels are five to a round of CTAs, and a round waits for its
// own chain, 2.9 us; gr_roles.cu does better there (269 us). What did not shorten that: tiles of 64 or 128 tokens, 16
// channels, one CTA of 16 warps, clusters that exchange their maps on chip (377 us), all warps forming the next tile's map in
// front of this one's outputs (344 us). Ragged, sigmoid gates: 32 requests to 2000 tokens 102 us, 3.9 TB/s, the same chain with a row's
// marks besides; with gr_roles.cu's roles 113 us, since warps with a start or an end go a slower way twice (with log-gates they
// would take 82 instead of 92 us for 32 requests of 1000). With 32-bit gates 110 us, 4.8 TB/s, all in 32 bits 155 us, 5.1.
//
// y replaces x in shared memory and leaves by TMA; with 32-bit gates, whose stages are large and few, each lane writes it, and
// the stage is free after the first of the two rounds (B8 T8192 D2048: 156 instead of 169 us; with three smaller stages it
// would take 129 instead of 122 us, sigmoid gates 141 instead of 127 us: more instructions).
//
// Ragged batches are one long sequence of rows: a request's first token has a = 0 and its starting state in b, so requests
// of any lengths share tiles and nothing is padded.
#pragma once

#include "gr_chain.cuh"

namespace dplr {
namespace gr {
namespace {

// Stages of x and g: three of 32 KB, with 32-bit gates of 16-bit inputs two of 48 KB.
template <class XT, class GT> struct Shape {
    static constexpr int TT = forward_tile(sizeof(XT) == 2), L = TT / (kWarps * kRuns);
    static constexpr int XR = kCols * (int)sizeof(XT), GR = kCols * (int)sizeof(GT);    // bytes of a token
    static constexpr int XB = TT * XR, SB = TT * (XR + GR);
    static constexpr int S = 196608 / kCtas / SB;
    static constexpr bool DIRECT = sizeof(GT) != sizeof(XT);
    static constexpr int bytes = S * SB + 128;
};

// What a ragged batch's row says of its request.
constexpr unsigned kStarts = 1u << 20, kHasState = 1u << 21, kEnds = 1u << 22;
constexpr unsigned kSlotMask = kStarts - 1;

// Whether a request's first row is `row`.
__device__ __noinline__ bool is_first_row(const int* starts, int R, int row) {
    int lo = 0, hi = R;                        // the first of starts that is not in front of the row lies in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] < row) lo = mid + 1; else hi = mid;
    }
    return starts[lo] == row;
}

template <class XT, class GT, int GATE, int INPUT, bool PACKED>
__global__ void __launch_bounds__(kThreads, kCtas)
gr_forward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                  const __grid_constant__ CUtensorMap my, const __grid_constant__ ForwardArgs a) {
    using Sh = Shape<XT, GT>;
    constexpr int TT = Sh::TT, L = Sh::L, S = Sh::S, XR = Sh::XR, GR = Sh::GR;
    constexpr bool DIRECT = Sh::DIRECT;
    static_assert(!PACKED || TT <= kThreads, "a thread a row");
    static_assert(DIRECT ? S >= 2 : S >= 3, "the next tile is known before this one is done");
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    __shared__ uint64_t full[S];
    __shared__ int4 drawn[S];                  // tile in time (-1: none), batch entry, group of channels
    __shared__ __align__(16) float aggA[kWarps][kCols], aggB[kWarps][kCols];      // each warp's map; read in pairs
    __shared__ __align__(16) float preA[kWarps][kCols], preB[kWarps][kCols];      // the map of the warps in front of each
    __shared__ __align__(16) float carry[kCols];                                  // the state in front of the tile
    __shared__ float2 stash[kBatch * (kBatches - 1)][kCols];
    __shared__ unsigned marks[2][PACKED ? TT : 1];      // of this tile, and of the one that some warps may still write
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int li = lane % 16, run = w * kRuns + lane / 16, t0 = run * L;    // two channels of a run of L tokens
    const Dims d = a.c.d;
    const int BG = d.B * d.G;
    const int total = PACKED ? min(max(a.starts[a.R], 0), d.T) : d.T;
    const int NT = PACKED ? (total + TT - 1) / TT : d.NT;
    const unsigned tiles = (unsigned)NT * BG;
    const unsigned long long stamp = 4 * (__ldcg(&a.c.head->epoch) + 1);

    auto draw = [&](int s, unsigned tile) {
        if (tile >= tiles) { drawn[s].x = -1; return; }
        const int j = tile / BG, r = tile - j * BG, b = r / d.G, cg = r - b * d.G;
        drawn[s] = make_int4(j, b, cg, 0);
        sm100::mbar_expect_tx(&full[s], Sh::SB);
        tile_load<TT, XR>(sm + s * Sh::SB, &mx, cg * kCols, j * TT, b, &full[s]);
        tile_load<TT, GR>(sm + s * Sh::SB + Sh::XB, &mg, cg * kCols, j * TT, b, &full[s]);
    };
    if (tid == 0) {
        for (int s = 0; s < S; ++s) sm100::mbar_init(&full[s], 1);
        sm100::mbar_fence_init();
        draw(0, atomicAdd(&a.c.head->ticket, 1u));
    }
    __syncthreads();
    if (tid == 0)                              // while the first tile is on its way
        for (int s = 1; s < (DIRECT ? S : S - 1); ++s) draw(s, atomicAdd(&a.c.head->ticket, 1u));
    bool lost = false;
    // A thread's row of tile j, and what its neighbours say of it.
    auto mark = [&](int j, unsigned* to) {
        const int row = j * TT + tid;
        unsigned f = 0;
        if (j >= 0 && tid < TT && row < total) {
            const int me = a.slot[row], place = a.pos[row];
            const int before = row > 0 ? a.slot[row - 1] : -1, behind = row + 1 < total ? a.slot[row + 1] : -1;
            const bool good = me >= 0 && me < a.n_slots;
            f = good ? (unsigned)me : 0u;
            if (me != before) f |= kStarts | (good && place > 0 ? kHasState : 0u);
            if (me != behind && good) f |= kEnds;
            if (!good) {                       // neighbours may have the same slot
                if (is_first_row(a.starts, a.R, row)) f |= kStarts;
                a.c.head->status = DPLR_ERR_INVALID_ARG;
            }
        }
        if (tid < TT) to[tid] = f;
    };
    const unsigned* rows = marks[0];
    if (PACKED) {
        mark(drawn[0].x, marks[0]);
        __syncthreads();
    }
    for (int s = 0, phase = 0, turn = 0;; turn ^= 1) {
        const int4 tile = drawn[s];
        const int j = tile.x, b = tile.y, cg = tile.z;
        if (j < 0) break;
        unsigned next = 0;
        if (tid == 0) next = atomicAdd(&a.c.head->ticket, 1u);
        const int nv = min(TT, total - j * TT);                 // tokens of this tile
        const int c0 = cg * kCols + 2 * li;                   // this lane's channels in the scan
        // the last warp looks after the chain, a channel a lane; the first one's thread 0 after the copies
        const bool chains = tid >= kThreads - kCols;
        const int cc = tid - (kThreads - kCols), ch = cg * kCols + cc;
        Walk wk;
        Record* rec = a.c.rec + ((long long)(b * d.G + cg) * d.NT) * kCols + cc;
        Ahead ahead;
        if (chains) {
            wk.rec = rec; wk.from = j - 1; wk.step = -1; wk.NT = NT; wk.end = NT; wk.stamp = stamp;
            // read for the first tile alone, whose state is every other's: h_T may then be written in h0's place
            wk.outer = !PACKED && j == 0 && a.h0 && ch < d.D ? a.h0[(long long)b * d.D + ch] : 0.f;
            ahead.start(wk, a.c.far);
        }
        unsigned starts = 0, ends = 0;                          // tokens of this lane's half at which a request starts or ends
        if (PACKED) {
            rows = marks[turn];
            const unsigned f = lane % 16 < L ? rows[t0 + lane % 16] : 0u;
            starts = __ballot_sync(0xffffffffu, f & kStarts);
            ends = __ballot_sync(0xffffffffu, f & kEnds);
        }
        const unsigned any_start = starts | (starts >> 16), any_end = ends | (ends >> 16);
        starts >>= lane & 16;
        ends >>= lane & 16;
        // the state that the first of them starts from
        const int first_start = __ffs(starts & 0xffffu) - 1;
        float2 from_pool = both(0.f);
        if (PACKED && first_start >= 0) {
            const unsigned f = rows[t0 + first_start];
            const float* S0 = a.pool + (long long)(f & kSlotMask) * d.D + c0;
            if ((f & kHasState) && c0 < d.D) from_pool.x = __ldcg(S0);
            if ((f & kHasState) && c0 + 1 < d.D) from_pool.y = __ldcg(S0 + 1);
        }
        if (!sm100::mbar_wait(&full[s], phase)) lost = true;
        uint8_t* X = sm + s * Sh::SB;
        uint8_t* Gt = X + Sh::XB;
        if (nv < TT && (PACKED || GATE != kLog)) {              // behind the last token
            for (int t = max(nv, t0); t < t0 + L; ++t) {        // a lane's own
                if (PACKED) Pair<XT>::store(X + t * XR, li, make_float2(0.f, 0.f));
                Pair<GT>::store(Gt + t * GR, li, both(open_gate<GATE>()));
            }
            if (DIRECT) sm100::fence_async_smem();
        }
        // each warp's map
        float2 av[L], bv[L], A = both(1.f), H = both(0.f);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int t = t0 + i;
            const float2 g = Pair<GT>::load(Gt + t * GR, li), x = Pair<XT>::load(X + t * XR, li);
            float2 m;
            decay<GATE, INPUT, INPUT != kPlain>(g, av[i], m);
            bv[i] = entering<INPUT>(m, x);
            if (!PACKED) {
                A = mul2(A, av[i]);
                H = fma2(av[i], H, bv[i]);
            }
        }
        if (PACKED) {
            if (any_start) {                                    // a request starts in one of the warp's runs: a = 0, its state in b
                if (__any_sync(0xffffffffu, starts & (starts - 1) & 0xffffu)) {     // several in a run: all but the first one's states
#pragma unroll
                    for (int i = 1; i < L; ++i) {
                        const unsigned f = (starts >> i) & 1u && i != first_start ? rows[t0 + i] : 0u;
                        if (f & kHasState) {
                            const float* S0 = a.pool + (long long)(f & kSlotMask) * d.D + c0;
                            if (c0 < d.D) bv[i].x = fmaf(av[i].x, __ldcg(S0), bv[i].x);
                            if (c0 + 1 < d.D) bv[i].y = fmaf(av[i].y, __ldcg(S0 + 1), bv[i].y);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < L; ++i) {                   // selections, no branches: others wait for this tile
                    const bool start = (starts >> i) & 1u;
                    if (i == first_start) bv[i] = fma2(av[i], from_pool, bv[i]);
                    if (start) av[i] = both(0.f);
                    A = mul2(A, av[i]);
                    H = fma2(av[i], H, bv[i]);
                    if (start) { A = both(kReset); H = bv[i]; }    // whatever came before
                }
            } else {
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    A = mul2(A, av[i]);
                    H = fma2(av[i], H, bv[i]);
                }
            }
        }
        float2 Ax, Hx;
        join_runs<false, PACKED>(A, H, Ax, Hx, lane);
        if (lane >= 16) {                            // the warp's last run knows all
            reinterpret_cast<float2*>(aggA[w])[li] = A;
            reinterpret_cast<float2*>(aggB[w])[li] = H;
        }
        // a tile in which a request starts has its last state from itself
        const bool own_end = PACKED ? __syncthreads_or(any_start & 0xffffu) : (__syncthreads(), false);
        if (tid == 0) {                                         // into this stage, or that of the tile before, whose y has left by now
            if (!DIRECT) stores_read();
            draw(DIRECT ? s : s == 0 ? S - 1 : s - 1, next);
        }
        if (chains) {
            float At = 1.f, Ht = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float Av = aggA[v][cc];
                preA[v][cc] = At;
                preB[v][cc] = Ht;
                At = joined<PACKED>(Av, At);
                Ht = after<PACKED>(Av, Ht, aggB[v][cc]);
            }
            Record* mine = rec + (long long)j * kCols;
            if (own_end && j + 1 < NT) store_record(mine, 0.f, Ht, stamp | kState);
            auto publish = [&] { if (!own_end && j + 1 < NT) store_record(mine, At, Ht, stamp | kMap); };
            bool gave_up = false;
            const float h = walk<PACKED>(wk, ahead, a.c.far, &stash[0][cc], a.c.wait_cycles, publish, &gave_up);
            lost |= gave_up;
            const float end = after<PACKED>(At, h, Ht);
            if (j + 1 < NT) { if (!own_end) store_record(mine, 0.f, end, stamp | kState); }
            else if (!PACKED && a.hT && ch < d.D) a.hT[(long long)b * d.D + ch] = end;
            carry[cc] = h;
        }
        // the next tile's rows, while the chain's warp is at it
        if (PACKED) mark(drawn[s + 1 == S ? 0 : s + 1].x, marks[turn ^ 1]);
        __syncthreads();
        // the tokens from the state in front of them
        const float2 pa = reinterpret_cast<const float2*>(preA[w])[li], pb = reinterpret_cast<const float2*>(preB[w])[li];
        float2 h = reinterpret_cast<const float2*>(carry)[li];
        h = make_float2(after<PACKED>(pa.x, h.x, pb.x), after<PACKED>(pa.y, h.y, pb.y));
        h = make_float2(after<PACKED>(Ax.x, h.x, Hx.x), after<PACKED>(Ax.y, h.y, Hx.y));
        if (!PACKED && a.states && t0 % kStateStep == 0) {
            const int ns = (d.T + kStateStep - 1) / kStateStep, at = (j * TT + t0) / kStateStep;
            if (at < ns) {
                float* p = a.states + ((long long)b * ns + at) * d.D + c0;
                if (c0 < d.D) p[0] = h.x;
                if (c0 + 1 < d.D) p[1] = h.y;
            }
        }
        const Writer<XT> out(a.y, b, (long long)j * TT + t0, c0, d.D);
        if (PACKED && (any_start | any_end)) {
            const int last_end = 31 - __clz(ends & 0xffffu);    // -1: none
            float2 left = both(0.f);
            const bool several = __any_sync(0xffffffffu, ends & 0xffffu & ~(1u << (last_end & 31)));
            auto leave_state = [&](int i, float2 v) {
                float* p = a.pool + (long long)(rows[t0 + i] & kSlotMask) * d.D + c0;
                if (c0 < d.D) p[0] = v.x;
                if (c0 + 1 < d.D) p[1] = v.y;
            };
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int t = t0 + i;
                const float2 going = fma2(av[i], h, bv[i]);
                h = (starts >> i) & 1u ? bv[i] : going;
                if (DIRECT) out.write(i, t < nv, h);
                else Pair<XT>::store(X + t * XR, li, h);
                if (i == last_end) left = h;
                else if (several && ((ends >> i) & 1u)) leave_state(i, h);
            }
            if (last_end >= 0) leave_state(last_end, left);
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int t = t0 + i;
                h = fma2(av[i], h, bv[i]);
                if (DIRECT) out.write(i, t < nv, h);
                else Pair<XT>::store(X + t * XR, li, h);
            }
        }
        if (DIRECT) {
        } else if (PACKED && nv < TT) {                         // rows behind the last token stay as they are
            const Writer<XT> rows_out(a.y, b, (long long)j * TT, c0, d.D);
            __syncthreads();
            for (int t = run; t < nv; t += kWarps * kRuns) rows_out.write(t, true, Pair<XT>::load(X + t * XR, li));
            sm100::fence_async_smem();
            __syncthreads();
        } else {
            sm100::fence_async_smem();
            __syncthreads();
            if (tid == 0 && a.y.p) {
                tile_store<TT, XR>(&my, X, cg * kCols, j * TT, b, d.T);
                stores_commit();
            }
        }
        if (++s == S) { s = 0; phase ^= 1; }
    }
    if (lost) a.c.head->status = DPLR_ERR_TIMEOUT;
    __syncthreads();
    if (tid == 0) {
        stores_done();
        leave(a.c.head);
    }
}

template <class XT, class GT, int GATE, int INPUT, bool PACKED>
cudaError_t launch_one(const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y, const ForwardArgs& a, cudaStream_t s) {
    constexpr int bytes = Shape<XT, GT>::bytes;
    static std::atomic<uint64_t> done{0};
    const auto f = gr_forward_kernel<XT, GT, GATE, INPUT, PACKED>;
    const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(f), bytes, done);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.c.d.NT * a.c.d.B * a.c.d.G, most = (long long)kCtas * sm_count();
    f<<<(unsigned)(tiles < most ? tiles : most), kThreads, bytes, s>>>(x, g, y, a);
    return cudaGetLastError();
}

template <class XT, class GT, bool PACKED>
cudaError_t by_form(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y, const ForwardArgs& a,
                    cudaStream_t s) {
    switch (t.gate * 4 + t.input) {
        case kLog * 4 + kPlain: return launch_one<XT, GT, kLog, kPlain, PACKED>(x, g, y, a, s);
        case kLog * 4 + kComplement: return launch_one<XT, GT, kLog, kComplement, PACKED>(x, g, y, a, s);
        case kLog * 4 + kUnit: return launch_one<XT, GT, kLog, kUnit, PACKED>(x, g, y, a, s);
        case kSigmoid * 4 + kPlain: return launch_one<XT, GT, kSigmoid, kPlain, PACKED>(x, g, y, a, s);
        case kSigmoid * 4 + kComplement: return launch_one<XT, GT, kSigmoid, kComplement, PACKED>(x, g, y, a, s);
        case kSigmoid * 4 + kUnit: return launch_one<XT, GT, kSigmoid, kUnit, PACKED>(x, g, y, a, s);
    }
    return cudaErrorInvalidValue;
}

template <bool PACKED>
cudaError_t by_type(const Types& t, const CUtensorMap& x, const CUtensorMap& g, const CUtensorMap& y, const ForwardArgs& a,
                    cudaStream_t s) {
    if (!t.xbf16) return by_form<float, float, PACKED>(t, x, g, y, a, s);
    return t.gbf16 ? by_form<__nv_bfloat16, __nv_bfloat16, PACKED>(t, x, g, y, a, s)
                   : by_form<__nv_bfloat16, float, PACKED>(t, x, g, y, a, s);
}

}  // namespace
}  // namespace gr
}  // namespace dplr
