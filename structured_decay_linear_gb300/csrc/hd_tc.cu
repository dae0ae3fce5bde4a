// Linear attention with one decay per head on the tensor cores: bf16 rows, DX and DZ in {64, 128}, both directions of
// time, dense and ragged batches (hd_internal.h has the operator).
//
// One CTA walks a segment of one (batch, head) in chunks of 128 tokens and keeps the fp32 state R [DX][DZ] in tensor
// memory (lane i, column j) for the whole segment. G: inclusive cumulative log-gates of the chunk, n its tokens,
//   D  = X Y^T                                  (tcgen05 M = 128, N = 128, K = DX)
//   P  = D . e^{G_r - G_c} (c <= r)             (CUDA cores; back into tensor memory as bf16)    backward: e^{G_c - G_r}, c >= r
//   Op = P Z                                    (M = 128, N = DZ, K = 128; A in tensor memory)
//   Oi = X R                                    (M = 128, N = DZ, K = DX; R as bf16 in shared memory)
//   o  = e^{G_r} Oi + Op                        (CUDA cores)                                     backward: e^{G_n - G_r}
//   R <- e^{G_n} R + Y~^T Z, Y~_c = e^{G_n - G_c} y_c (M = DX, N = DZ, K = 128, fp32 accumulator) backward: Y~_c = e^{G_c} y_c
//
// Roundings. x, y, z are bf16 already: D is exact up to fp32 accumulation. Y~ enters the state, which is returned and
// carried over whole sequences in fp32, as two bf16 parts (hi + lo, 2^-17). P and the R in front of the readout are
// rounded to bf16 once: they only reach o, which is rounded to bf16 itself. Where per-token dots of the unrounded o
// are asked for (the gradient of the gates is a sum in which they nearly cancel), P and R have two parts too (SPLIT).
//
// Exponents. Sums of gates are formed in 64-bit fixed point (in units of log2) and kept as fp32 offsets from the start of blocks of
// 32 tokens, so that they are accurate however much was forgotten before. Within a diagonal 32 x 32 block of P the
// factor of a pair is one exponential; between blocks it is a product of three, each of a sum that is not positive
// (forward: row to its block's start, that start to the column block's end, that end to the column), two of them per
// token and one per pair of blocks: a quarter of the exponentials, and nothing overflows for any gate.
//
// Work split: groups of four warps (thread = lane of tensor memory) and three single warps:
//   A   the state: R to bf16 in shared memory, e^{G_n} R back      B1, B2  Y~ from Y, of the chunk's two halves
//   C   P from D                                                   O   o from Oi and Op
//   copies (TMA), MMA issue, gates
// The gate warp also says for each chunk what the others need to know of it; they only follow. Warps of a group do not
// wait for each other: each hands its part on by itself (a barrier of the group's threads took 300 cycles, several times
// a chunk). The issuer's order within a chunk, D Oi R Op, leaves the CUDA-core phases of a chunk under the other products.
// Each row sequence is read once by TMA in the 128-byte swizzle; the same tile serves K-major (D, Oi) and MN-major (Op,
// R) operands. A full chunk's o leaves by TMA from a tile of its own (16-byte stores of rows by lanes took 3.2 K cycles
// of the SM's store path); a ragged one, an fp32 one, and with SPLIT (whose second part of R takes the tile's place)
// every one is stored from registers.
//
// A pass for states only (the segments' own contributions) walks the chunks from the far end, so that the weights
// e^{(gates behind the token)} need no rescaling of R: its accumulator is touched by MMAs alone. Sixteen warps
// form Y~, and four bring finished states to memory while the next unit goes on in another accumulator.
//
// Bound: by the bytes of x, y, z and o (1 KB a token and head at 128 x 128): a chunk is 128 KB, 5.6 K cycles of its
// share of HBM bandwidth on 152 SMs, against 2.6 K cycles of products and about 2.5 K of each group's work, which their
// hand-offs string to a chain of about 5 K. Measured (bf16, 128 x 128, H 16): B8 T8192 178 us, 6.1 TB/s; B1 T32768 in 144
// segments: states 53 us, outputs 83 us, 6.4 TB/s; gradients of B4 T4096: states 65 us, dq and dk with SPLIT 153 us
// (5.7 us a chunk: the outputs' group, which also reads w), dv 71 us. With 64 columns or features (B8 H16 T8192: 159 and
// 152 us, 5.1 and 5.3 TB/s) the chain sets the time. One chunk alone: 10 us.
#include <cstring>
#include <type_traits>

#include "hd_internal.h"
#include "tc_common.cuh"

namespace dplr {
namespace hd {
namespace {

using namespace tc;

constexpr int C = kChunk;                  // 128
constexpr int kGrp = 128;
constexpr int kWorkers = 20;                // warps of the groups A (0-3), B1 (4-7), B2 (8-11), C (12-15), O (16-19)
constexpr int NT = 32 * kWorkers + 128;    // and warps 20 (copies), 21 (MMA issue), 22 (gates), 23 (none)
constexpr uint32_t kHalf = C * 128;        // bytes of a half tile: 128 rows of 64 bf16
constexpr uint32_t TM_R = 0, TM_D = 128, TM_OI = 256, TM_OP = 384, kTmemCols = 512;
constexpr double kLog2e = 1.4426950408889634;

struct alignas(128) Args {
    CUtensorMap map[3][4];    // [pass][x, y, z, o]
    Launch l;
    int total;                // units of work: segments times passes
    // A call's passes that differ in kind are launches that need the same states and nothing of each other. The first lets the
    // next begin once these are there (late), and that one waits for nothing (independent): its CTAs start on SMs as these get
    // done with the first, so that the two leave one ragged end, not two.
    int late, independent;
    int* counter;             // (outputs of a ragged batch) a CTA's first unit is blockIdx.x, all others come from here (0 at first)
};

// What the gate warp says of a chunk, double-buffered; A_i: cumulative gates at the start of block i of 32 tokens (log2
// units).
struct alignas(16) GateBuf {
    float rc[C];        // G_t minus its block's start
    float cf[C];        // forward e^{A_{i+1} - G_t}, backward e^{G_t - A_i}: a token as a column of P, and as a row of Y~
    float f[4][4];      // between row block i and column block j: forward e^{A_i - A_{j+1}}, backward e^{A_j - A_{i+1}}
    float bl[4];        // A_{i+1} - A_i
    float ce[4];        // Y~: times this. Forward e^{G_n - A_{i+1}}, backward e^{A_i} (a states pass: and the chunks between)
    float re[4];        // Oi: a row's factor times this. Forward e^{A_i}, backward e^{G_n - A_{i+1}}
    float en;           // e^{G_n}
    int n;              // tokens
    int flags;          // kFirst .. kEnd
    int t0, h, b;       // where its rows lie
    int pass;
    const float* src;   // first chunk: the state to start from (null: zero)
    float* dst;         // last chunk: where the state goes (null: nowhere)
    char* o;            // the head's first output row
    const __nv_bfloat16* w;
    float* dots;        // the head's
    long long ostep, wstep;
};
enum : int { kFirst = 1, kLast = 2, kRev = 4, kTurned = 8, kOutF32 = 16, kEnd = 32, kWide = 64, kOutTurned = 128 };   // kTurned: src;
                                                            // kOutTurned: dst; kWide: rows of o and w on 32 bytes
static_assert(sizeof(GateBuf) % 16 == 0, "16-byte rows");

template <int DX, int DZ, bool SPLIT, bool STATES>
struct Layout {
    static constexpr int XB = DX * 256, ZB = DZ * 256;        // bytes of a tile: D / 64 half tiles
    static constexpr int NZ = STATES ? 2 : 1;                 // z buffers
    static constexpr int NY = STATES ? 2 : 1;                 // y buffers (a states pass has no x)
    static constexpr int RB = STATES ? DX * 128 : DX * DZ * 2;  // R as bf16: DZ / 64 halves of DX rows of 128 bytes
    static constexpr int T_X = 0;
    static constexpr int T_Y = T_X + (STATES ? 0 : XB);
    static constexpr int T_YH = STATES ? T_Y : T_Y + NY * XB; // a states pass, which has no D, writes hi over y
    static constexpr int T_YL = T_YH + NY * XB;
    static constexpr int T_Z = T_YL + NY * XB;                // (a 64-feature Y~ read as M = 128 runs into what follows)
    static constexpr int T_R = T_Z + NZ * ZB;
    static constexpr int T_O = T_R + RB * (SPLIT ? 2 : 1);    // o on its way out
    static constexpr bool STAGED = !SPLIT && !STATES;
    // With 64 columns tensor memory has room for two Oi and two Op: the products of a chunk then do not wait for the outputs
    // of the one before.
    static constexpr bool TWO = DZ == 64 && !STATES;
    static constexpr int GATES = T_O + (STAGED ? ZB : 0);
    static constexpr int BARS = GATES + 2 * (int)sizeof(GateBuf);
    static constexpr int TOTAL = BARS + 256;   // 27 barriers, the address of the tensor memory, a unit's number
    static_assert(TOTAL <= 227 * 1024, "shared memory budget");
};

// Registers of a group's threads. The block is launched with 80 a thread (65536 / 768); B gives some up for C and O. With
// what is left of the L1 cache beside the tiles, a spilled register is read back from L2: 32 of them a chunk had doubled
// the time of the gradient passes.
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
constexpr int kRegsLaunch = 80, kRegsB = 64, kRegsC = 88, kRegsO = 104;
static_assert(2 * kRegsB + kRegsC + kRegsO <= 4 * kRegsLaunch, "the groups' shares come out of the launch's registers");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 4-D tiled copy: 64 features x 128 tokens of one head.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int t, int h, int b, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(t), "r"(h), "r"(b), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int t, int h, int b) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(t), "r"(h), "r"(b) : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int c0, int t, int h, int b, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(t), "r"(h), "r"(b), "r"(src) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 16 columns of two accumulators, both loads in flight at once.
__device__ __forceinline__ void tmem_ld16_pair(uint32_t ta, uint32_t tb, float (&x)[16], float (&y)[16]) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t* q = r + 16 * i;
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]),
              "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
            : "r"(i ? tb : ta));
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // no use of the values moves in front of the wait
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
#pragma unroll
    for (int i = 0; i < 16; ++i) { x[i] = __uint_as_float(r[i]); y[i] = __uint_as_float(r[16 + i]); }
}
// 32 bytes at once (addresses on 32 bytes): rows apart, a lane's access is then a whole sector.
__device__ __forceinline__ void ldg256(const void* p, uint4& x, uint4& y) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "l"(p));
}
__device__ __forceinline__ void stg256(void* p, uint4 x, uint4 y) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const float (&v)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
}

__device__ __forceinline__ void tmem_st32_nowait(uint32_t taddr, const float (&v)[32]) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
    tmem_st16(taddr + 16, r + 16);
}

// Sixteen bytes of a y row times the row's weight, as hi + lo.
__device__ __forceinline__ void scale16(const uint32_t (&u)[4], float w, uint32_t th, uint32_t tl) {
    const float2 w2 = make_float2(w, w);
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = __fmul2_rn(make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u)), w2);
        h[e] = pack_bf16(x.x, x.y);
        const float2 r = __ffma2_rn(make_float2(__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xFFFF0000u)),
                                    make_float2(-1.f, -1.f), x);
        l[e] = pack_bf16(r.x, r.y);
    }
    sts128(th, h[0], h[1], h[2], h[3]);
    sts128(tl, l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&u)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(addr));
}

// The y rows of a chunk times their weights, as hi + lo, by `nt` threads; rows from n on become zero whatever they hold.
template <int DX>
__device__ __forceinline__ void scale_rows(uint32_t ty, uint32_t th, uint32_t tl, const GateBuf& g, int n, int tid, int nt) {
    constexpr int PER = DX / 8;     // 16-byte pieces of a row
#pragma unroll 2
    for (int i = tid; i < C * PER; i += nt) {
        const int t = i / PER, c = i % PER;
        const uint32_t off = (uint32_t)(c >> 3) * kHalf + swz(t, c & 7);
        uint32_t u[4];
        lds128(ty + off, u);
        float w = g.cf[t] * g.ce[t >> 5];
        if (t >= n) u[0] = u[1] = u[2] = u[3] = 0u, w = 0.f;
        scale16(u, w, th + off, tl + off);
    }
}

// Rows r0 .. r1 - 1 of a z tile become zero: they may belong to another request and hold anything.
template <int DZ>
__device__ __forceinline__ void clear_rows(uint32_t tz, int r0, int r1, int tid, int nt) {
    constexpr int PER = DZ / 8;
    for (int i = r0 * PER + tid; i < r1 * PER; i += nt) {
        const int t = i / PER, c = i % PER;
        sts128(tz + (uint32_t)(c >> 3) * kHalf + swz(t, c & 7), 0u, 0u, 0u, 0u);
    }
}

// States in memory. A thread holds a row of the state, a warp 32 rows; lane by lane, 16-byte accesses to rows 512 bytes
// apart keep the SM's load path busy for 4 K cycles per state. So a warp moves 32 x 32 blocks with eight lanes to a row
// and turns them in 4 KB of shared memory of its own (the rows of the R tile that it alone writes).
__device__ __forceinline__ uint32_t turn_at(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Starts columns c .. c + 31 of the warp's 32 rows (first row r0) of a state [DX][DZ], or `turned` of one [DZ][DX], on
// their way to the 4 KB at `turn`; after copies_done() and a __syncwarp(), block_row() gives this lane's row.
template <int DX, int DZ>
__device__ __forceinline__ void start_block(const float* state, bool turned, int r0, int c, uint32_t turn) {
    const int lane = threadIdx.x & 31;
    if (!turned) {
        const float* src = state + (r0 + (lane >> 3)) * DZ + c + 4 * (lane & 7);
#pragma unroll
        for (int k = 0; k < 8; ++k) copy_async16(turn + turn_at(4 * k + (lane >> 3), lane & 7), src + 4 * k * DZ);
    } else {        // a column's 32 rows lie together: they stay so, and block_row() reads across
        const float* src = state + (c + (lane >> 3)) * DX + r0 + 4 * (lane & 7);
#pragma unroll
        for (int k = 0; k < 8; ++k) copy_async16(turn + (4 * k + (lane >> 3)) * 128 + 16 * (lane & 7), src + 4 * k * DX);
    }
}
__device__ __forceinline__ void block_row(uint32_t turn, bool turned, float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    if (turned) {
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(turn + 128 * i + 4 * lane));
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t u[4];
        lds128(turn + turn_at(lane, k), u);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = __uint_as_float(u[e]);
    }
}

template <int DX, int DZ>
__device__ __forceinline__ void store_block(float* state, bool turned, int r0, int c, uint32_t turn, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    if (!turned) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sts128(turn + turn_at(lane, k), __float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                   __float_as_uint(v[4 * k + 3]));
        __syncwarp();
        float* dst = state + (r0 + (lane >> 3)) * DZ + c + 4 * (lane & 7);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t u[4];
            lds128(turn + turn_at(4 * k + (lane >> 3), lane & 7), u);
            *reinterpret_cast<uint4*>(dst + 4 * k * DZ) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        __syncwarp();
    } else {
        float* dst = state + r0 + lane + c * DX;
#pragma unroll
        for (int i = 0; i < 32; ++i) dst[i * DX] = v[i];
    }
}

// The warp's rows of the state in tensor memory to an array of [DX][DZ] states.
template <int DX, int DZ>
__device__ __forceinline__ void store_state(float* state, bool turned, int r0, uint32_t turn, uint32_t taddr) {
#pragma unroll 1
    for (int c = 0; c < DZ; c += 32) {
        float v[32];
        tmem_ld32(taddr + c, v);
        store_block<DX, DZ>(state, turned, r0, c, turn, v);
    }
}

// One unit of work: a segment in a pass. A CTA takes u = blockIdx.x, + gridDim.x, ..; of a ragged batch the gate warp finds
// its units and names them to the copy warp. A CTA's chunks are numbered through, so that copies, gates and products of a
// unit run into those of the one before.
struct Work {
    const Pass* p;
    const CUtensorMap* maps;
    Segment sg;
    bool rev, down;
    int nchunk;
    __device__ __forceinline__ int chunk(int j) const { return down ? nchunk - 1 - j : j; }
    __device__ __forceinline__ int rows(int j) const { return min(C, sg.n - chunk(j) * C); }
};

// False: nothing to do.
template <bool STATES, bool RAGGED>
__device__ __forceinline__ bool find_work(const Args& a, int u, Work& w) {
    const int pi = u % a.l.npass;      // the passes of a segment side by side: they read the same rows
    w.p = &a.l.pass[pi];
    w.maps = a.map[pi];
    __builtin_assume(RAGGED == (a.l.geo.blocks != nullptr));
    int at = u / a.l.npass;
    if (RAGGED && !STATES && a.l.order) {
        if (at / a.l.geo.H >= a.l.geo.block_starts[a.l.geo.R]) return false;      // (the order ends with the batch's blocks)
        at = a.l.order[at / a.l.geo.H] * a.l.geo.H + at % a.l.geo.H;
    }
    // Each of a ragged batch's blocks is a unit of the outputs pass, which those who name it, copy its rows and follow count
    // on: a request whose slot has become bad is one chunk without tokens. (As a unit to be skipped it cost the gate warp
    // registers or the copy warp a wait for the slot: 32 requests of up to 2000 tokens 104 -> 107 to 110 us.)
    if (!locate<RAGGED && !STATES>(a.l.geo, at, w.sg)) return false;
    w.rev = w.p->reverse;
    if (w.p->states_only == 1 && (w.rev ? w.sg.first : w.sg.last)) return false;
    w.nchunk = RAGGED && !STATES ? max((w.sg.n + C - 1) / C, 1) : (w.sg.n + C - 1) / C;
    // chunk of step j: in the pass's direction; a states pass comes from the far end
    w.down = STATES ? !w.rev : w.rev;
    return w.nchunk > 0;
}

// The state a unit starts from (null: zero).
template <int DX, int DZ>
__device__ __forceinline__ const float* start_state(const Work& w) {
    const Pass& p = *w.p;
    if (p.bound && !w.sg.alone) return p.bound + (w.rev ? w.sg.entry + w.sg.step : w.sg.entry) * (long long)(DX * DZ);
    return p.ext_in && !w.sg.fresh ? p.ext_in + w.sg.ext * (long long)(DX * DZ) : nullptr;
}

// RAGGED: of a ragged batch, whose units are found in tables and shared out as the CTAs get done. A batch of equal lengths
// has its own variant: with the table's branches in the unit loop its passes took 3 % longer (B4 H16 T4096, gradients 349
// instead of 335 us).
template <int DX, int DZ, bool SPLIT, bool STATES, bool RAGGED>
__global__ void __launch_bounds__(NT, 1) hd_tc_kernel(const __grid_constant__ Args a) {
    using Ly = Layout<DX, DZ, SPLIT, STATES>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sb = smem_addr(smem);
    if (sb & 1023u) {   // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) atomicExch(a.l.status, (int)DPLR_ERR_CUDA);
        return;
    }

    // completed copies and products (one arrival each); parts handed on by warps (one arrival per warp)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::BARS);
    uint64_t* full_x = bars + 0;
    uint64_t* full_y = bars + 1;     // [2]
    uint64_t* full_z = bars + 3;     // [2]
    uint64_t* free_z = bars + 5;     // [2] Op of the chunk that used the buffer
    uint64_t* d_done = bars + 7;     // D
    uint64_t* oi_done = bars + 8;    // Oi
    uint64_t* r_half = bars + 9;     // R from the first 64 tokens
    uint64_t* r_done = bars + 10;    // R from all
    uint64_t* op_done = bars + 11;   // Op
    uint64_t* drain = bars + 12;
    uint64_t* g_full = bars + 13;    // [2] gates, one arrival
    uint64_t* g_free = bars + 15;    // [2] every worker warp and the issuer
    uint64_t* r_ready = bars + 17;   // A: R scaled, its bf16 copy written
    uint64_t* y_read = bars + 18;    // B1, B2: the y tile is in their registers
    uint64_t* y_ready = bars + 19;   // B1: Y~ of the first 64 tokens
    uint64_t* y_rest = bars + 20;    // B2: of the others
    uint64_t* p_ready = bars + 21;   // C: P
    uint64_t* o_free = bars + 22;    // O: Oi and Op read
    // A states pass has no halves, P or outputs: Y~ and R of even and odd chunks, stored states of even and odd units. (Two
    // barriers each: while the issuer waits for a state to be stored, Y~ of the next chunk may be handed on as well, and a
    // wait for a phase takes the one after the next for it.)
    // (chosen by arithmetic: an array of them goes to local memory, and its loads to L2)
    auto y_states = [=](uint32_t par) { return y_ready + par; };
    auto r_states = [=](uint32_t par) { return r_half + par; };
    auto state_out = [=](uint32_t par) { return p_ready + par; };
    uint64_t* u_full = bars + 23;    // gates: the next unit's number (-1: none)
    uint64_t* u_free = bars + 24;    // copies: taken
    // of even and odd chunks, where these have accumulators of their own
    auto o_frees = [=](uint32_t par) { return o_free + (Ly::TWO ? 3 * par : 0); };
    auto op_dones = [=](uint32_t par) { return op_done + (Ly::TWO ? 15 * par : 0); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 27);
    volatile int* next_unit = reinterpret_cast<volatile int*>(bars + 27) + 1;
    GateBuf* gates = reinterpret_cast<GateBuf*>(smem + Ly::GATES);

    // (what is the same for a warp goes through a shuffle, which tells the compiler so: branches on it then cost no
    // re-convergence, 100 cycles and more in a loop of a few hundred)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rw = warp & 3, row = tid & (kGrp - 1);     // a worker's 32 lanes of tensor memory, and this thread's
    const uint32_t lane_off = static_cast<uint32_t>(32 * rw) << 16;
    const long long wl = a.l.wait_cycles;

    if (tid == 0) {
        for (int i = 0; i < 27; ++i) {
            uint32_t n = 1;
            if (i == 15 || i == 16) n = kWorkers + 1;
            else if (STATES && (i == 19 || i == 20)) n = kWorkers - 4;
            else if (i == 17 || (i >= 19 && i <= 22) || i == 25) n = 4;
            else if (i == 18) n = 8;
            mbar_init(bars + i, n);
        }
        mbar_fence_init();
    }
    if (!a.late) let_next_kernel_begin();
    if (warp == 0) tmem_alloc(tmem_holder, kTmemCols);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    bool failed = false;

    // A bounded wait of a warp. One that gives up leaves its loop; the others run into their own limits.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, wl));
        fence_after_sync();
        return ok;
    };
    // Gives back a buffer that the warp's lanes have read: `seen` is formed from all that each lane loaded. Shared loads and
    // barrier arrivals take different ways, so an arrival issued behind a load may be seen before the load has read; the
    // vote waits for every lane's values, and which lane arrives depends on it.
    auto give_back = [&](uint64_t* bar, uint32_t seen) {
        const int who = __any_sync(0xffffffffu, seen == 0x9e3779b9u) ? 1 : 0;
        if (lane == who) mbar_arrive(bar);
    };
    // Hands on what the warp's lanes have written.
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp == 20) {
        // =================== copies ===================
        if (lane == 0) {
            uint32_t it = 0, nx = 0, ny = 0, nz = 0;    // chunks; copies started
            if (RAGGED && !STATES) wait_for_kernel_before();      // the order of the blocks
            constexpr bool by_name = RAGGED;       // all but the CTA's own number's, if that has work
            int u = blockIdx.x;
            for (uint32_t named = 0; !failed; u = by_name ? -1 : u + (int)gridDim.x) {
                Work w;
                if (!by_name) {
                    if (u >= a.total) break;
                    if (!find_work<STATES, RAGGED>(a, u, w)) continue;
                } else if (u < 0 || !find_work<STATES, RAGGED>(a, u, w)) {
                    if (!mbar_wait(u_full, named & 1, wl)) { failed = true; break; }
                    u = *next_unit;
                    if (u < 0) break;
                    mbar_arrive(u_free);       // (behind the branch: the load has returned)
                    ++named;
                    const bool found = find_work<STATES, RAGGED>(a, u, w);
                    if (STATES && !found) { failed = true; break; }      // (a slot that was changed since the unit was named)
                }
                const CUtensorMap* maps = w.maps;
                const int hx = w.sg.h / w.p->x.div, hy = w.sg.h / w.p->y.div, hz = w.sg.h / w.p->z.div, bb = w.sg.b;
                if (const float* src = !STATES && it > 0 ? start_state<DX, DZ>(w) : nullptr)    // (the first: A is about to load it)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(src), "r"(DX * DZ * 4) : "memory");
                for (int j = 0; j < w.nchunk; ++j, ++it) {
                    const int t = w.sg.t0 + w.chunk(j) * C;
                    const uint32_t s = it % Ly::NZ;
                    auto load = [&](uint32_t dst, int which, int D, int h, uint64_t* bar) {
                        mbar_expect_tx(bar, D * 256);
                        for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * kHalf, &maps[which], 64 * x, t, h, bb, bar);
                    };
                    if (STATES) {
                        if (it >= 2 && !mbar_wait(&free_z[s], ((it - 2) >> 1) & 1, wl)) { failed = true; break; }
                        load(sb + Ly::T_Y + s * Ly::XB, 1, DX, hy, &full_y[s]);
                    } else {
                        // Shared memory has room for one x, y and z tile: the rows start on their way into L2 while the
                        // buffers are still in use.
                        for (int x = 0; x < DX / 64; ++x) {
                            tma_prefetch_4d(&maps[1], 64 * x, t, hy, bb);
                            tma_prefetch_4d(&maps[0], 64 * x, t, hx, bb);
                        }
                        for (int x = 0; x < DZ / 64; ++x) tma_prefetch_4d(&maps[2], 64 * x, t, hz, bb);
                        // y once the D before is formed and its tile in registers, x once its Oi is, z once its Op is
                        if (it >= 1 && (!mbar_wait(d_done, (it - 1) & 1, wl) || !mbar_wait(y_read, (it - 1) & 1, wl))) { failed = true; break; }
                        load(sb + Ly::T_Y, 1, DX, hy, full_y);
                        ++ny;
                        if (it >= 1 && !mbar_wait(oi_done, (it - 1) & 1, wl)) { failed = true; break; }
                        load(sb + Ly::T_X, 0, DX, hx, full_x);
                        ++nx;
                        if (it >= 1 && !mbar_wait(free_z, (it - 1) & 1, wl)) { failed = true; break; }
                    }
                    if (STATES) ++ny;
                    load(sb + Ly::T_Z + s * Ly::ZB, 2, DZ, hz, &full_z[s]);
                    ++nz;
                }
                if (RAGGED && !STATES && w.sg.n == 0) atomicExch(a.l.status, (int)DPLR_ERR_INVALID_ARG);   // its slot is bad
            }
            if (failed) atomicExch(a.l.status, (int)DPLR_ERR_TIMEOUT);
            // no copy may land after the CTA has gone (another role may have given up): wait for the last into each buffer
            const long long most = 400000000LL;
            if (nx > 0) mbar_wait(full_x, (nx - 1) & 1, most);
            for (uint32_t s = 0; s < Ly::NY; ++s)
                if (ny > s) mbar_wait(&full_y[s], ((ny - 1 - s) / Ly::NY) & 1, most);
            for (uint32_t s = 0; s < Ly::NZ; ++s)
                if (nz > s) mbar_wait(&full_z[s], ((nz - 1 - s) / Ly::NZ) & 1, most);
        }
        __syncwarp();
    } else if (warp == 21) {
        // =================== MMA issue (lane 0; the others wait at the end) ===================
        if (lane == 0) {
            auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {
                const bool ok = mbar_wait(bar, parity, wl);
                fence_after_sync();
                return ok;
            };
            const uint32_t idD = idesc_bf16(128, C, false, false);
            const uint32_t idO = idesc_bf16(128, DZ, false, true);
            const uint32_t idR = idesc_bf16(128, DZ, true, true);
            auto mma_D = [&]() {
#pragma unroll 1
                for (int h = 0; h < DX / 64; ++h)
                    mma_chain(tmem + TM_D, smem_desc_sw128(sb + Ly::T_X + h * kHalf, 16, 1024), 32,
                              smem_desc_sw128(sb + Ly::T_Y + h * kHalf, 16, 1024), 32, idD, 64, h > 0);
                mma_commit(d_done);
            };
            auto mma_Oi = [&](uint32_t acc) {
#pragma unroll 1
                for (int i = 0; i < (SPLIT ? 2 : 1) * (DX / 64); ++i) {
                    const int h = i % (DX / 64), s = i / (DX / 64);
                    mma_chain(acc + TM_OI, smem_desc_sw128(sb + Ly::T_X + h * kHalf, 16, 1024), 32,
                              smem_desc_sw128(sb + Ly::T_R + s * Ly::RB + h * 64 * 128, DX * 128, 1024), 2048, idO, 64, i > 0);
                }
                mma_commit(oi_done);
            };
            uint32_t tm_r = tmem + TM_R;      // a states pass has two, in turn
            auto mma_R = [&](uint32_t buf, uint32_t tz, int half, bool acc) {      // 64 tokens: four slices of 2048 bytes
#pragma unroll 1
                for (int s = 0; s < 2; ++s)
                    mma_chain(tm_r, smem_desc_sw128(sb + (s ? Ly::T_YL : Ly::T_YH) + buf * Ly::XB + 8192 * half, kHalf, 1024), 2048,
                              smem_desc_sw128(tz + 8192 * half, kHalf, 1024), 2048, idR, 64, acc || s > 0);
            };
            auto mma_Op = [&](uint32_t acc, uint32_t tz) {
                const uint64_t dz = smem_desc_sw128(tz, kHalf, 1024);
#pragma unroll 1
                for (int s = 0; s < (SPLIT ? 2 : 1); ++s)
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)     // 16 tokens: 8 columns of P
                        mma_bf16_tmem_a(acc + TM_OP, tmem + TM_D + 32 * (ks >> 1) + 8 * (ks & 1) + 16 * s,
                                        dadd(dz, 2048 * ks), idO, (s > 0 || ks > 0) ? 1u : 0u);
            };
            [[maybe_unused]] uint32_t unit = 0;       // (states pass) units begun
            for (uint32_t it = 0;; ++it) {
                const uint32_t par = it & 1, s = it % Ly::NZ, zpar = (it / Ly::NZ) & 1;
                const uint32_t tz = sb + Ly::T_Z + s * Ly::ZB;
                if (!wait1(&g_full[par], (it >> 1) & 1)) { failed = true; break; }
                const int flags = gates[par].flags;
                if (flags & kEnd) break;
                mbar_arrive(&g_free[par]);       // (behind the branch: the load has returned)
                if (STATES) {
                    if (flags & kFirst) {      // the accumulator of the unit before the last: once it has been stored
                        if (unit >= 2 && !wait1(state_out(unit & 1), ((unit >> 1) - 1) & 1)) { failed = true; break; }
                        tm_r = tmem + TM_R + (unit & 1) * 128;
                        ++unit;
                    }
                    if (!wait1(y_states(par), (it >> 1) & 1) || !wait1(&full_z[s], zpar)) { failed = true; break; }
                    mma_R(s, tz, 0, !(flags & kFirst));
                    mma_R(s, tz, 1, true);
                    mma_commit(&free_z[s]);
                    mma_commit(r_states(par));
                    continue;
                }
                if (!wait1(full_x, par) || !wait1(full_y, par)) { failed = true; break; }
                mma_D();
                // its accumulators, once the outputs of the chunk that used them have been read
                const uint32_t acc = tmem + (Ly::TWO ? 64 * par : 0);
                const bool free = Ly::TWO ? it < 2 || wait1(o_frees(par), ((it - 2) >> 1) & 1) : it < 1 || wait1(o_free, par ^ 1);
                if (!free || !wait1(r_ready, par)) { failed = true; break; }
                mma_Oi(acc);
                if (!wait1(y_ready, par) || !wait1(&full_z[s], zpar)) { failed = true; break; }
                if (SPLIT) {      // O takes longest here: Op before R (z has been cleared once both halves of Y~ are there)
                    if (!wait1(y_rest, par) || !wait1(p_ready, par)) { failed = true; break; }
                    mma_Op(acc, tz);
                    mma_commit(op_dones(par));
                }
                mma_R(0, tz, 0, true);
                mma_commit(r_half);
                if (!SPLIT && !wait1(y_rest, par)) { failed = true; break; }
                mma_R(0, tz, 1, true);
                mma_commit(r_done);
                if (!SPLIT) {
                    if (!wait1(p_ready, par)) { failed = true; break; }
                    mma_Op(acc, tz);
                }
                mma_commit(&free_z[s]);
                if (!SPLIT) mma_commit(op_dones(par));
            }
            if (failed) atomicExch(a.l.status, (int)DPLR_ERR_TIMEOUT);
            mma_commit(drain);       // every MMA this thread issued: none may run on freed tensor memory
            mbar_wait(drain, 0, 400000000LL);
        }
        __syncwarp();
    } else if (warp == 22) {
        // =================== gates: lane holds tokens 4 lane .. 4 lane + 3 ===================
        // Sums in fixed point (units of log2, 40 fractional bits, 64 in all): exact, and unlike 64-bit floating point (with
        // which this warp took 6.6 K cycles a chunk and held up all others) a few integer instructions each.
        auto real = [](long long x) { return (float)x * kGateUnit; };
        uint32_t it = 0;
        auto take = [&]() -> GateBuf* {       // the next buffer, once its chunk before the last is done with
            const uint32_t b = it & 1;
            if (it >= 2 && !wait(&g_free[b], ((it - 2) >> 1) & 1)) { failed = true; return nullptr; }
            return gates + b;
        };
        if (RAGGED && !STATES) wait_for_kernel_before();
        // a ragged batch's blocks end before its table does
        int total = a.total;
        if (RAGGED) total = min(total, a.l.geo.block_starts[a.l.geo.R] * a.l.geo.H * a.l.npass);
        uint32_t named = 0;
        auto name = [&](int u) {          // tells the copy warp of a unit
            if (!RAGGED) return;
            if (named > 0 && !wait(u_free, (named - 1) & 1)) { failed = true; return; }
            if (lane == 0) *next_unit = u;
            arrive(u_full);
            ++named;
        };
        int unit = blockIdx.x, after = 0;
        for (bool begun = false; unit < total && !failed; unit = after, begun = true) {
            Work w;
            if (STATES && RAGGED) {      // most of a ragged batch's requests have one block and no boundary: 32 at a time
                Work v;
                const int mine = unit + lane * (int)gridDim.x;
                const uint32_t some = __ballot_sync(0xffffffffu, mine < total && find_work<STATES, RAGGED>(a, mine, v));
                if (some == 0) {
                    after = unit + 32 * (int)gridDim.x;
                    continue;
                }
                const int skip = __ffs(some) - 1;
                unit += skip * (int)gridDim.x;
                begun |= skip > 0;
            }
            after = unit + (int)gridDim.x;
            if (!STATES && RAGGED && lane == 0) after = (int)gridDim.x + atomicAdd(a.counter, 1);
            // An outputs pass has no unit without work: the next one is named as soon as this one's first chunk is out. In a
            // states pass a unit is named when it has been found to have some.
            const bool some = find_work<STATES, RAGGED>(a, unit, w);
            if (STATES && some && begun) name(unit);
            if (!some || failed) continue;
            const Pass& p = *w.p;
            const bool rev = w.rev;
            const long long gstep = p.gt;     // (in registers: the loops below would read the pass from memory again and again)
            const float* gp = p.g + w.sg.b * p.gb + w.sg.h * p.gh + w.sg.t0 * gstep;
            auto raw = [&](int j, float (&r)[4]) {
                const int n = w.rows(j);
                const int t0 = w.chunk(j) * C + 4 * lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = 4 * lane + i < n ? gp[(t0 + i) * gstep] : 0.f;
            };
            float cur[4], nxt[4];
            raw(0, cur);
            // what the others need to know of the unit
            const float* src = STATES ? nullptr : start_state<DX, DZ>(w);
            float* dst = nullptr;
            if (STATES) dst = p.bound + (rev ? w.sg.entry : w.sg.entry + w.sg.step) * (long long)(DX * DZ);
            else if (p.ext_out && (rev ? w.sg.first : w.sg.last)) dst = p.ext_out + w.sg.ext * (long long)(DX * DZ);
            const long long ostep = p.ot, wstep = p.w.st;
            char* o = static_cast<char*>(p.o) + (w.sg.b * p.ob + w.sg.h * p.oh) * (p.o_f32 ? 4 : 2);
            const __nv_bfloat16* wv = SPLIT ? static_cast<const __nv_bfloat16*>(p.w.p) + w.sg.b * p.w.sb + (w.sg.h / p.w.div) * p.w.sh : nullptr;
            float* dots = SPLIT ? p.dots + ((long long)w.sg.b * a.l.geo.H + w.sg.h) * a.l.geo.T : nullptr;
            float* gsum = STATES && p.gsum ? p.gsum + w.sg.entry : nullptr;
            const int kind = (rev ? kRev : 0) | ((p.bound && !w.sg.alone ? p.bound_turned : p.ext_turned) ? kTurned : 0) |
                             ((STATES ? p.bound_turned : p.ext_turned) ? kOutTurned : 0) | (p.o_f32 ? kOutF32 : 0) |
                             (((reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(wv)) & 31) == 0 && ((ostep | wstep) & 15) == 0 ? kWide : 0);
            long long passed = 0;    // gates of the chunks before
            float lost = 0.f;        // NaN once a gate was: it then reaches everything behind
            for (int j = 0; j < w.nchunk; ++j, ++it) {
                if (j + 1 < w.nchunk) raw(j + 1, nxt);
                long long x[4];
                bool nan = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    nan |= !(cur[i] <= 1e4f);        // (gates are not positive; one that large is no gate either)
                    const float g = cur[i] < kMinGate ? kMinGate : cur[i];
                    x[i] = __float2ll_rn(g * (float)kLog2e * kGateUnits) + (i > 0 ? x[i - 1] : 0);
                }
                if (__any_sync(0xffffffffu, nan)) lost = __int_as_float(0x7fc00000);
                long long s = x[3];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, s, off);
                    if (lane >= off) s += y;
                }
                const long long all = __shfl_sync(0xffffffffu, s, 31);
                const long long before = s - x[3];                                       // exclusive
                // this lane's block: its start, its end
                const long long start = __shfl_sync(0xffffffffu, before, lane & ~7), end = __shfl_sync(0xffffffffu, s, lane | 7);
                // lanes 4 i + j of the first 16: blocks i and j
                const int bi = (lane >> 2) & 3, bj = lane & 3;
                const long long si = __shfl_sync(0xffffffffu, before, 8 * bi), sj = __shfl_sync(0xffffffffu, before, 8 * bj);
                const long long ei = __shfl_sync(0xffffffffu, s, 8 * bi + 7), ej = __shfl_sync(0xffffffffu, s, 8 * bj + 7);
                GateBuf* gb = take();
                if (!gb) break;
                GateBuf& g = *gb;
                const long long far = STATES ? passed : 0;
                float up[4], cf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    up[i] = real(before - start + x[i]) + lost;
                    cf[i] = ex2(rev ? up[i] : real(end - before - x[i])) + lost;
                }
                *reinterpret_cast<float4*>(g.rc + 4 * lane) = make_float4(up[0], up[1], up[2], up[3]);
                *reinterpret_cast<float4*>(g.cf + 4 * lane) = make_float4(cf[0], cf[1], cf[2], cf[3]);
                if (lane < 16) g.f[bi][bj] = ex2(real(rev ? sj - ei : si - ej));
                if (lane < 4) {
                    g.bl[lane] = real(ej - sj);
                    g.ce[lane] = ex2(real((rev ? sj : all - ej) + far));
                    g.re[lane] = ex2(real(rev ? all - ej : sj));
                }
                if (lane == 0) {
                    g.en = ex2(real(all)) + lost;
                    g.n = w.rows(j);
                    g.flags = kind | (j == 0 ? kFirst : 0) | (j == w.nchunk - 1 ? kLast : 0);
                    g.t0 = w.sg.t0 + w.chunk(j) * C;
                    g.h = w.sg.h;
                    g.b = w.sg.b;
                    g.pass = (int)(w.p - a.l.pass);
                    g.src = src;
                    g.dst = dst;
                    g.o = o;
                    g.w = wv;
                    g.dots = dots;
                    g.ostep = ostep;
                    g.wstep = wstep;
                }
                passed = max(passed + all, -kForgotten);      // (over a block of many forgetting tokens it would pass 63 bits)
                arrive(&g_full[it & 1]);
                if (!STATES && j == 0) {
                    after = __shfl_sync(0xffffffffu, after, 0);
                    if (after < total) name(after);
                    if (failed) break;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
            }
            if (gsum && lane == 0 && !failed) *gsum = real(passed) * 0.6931471805599453f + lost;
        }
        if (!failed) name(-1);
        if (!failed) {
            if (GateBuf* g = take()) {
                if (lane == 0) g->flags = kEnd;
                arrive(&g_full[it & 1]);
            }
        }
        if (failed && lane == 0) atomicExch(a.l.status, (int)DPLR_ERR_TIMEOUT);
    } else if (warp < kWorkers) {
        // =================== the groups ===================
        const int grp = warp >> 2;
        const uint32_t tr = sb + Ly::T_R, turn = tr + 4096 * rw;     // rows 32 rw .. of the R tile's first half: A's warp's own
        bool storing = false;      // (O, lane 0) a store may still read the warp's rows of the o tile
        auto work = [&](auto role_) {      // one loop for each role: 0 A, 1 B1 and B2, 3 C, 4 O (a states pass: 0 and 4)
        constexpr int role = decltype(role_)::value;
        [[maybe_unused]] uint32_t unit = 0;       // (states pass) units done
        for (uint32_t it = 0;; ++it) {
            const uint32_t b = it & 1, s = it % Ly::NZ, zpar = (it / Ly::NZ) & 1;
            const GateBuf& g = gates[b];
            if constexpr (!STATES && role == 1) {
                // ---- B1, B2: Y~ of 64 tokens
                constexpr int PER = DX / 8, IT = C / 2 * PER / kGrp, TS = kGrp / PER;     // pieces of a row, of a thread; tokens between two
                if (!wait(&g_full[b], (it >> 1) & 1)) { failed = true; break; }
                if (__shfl_sync(0xffffffffu, g.flags, 0) & kEnd) break;
                const int h = grp - 1, n = __shfl_sync(0xffffffffu, g.n, 0), t0 = 64 * h + row / PER, c = row % PER;
                const uint32_t off = (uint32_t)(c >> 3) * kHalf + swz(t0, c & 7);      // TS is a multiple of 8: the swizzle stays
                // Their part of the y tile goes into registers as soon as it has landed, so that the next one is on its
                // way while this one's parts are formed and while the R of the chunk before still reads the parts of its own.
                if (!wait(full_y, b)) { failed = true; break; }
                uint32_t u[IT][4];
#pragma unroll
                for (int i = 0; i < IT; ++i) lds128(sb + Ly::T_Y + off + i * TS * 128, u[i]);
                uint32_t seen = 0;
#pragma unroll
                for (int i = 0; i < IT; ++i) seen ^= (u[i][0] ^ u[i][1]) ^ (u[i][2] ^ u[i][3]);
                give_back(y_read, seen);
                if (it > 0 && !wait(h ? r_done : r_half, b ^ 1)) { failed = true; break; }
                if (n < C) {
                    if (!wait(&full_z[s], zpar)) { failed = true; break; }
                    clear_rows<DZ>(sb + Ly::T_Z + s * Ly::ZB, max(n, 64 * h), 64 * h + 64, row, kGrp);
#pragma unroll
                    for (int i = 0; i < IT; ++i)
                        if (t0 + i * TS >= n) u[i][0] = u[i][1] = u[i][2] = u[i][3] = 0u;
                }
#pragma unroll
                for (int i0 = 0; i0 < IT; i0 += 4) {
                    float wt[4];      // read ahead of the stores, which the compiler moves no load across
#pragma unroll
                    for (int i = 0; i < 4; ++i) wt[i] = g.cf[t0 + (i0 + i) * TS] * g.ce[2 * h + (i0 + i) * TS / 32];
                    if (n < C) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (t0 + (i0 + i) * TS >= n) wt[i] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        scale16(u[i0 + i], wt[i], sb + Ly::T_YH + off + (i0 + i) * TS * 128, sb + Ly::T_YL + off + (i0 + i) * TS * 128);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) { mbar_arrive(h ? y_rest : y_ready); mbar_arrive(&g_free[b]); }
            } else {
            if (!wait(&g_full[b], (it >> 1) & 1)) { failed = true; break; }
            const int flags = __shfl_sync(0xffffffffu, g.flags, 0), n = __shfl_sync(0xffffffffu, g.n, 0);
            if (flags & kEnd) break;
            [[maybe_unused]] const bool rev = flags & kRev;
            if constexpr (STATES) {
                if constexpr (role == 0) {
                    // ---- sixteen warps: Y~
                    // (lo's buffer too is free once y has landed in its own: the copy waited for the product that read both)
                    if (!wait(&full_y[s], zpar) || (n < C && !wait(&full_z[s], zpar))) { failed = true; break; }
                    scale_rows<DX>(sb + Ly::T_Y + s * Ly::XB, sb + Ly::T_YH + s * Ly::XB, sb + Ly::T_YL + s * Ly::XB, g, n, tid,
                                   32 * (kWorkers - 4));
                    if (n < C) clear_rows<DZ>(sb + Ly::T_Z + s * Ly::ZB, n, C, tid, 32 * (kWorkers - 4));
                    fence_async_smem();
                    arrive(y_states(b));
                    give_back(&g_free[b], 0);       // (what was loaded has gone into the rows)
                } else {
                    // ---- four warps: the state, behind a unit's last chunk
                    // (Every product is waited for, and the gates given back behind that: the barrier is then neither a
                    // product behind nor one ahead of the one that is asked for.)
                    if (!wait(r_states(b), (it >> 1) & 1)) { failed = true; break; }
                    float* dst = g.dst;
                    give_back(&g_free[b], (uint32_t)(uintptr_t)dst);
                    if (flags & kLast) {
                        if (DX == 128 || rw < 2)
                            store_state<DX, DZ>(dst, flags & kOutTurned, 32 * rw, turn, tmem + TM_R + (unit & 1) * 128 + lane_off);
                        fence_before_sync();
                        arrive(state_out(unit & 1));
                        ++unit;
                    }
                }
            } else if constexpr (role == 0) {
                // ---- A: the state (thread = row of R; with DX = 64 two warps only keep step)
                const bool mine = DX == 128 || warp < 2;
                if (it == 0) {
                    if (!a.independent) wait_for_kernel_before();      // the states that it starts from; the other roles read inputs
                    if (a.late) let_next_kernel_begin();
                }
                if (it > 0 && (!wait(oi_done, b ^ 1) || !wait(r_done, b ^ 1))) { failed = true; break; }
                const float en = g.en;
                const float* src = g.src;
                float* dst = g.dst;
                const bool turned = flags & kTurned;
                if (mine && (flags & kFirst)) {
                    // From memory to tensor memory, through the places of the tile's rows that only this warp writes: as many
                    // blocks at once as those hold (one by one, each waited for the memory's latency: 10 K cycles a state).
                    constexpr int HB = DZ / 64, NB = DZ / 32, AT = (SPLIT ? 2 : 1) * HB;
                    auto place = [&](int i) { return turn + (uint32_t)(i % HB) * (DX * 128) + (uint32_t)(i / HB) * Ly::RB; };
#pragma unroll 1
                    for (int g0 = 0; g0 < NB; g0 += AT) {
                        if (src) {
#pragma unroll 1
                            for (int i = 0; i < AT; ++i) start_block<DX, DZ>(src, turned, 32 * warp, 32 * (g0 + i), place(i));
                            copies_done();
                            __syncwarp();
                        }
#pragma unroll 1
                        for (int i = 0; i < AT; ++i) {
                            float v[32];
                            if (src) {
                                block_row(place(i), turned, v);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = 0.f;
                            }
                            tmem_st32_nowait(tmem + TM_R + lane_off + 32 * (g0 + i), v);
                        }
                        __syncwarp();
                    }
                    tmem_wait_st();
                }
                if (mine) {
#pragma unroll 2
                    for (int c = 0; c < DZ; c += 16) {
                        float v[16];
                        tmem_ld16(tmem + TM_R + lane_off + c, v);
#pragma unroll
                        for (int i = 0; i < 16; i += 8) {
                            const uint32_t off = (uint32_t)((c + i) >> 6) * (DX * 128) + swz(row, ((c + i) & 63) >> 3);
                            uint32_t h[4], l[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (SPLIT) split2(v[i + 2 * e], v[i + 2 * e + 1], h[e], l[e]);
                                else h[e] = pack_bf16(v[i + 2 * e], v[i + 2 * e + 1]);
                            }
                            sts128(tr + off, h[0], h[1], h[2], h[3]);
                            if (SPLIT) sts128(tr + Ly::RB + off, l[0], l[1], l[2], l[3]);
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 x = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(en, en));
                            v[i] = x.x; v[i + 1] = x.y;
                        }
                        tmem_st16_nowait(tmem + TM_R + lane_off + c, v);
                    }
                    tmem_wait_st();
                }
                fence_async_smem();
                fence_before_sync();
                arrive(r_ready);
                give_back(&g_free[b], (uint32_t)(uintptr_t)dst);
                if ((flags & kLast) && dst) {       // the state it ends with
                    if (!wait(oi_done, b) || !wait(r_done, b)) { failed = true; break; }
                    if (mine) store_state<DX, DZ>(dst, flags & kOutTurned, 32 * warp, turn, tmem + TM_R + lane_off);
                }
            } else if constexpr (role == 3) {
                // ---- C: P (thread = row)
                if (!wait(d_done, b)) { failed = true; break; }
                const float sgn = rev ? 1.f : -1.f;
                const float rc = g.rc[row], rfac = ex2(rev ? g.bl[rw] - rc : rc);
                // pieces of W columns, each block of 32 columns packed in place: hi in its first 16 columns, lo in the others
                constexpr int W = SPLIT ? 32 : 16;
                auto load = [&](int c0, float (&v)[W]) {
                    if constexpr (SPLIT) tmem_ld32(tmem + TM_D + lane_off + c0, v);
                    else tmem_ld16(tmem + TM_D + lane_off + c0, v);
                };
                auto store = [&](int c0, const float (&v)[W]) {
                    uint32_t h[W / 2], l[W / 2];
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        if (SPLIT) split2(v[2 * i], v[2 * i + 1], h[i], l[i]);
                        else h[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                    }
                    const uint32_t at = tmem + TM_D + lane_off + (c0 & ~31);
                    if constexpr (SPLIT) {
                        tmem_st16(at, h);
                        tmem_st16(at + 16, l);
                    } else {
                        tmem_st8(at + ((c0 & 16) >> 1), h);
                    }
                };
                // of `seen` bits, one per column of the block, the others become zero
                auto mask = [&](int c0, uint32_t seen, float (&v)[W]) {
                    seen >>= c0 & 31;
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (!(seen & (1u << i))) v[i] = 0.f;
                };
                const int here = 32 * rw;
                // blocks that the rows see whole
#pragma unroll 1
                for (int c0 = rev ? here + 32 : 0; c0 < (rev ? C : here); c0 += W) {
                    const float rf = rfac * g.f[rw][c0 >> 5];
                    const float2 r2 = make_float2(rf, rf);
                    const float4* col = reinterpret_cast<const float4*>(g.cf + c0);
                    float v[W];
                    load(c0, v);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 cc = col[i >> 2];
                        const float2 x = __fmul2_rn(make_float2(v[i], v[i + 1]), __fmul2_rn(make_float2(cc.x, cc.y), r2));
                        const float2 y = __fmul2_rn(make_float2(v[i + 2], v[i + 3]), __fmul2_rn(make_float2(cc.z, cc.w), r2));
                        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = y.x; v[i + 3] = y.y;
                    }
                    if (rev && n < C) {     // up to the chunk's last token
                        const int left = n - (c0 & ~31);
                        mask(c0, left <= 0 ? 0u : left >= 32 ? ~0u : ~0u >> (32 - left), v);
                    }
                    store(c0, v);
                }
                // their own block: up to their own token, or from it to the chunk's last
#pragma unroll 1
                for (int c0 = here; c0 < here + 32; c0 += W) {
                    const float2 s2 = make_float2(sgn, sgn), b2 = make_float2(-sgn * rc, -sgn * rc);
                    const float4* col = reinterpret_cast<const float4*>(g.rc + c0);
                    float v[W];
                    load(c0, v);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 cc = col[i >> 2];
                        const float2 x = __ffma2_rn(make_float2(cc.x, cc.y), s2, b2), y = __ffma2_rn(make_float2(cc.z, cc.w), s2, b2);
                        const float2 vx = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(ex2(x.x), ex2(x.y)));
                        const float2 vy = __fmul2_rn(make_float2(v[i + 2], v[i + 3]), make_float2(ex2(y.x), ex2(y.y)));
                        v[i] = vx.x; v[i + 1] = vx.y; v[i + 2] = vy.x; v[i + 3] = vy.y;
                    }
                    uint32_t seen = rev ? ~0u << lane : ~0u >> (31 - lane);
                    if (rev && n - here < 32) seen &= n <= here ? 0u : ~0u >> (32 - (n - here));
                    mask(c0, seen, v);
                    store(c0, v);
                }
                // and blocks that they do not see
#pragma unroll 1
                for (int c0 = rev ? 0 : here + 32; c0 < (rev ? here : C); c0 += W) {
                    float v[W];
#pragma unroll
                    for (int i = 0; i < W; ++i) v[i] = 0.f;
                    store(c0, v);
                }
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) { mbar_arrive(p_ready); mbar_arrive(&g_free[b]); }
            } else {
                // ---- O: the outputs (thread = row)
                const float rc = g.rc[row];
                const float cx = ex2(rev ? g.bl[rw] - rc : rc) * g.re[rw];
                const bool f32 = flags & kOutF32, staged = Ly::STAGED && n == C && !f32, live = row < n;
                const int t0 = g.t0, hh = g.h, bb = g.b, pi = g.pass;
                const long long at = (t0 + row) * g.ostep, wat = (t0 + row) * g.wstep;
                char* obase = g.o;
                const __nv_bfloat16* wv = g.w;
                float* dots = g.dots;
                give_back(&g_free[b], __float_as_uint(cx) ^ (uint32_t)t0 ^ (uint32_t)hh ^ (uint32_t)bb ^ (uint32_t)pi ^ (uint32_t)at ^
                                          (uint32_t)wat ^ (uint32_t)(uintptr_t)obase ^ (uint32_t)(uintptr_t)wv ^
                                          (uint32_t)(uintptr_t)dots);
                if (lane == 0 && storing) bulk_wait_read();
                // the rows of the dots, kWAhead pieces of 16 columns ahead (waited for one by one they took 8 K cycles a chunk)
                constexpr int kWAhead = 3;
                const uint4* wp = reinterpret_cast<const uint4*>(wv + wat);
                const bool wide = flags & kWide;
                uint4 wq[2 * kWAhead];
                auto dot_rows = [&](int piece, uint4& x, uint4& y) {
                    if (wide) ldg256(wp + 2 * piece, x, y);
                    else { x = wp[2 * piece]; y = wp[2 * piece + 1]; }
                };
                if (SPLIT && live) {
#pragma unroll
                    for (int i = 0; i < kWAhead; ++i) dot_rows(i, wq[2 * i], wq[2 * i + 1]);
                }
                if (Ly::TWO ? !wait(op_dones(b), (it >> 1) & 1) : !wait(oi_done, b) || !wait(op_done, b)) { failed = true; break; }    // (Oi goes before Op)
                const uint32_t acc = tmem + (Ly::TWO ? 64 * b : 0);
                auto values = [&](int c, float (&v)[16]) {       // columns c .. c + 15 of o
                    float u[16];
                    __syncwarp();        // (dead rows come from another way: these loads are the whole warp's)
                    tmem_ld16_pair(acc + TM_OI + lane_off + c, acc + TM_OP + lane_off + c, u, v);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 x = __ffma2_rn(make_float2(u[i], u[i + 1]), make_float2(cx, cx), make_float2(v[i], v[i + 1]));
                        v[i] = x.x; v[i + 1] = x.y;
                    }
                };
                if (staged) {
#pragma unroll 2
                    for (int c = 0; c < DZ; c += 16) {
                        float v[16];
                        values(c, v);
#pragma unroll
                        for (int i = 0; i < 16; i += 8)
                            sts128(sb + Ly::T_O + (uint32_t)((c + i) >> 6) * kHalf + swz(row, ((c + i) & 63) >> 3),
                                   pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]), pack_bf16(v[i + 4], v[i + 5]),
                                   pack_bf16(v[i + 6], v[i + 7]));
                    }
                } else {
                    float dot = 0.f, dot2 = 0.f;
#pragma unroll (SPLIT ? DZ / 16 : 1)
                    for (int c = 0; c < DZ; c += 16) {
                        float v[16];
                        values(c, v);
                        if (!live) continue;
                        if constexpr (SPLIT) {
                            const int k = (c / 16 % kWAhead) * 2;
                            const uint32_t xs[8] = {wq[k].x, wq[k].y, wq[k].z, wq[k].w, wq[k + 1].x, wq[k + 1].y, wq[k + 1].z, wq[k + 1].w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                dot = fmaf(__uint_as_float(xs[e] << 16), v[2 * e], dot);
                                dot2 = fmaf(__uint_as_float(xs[e] & 0xFFFF0000u), v[2 * e + 1], dot2);
                            }
                            if (c + 16 * kWAhead < DZ) dot_rows(c / 16 + kWAhead, wq[k], wq[k + 1]);
                        }
                        if (f32) {
                            float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(obase) + at + c);
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        } else {
                            uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(obase) + at + c);
                            uint4 x[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                x[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                  pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                            if (wide) stg256(d, x[0], x[1]);
                            else { d[0] = x[0]; d[1] = x[1]; }
                        }
                    }
                    if (SPLIT && live) dots[t0 + row] = dot + dot2;
                }
                if (staged) fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_frees(b));
                    if (staged) {     // the warp's 32 rows
#pragma unroll
                        for (int x = 0; x < DZ / 64; ++x)
                            tma_store_4d(&a.map[pi][3], 64 * x, t0 + 32 * rw, hh, bb, sb + Ly::T_O + x * kHalf + 4096 * rw);
                        bulk_commit();
                        storing = true;
                    }
                }
            }
            }
        }
        };
        if constexpr (STATES) {
            if (grp < 4) work(std::integral_constant<int, 0>{});
            else work(std::integral_constant<int, 4>{});
        } else if (grp == 0) {
            work(std::integral_constant<int, 0>{});
        } else if (grp <= 2) {
            fewer_registers<kRegsB>();
            work(std::integral_constant<int, 1>{});
        } else if (grp == 3) {
            more_registers<kRegsC>();
            work(std::integral_constant<int, 3>{});
        } else {
            more_registers<kRegsO>();
            work(std::integral_constant<int, 4>{});
        }
        if (storing) bulk_wait_all();
        if (failed && lane == 0) atomicExch(a.l.status, (int)DPLR_ERR_TIMEOUT);
    } else {
        wait_for_kernel_before();      // a CTA that finds nothing to do does not end before it either
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// A row sequence as [batch][head][token][feature]: boxes of 64 features x `rows` tokens of one head.
bool map_rows(CUtensorMap* m, const View& v, int D, long long T, int heads, int B, int rows = C) {
    return tensor_map_rows(m, v.p, D, T, heads, B, v.st, v.sh, v.sb, rows);
}

template <int DX, int DZ, bool SPLIT, bool STATES, bool RAGGED>
cudaError_t run(const Args& a, cudaStream_t s) {
    static std::atomic<uint64_t> set{0};
    constexpr int bytes = Layout<DX, DZ, SPLIT, STATES>::TOTAL;
    auto f = hd_tc_kernel<DX, DZ, SPLIT, STATES, RAGGED>;
    const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(f), bytes, set);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    return launch_kernel(f, dim3((unsigned)(a.total < sms ? a.total : sms)), NT, bytes, s, a.l.follows != 0, a);
}

template <int DX, int DZ>
cudaError_t run_kind(const Args& a, bool split, bool states, cudaStream_t s) {
    if (a.l.geo.blocks) return states ? run<DX, DZ, false, true, true>(a, s) : run<DX, DZ, false, false, true>(a, s);
    if (states) return run<DX, DZ, false, true, false>(a, s);
    return split ? run<DX, DZ, true, false, false>(a, s) : run<DX, DZ, false, false, false>(a, s);
}

}  // namespace

bool tc_supported(bool bf16, int dk, int dv) { return bf16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

cudaError_t launch_tc(const Launch& l, cudaStream_t s) {
    const long long n = units(l.geo, l.B, l.max_blocks);
    if (n == 0) return cudaSuccess;
    if (n >= (1LL << 29)) return cudaErrorInvalidValue;    // three passes and a grid's stride stay within 31 bits
    // passes of one size and kind go in one launch
    bool done[3] = {};
    for (int i = 0; i < l.npass; ++i) {
        if (done[i]) continue;
        const Pass& q = l.pass[i];
        Args a;
        std::memset(&a, 0, sizeof(a));
        a.l = l;
        a.l.npass = 0;
        for (int j = i; j < l.npass; ++j) {
            const Pass& p = l.pass[j];
            if (done[j] || p.DX != q.DX || p.DZ != q.DZ || (p.dots != nullptr) != (q.dots != nullptr) ||
                (p.states_only != 0) != (q.states_only != 0))
                continue;
            done[j] = true;
            const int k = a.l.npass++;
            a.l.pass[k] = p;
            const int H = l.geo.H;
            const long long T = l.geo.T;
            if (!p.states_only && !map_rows(&a.map[k][0], p.x, p.DX, T, H / p.x.div, l.B)) return cudaErrorInvalidValue;
            if (!map_rows(&a.map[k][1], p.y, p.DX, T, H / p.y.div, l.B)) return cudaErrorInvalidValue;
            if (!map_rows(&a.map[k][2], p.z, p.DZ, T, H / p.z.div, l.B)) return cudaErrorInvalidValue;
            if (!p.states_only && !p.o_f32 &&
                !map_rows(&a.map[k][3], View{p.o, p.ob, p.oh, p.ot, 1}, p.DZ, T, H, l.B, 32))
                return cudaErrorInvalidValue;
        }
        a.total = (int)n * a.l.npass;
        // Lengths of a ragged batch differ: CTAs take their units as they get done with others. Which one takes a unit does
        // not touch its result.
        if (l.geo.blocks && !q.states_only) a.counter = l.status + 16;
        for (int j = i; j < l.npass; ++j) a.late |= !q.states_only && !done[j];
        a.independent = i > 0 && !q.states_only;
        if (i > 0) a.l.follows = 1;
        const bool split = q.dots != nullptr, states = q.states_only != 0;
        cudaError_t e;
        if (q.DX == 128 && q.DZ == 128) e = run_kind<128, 128>(a, split, states, s);
        else if (q.DX == 128) e = run_kind<128, 64>(a, split, states, s);
        else if (q.DZ == 128) e = run_kind<64, 128>(a, split, states, s);
        else e = run_kind<64, 64>(a, split, states, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace hd
}  // namespace dplr
