// Chaining tiles of one launch: tickets, records of the tiles' maps, and the walk over earlier tiles' records.
//
// A tile of a channel is the map h -> A h + b. CTAs draw tiles from a counter, first tiles of all sequences and channels
// first, so the tiles in front of a drawn tile are done or in the hands of running CTAs: every wait ends. A CTA forms its
// tile's map from the data alone, publishes it, and reads its predecessors' records from the nearest one back to the first
// that holds a state; from there it applies the maps in order. A state is published as soon as it is known.
//
// Results do not depend on which predecessor already had its state: a published state is its tile's map applied to the state
// before it, the same multiply-add that the walk makes with the map. A record carries its own tag and is one 16-byte access,
// so a reader needs no flag and no fence beside it. Tags hold the launch's number, which the launch's last CTA counts up.
#pragma once

#include "gr_internal.h"

namespace dplr {
namespace gr {

__device__ __forceinline__ Record load_record(const Record* p) {
    uint64_t lo, hi;
    asm volatile(
        "{\n\t.reg .b128 t;\n\tld.relaxed.gpu.global.b128 t, [%2];\n\tmov.b128 {%0, %1}, t;\n\t}"
        : "=l"(lo), "=l"(hi) : "l"(p) : "memory");
    Record r;
    r.A = __uint_as_float(static_cast<uint32_t>(lo));
    r.b = __uint_as_float(static_cast<uint32_t>(lo >> 32));
    r.tag = hi;
    return r;
}

__device__ __forceinline__ void store_record(Record* p, float A, float b, unsigned long long tag) {
    const uint64_t lo = static_cast<uint64_t>(__float_as_uint(A)) | (static_cast<uint64_t>(__float_as_uint(b)) << 32);
    asm volatile(
        "{\n\t.reg .b128 t;\n\tmov.b128 t, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], t;\n\t}"
        :: "l"(p), "l"(lo), "l"(static_cast<uint64_t>(tag)) : "memory");
}

// The map h -> A h + b. RESET: a request may start in its tokens. Such a map has A = -0, and what came before does not reach it
// even if it is not a number. Products of decays are +0 and above: one that underflowed is not taken for a start, and a NaN or
// an infinity goes on through it.
constexpr float kReset = -0.f;
__device__ __forceinline__ bool resets(float A) { return __float_as_uint(A) == 0x80000000u; }
template <bool RESET> __device__ __forceinline__ float after(float A, float h, float b) {
    return RESET && resets(A) ? b : fmaf(A, h, b);
}
// The factor of a map behind one of factor `before`.
template <bool RESET> __device__ __forceinline__ float joined(float A, float before) {
    return RESET && resets(A) ? kReset : A * before;
}

// The walk of one channel, by one lane of the warp that looks after a tile's channels. `rec` is the channel in tile 0 of
// the sequence, tiles kCols records apart; `from` the nearest predecessor, `step` -1 (forward in time) or +1 (backward).
// Outside [0, NT) stands the state `outer`: the first tile finds it there, and publishes its own state at once, so that no
// other tile's walk has use for what lies behind that one.
struct Walk {
    const Record* rec;
    int from, step, NT;
    int end;                       // from the end-th tile back on stands `outer`
    float outer;
    unsigned long long stamp;      // 4 * (epoch + 1)

    __device__ __forceinline__ Record look(int back) const {
        const int i = from + step * back;
        if (back >= end || i < 0 || i >= NT) return Record{0.f, outer, stamp | kState};
        return load_record(rec + (long long)i * kCols);
    }
    __device__ __forceinline__ bool is_state(const Record& r) const { return r.tag == (stamp | kState); }
};

// What the walk starts from, asked for as soon as the tile is known: the nearest tile, and the one far_at tiles back. Where CTAs
// work on several tiles of a channel at once, the nearest has no state yet, but that one, from the round before, does.
struct Ahead {
    Record near, far;
    __device__ __forceinline__ void start(const Walk& w, int far_at) { near = w.look(0); far = w.look(far_at); }
};

// The state in front of a tile. publish() announces the tile's own map, unless the tile before has its state already. `stash`:
// [kBatch * (kBatches - 1)][kCols] at this lane's channel. Gives up after `limit` cycles and sets *gave_up.
template <bool RESET, class Publish>
__device__ __forceinline__ float walk(Walk w, const Ahead& ahead, int far_at, float2* stash, long long limit, Publish publish,
                                      bool* gave_up) {
    constexpr unsigned kAll = (1u << kBatch) - 1;
    if (__all_sync(0xffffffffu, w.is_state(ahead.near))) return ahead.near.b;
    publish();                             // and only then a look at the others: theirs come at about the same time
    Record r[kBatch];
    if (w.is_state(ahead.far) && far_at < w.end) { w.end = far_at; w.outer = ahead.far.b; }
    unsigned states = 0;                   // bit i: the i-th tile back holds a state
    bool found = false;
    float h = 0.f;
    const long long t0 = clock64();
    for (int k = 0;; ++k) {
        unsigned st, ok;
        bool here, quit;
        for (;;) {
            st = ok = 0;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) r[q] = w.look(kBatch * k + q);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (w.is_state(r[q])) { st |= 1u << q; ok |= 1u << q; }
                if (r[q].tag == (w.stamp | kMap)) ok |= 1u << q;
            }
            here = st != 0 && ((ok + 1) & ~ok) > (st & (0u - st));              // no gap nearer than the nearest state
            quit = __any_sync(0xffffffffu, clock64() - t0 > limit);
            if (quit || __all_sync(0xffffffffu, found || here || (k + 1 < kBatches && ok == kAll))) break;
        }
        found |= here;
        const bool all = __all_sync(0xffffffffu, found);
        if (all || quit || k + 1 == kBatches) {        // from the farthest tile on; the nearest state overwrites what lies before it
#pragma unroll
            for (int q = kBatch - 1; q >= 0; --q)
                if ((ok >> q) & 1u) h = (st >> q) & 1u ? r[q].b : after<RESET>(r[q].A, h, r[q].b);
            for (int i = kBatch * k - 1; i >= 0; --i) {
                const float2 e = stash[i * kCols];
                h = (states >> i) & 1u ? e.y : after<RESET>(e.x, h, e.y);
            }
            if (!all) *gave_up = true;
            return h;
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            stash[(kBatch * k + q) * kCols] = (ok >> q) & 1u ? make_float2(r[q].A, r[q].b) : make_float2(0.f, 0.f);
        states |= st << (kBatch * k);
    }
}

// A warp's two runs of tokens, one behind the other in time: the map (A, H) of the later half's lanes becomes that of both runs,
// and (Ax, Hx) is that of the other run, which its own start then goes through; for the earlier half it changes nothing.
// BACK: with the halves changed over, for what flows backwards.
static_assert(kRuns == 2, "two halves of a warp");
template <bool BACK, bool RESET = false>
__device__ __forceinline__ void join_runs(float2& A, float2& H, float2& Ax, float2& Hx, int lane) {
    const bool last = (lane >= 16) != BACK;
    const float2 Ao = make_float2(__shfl_xor_sync(0xffffffffu, A.x, 16), __shfl_xor_sync(0xffffffffu, A.y, 16));
    const float2 Ho = make_float2(__shfl_xor_sync(0xffffffffu, H.x, 16), __shfl_xor_sync(0xffffffffu, H.y, 16));
    Ax = last ? Ao : both(1.f);
    Hx = last ? Ho : both(0.f);
    H = make_float2(after<RESET>(A.x, Hx.x, H.x), after<RESET>(A.y, Hx.y, H.y));
    A = make_float2(joined<RESET>(A.x, Ax.x), joined<RESET>(A.y, Ax.y));
}

// The launch's last CTA makes the counters ready for the next launch. By one thread, after its CTA's last access to the records.
__device__ __forceinline__ void leave(Header* head) {
    unsigned before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(&head->done) : "memory");
    if (before + 1u == gridDim.x) {
        head->ticket = 0;
        head->done = 0;
        head->epoch += 1;
    }
}

// ---- tiles of a [B][T][D] tensor by TMA, in boxes of up to kBoxRows tokens
__device__ __forceinline__ void box_load(void* dst, const CUtensorMap* map, int c, int t, int b, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(sm100::smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(b),
           "r"(sm100::smem_addr(mbar)) : "memory");
}
__device__ __forceinline__ void box_store(const CUtensorMap* map, const void* src, int c, int t, int b) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
        :: "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(b), "r"(sm100::smem_addr(src)) : "memory");
}
template <int TT, int ROW>      // tokens, and bytes of a token in shared memory
__device__ __forceinline__ void tile_load(uint8_t* dst, const CUtensorMap* map, int c, int t, int b, uint64_t* mbar) {
#pragma unroll
    for (int i = 0; i < TT; i += kBoxRows) box_load(dst + i * ROW, map, c, t + i, b, mbar);
}
template <int TT, int ROW>
__device__ __forceinline__ void tile_store(const CUtensorMap* map, const uint8_t* src, int c, int t, int b, int T) {
#pragma unroll
    for (int i = 0; i < TT; i += kBoxRows)
        if (t + i < T) box_store(map, src + i * ROW, c, t + i, b);
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace gr
}  // namespace dplr
