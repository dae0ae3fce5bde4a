// Host side of the elementwise gated recurrence's C ABI: checks, workspaces and launches (gr_internal.h has the operator).
#include "gr_internal.h"
#include "hd_internal.h"

namespace dplr {
namespace gr {
namespace {

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int esize(int dtype) { return dtype == DPLR_BF16 ? 2 : 4; }
int tiles_of(int T, int tile) { return (int)(((long long)T + tile - 1) / tile); }

int groups_of(const dplr_gr_desc* d) { return (d->D + kCols - 1) / kCols; }
int tile_of(const dplr_gr_desc* d) { return forward_tile(d->in_dtype == DPLR_BF16); }
int back_tile_of(const dplr_gr_desc* d) { return backward_tile(d->in_dtype == DPLR_BF16); }

long long tile_count(const dplr_gr_desc* d, int tile) { return (long long)tiles_of(d->T, tile) * d->B * groups_of(d); }

dplr_status check_desc(const dplr_gr_desc* d) {
    if (!d) return DPLR_ERR_INVALID_ARG;
    if (d->in_dtype != DPLR_F32 && d->in_dtype != DPLR_BF16) return DPLR_ERR_INVALID_ARG;
    if (d->gate_dtype != DPLR_F32 && d->gate_dtype != DPLR_BF16) return DPLR_ERR_INVALID_ARG;
    if (d->gate != kLog && d->gate != kSigmoid) return DPLR_ERR_INVALID_ARG;
    if (d->input != kPlain && d->input != kComplement && d->input != kUnit) return DPLR_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->D < 1) return DPLR_ERR_INVALID_ARG;
    if (d->in_dtype == DPLR_F32 && d->gate_dtype == DPLR_BF16) return DPLR_ERR_UNSUPPORTED;
    if (d->T > (1 << 30) || (long long)d->B * d->T >= (1LL << 31) || d->D > (1 << 25)) return DPLR_ERR_UNSUPPORTED;
    // tiles and the tickets behind the last one are counted in 32 bits, a state's index in a pool or batch in 64
    if ((long long)d->B * groups_of(d) >= (1LL << 24) || tile_count(d, kStateStep) >= (1LL << 31))
        return DPLR_ERR_UNSUPPORTED;
    return DPLR_OK;
}

Types types_of(const dplr_gr_desc* d) {
    return Types{d->in_dtype == DPLR_BF16, d->gate_dtype == DPLR_BF16, d->gate, d->input};
}

struct RowsOf { void* p; long long sb, st; };

// Rows of D channels; `out`: they must not overlap either.
dplr_status rows_of(const dplr_gr_desc* d, const dplr_hd_tensor* t, int dtype, bool out, RowsOf* r) {
    const int es = esize(dtype), unit = 16 / es;
    const long long row = ((long long)d->D + unit - 1) / unit * unit;
    *r = RowsOf{nullptr, row, row};
    if (d->T == 0) return DPLR_OK;
    if (!t || !t->data || (reinterpret_cast<uintptr_t>(t->data) & 15u)) return DPLR_ERR_INVALID_ARG;
    const long long n[2] = {d->B, d->T};
    long long st[2] = {t->sb, t->st};
    for (int i = 0; i < 2; ++i) {
        if (n[i] == 1) { st[i] = row; continue; }
        if (st[i] <= 0 || st[i] % unit != 0) return DPLR_ERR_INVALID_ARG;
        if (st[i] >= (1LL << 40) / es) return DPLR_ERR_UNSUPPORTED;
    }
    if (out) {
        const int in = n[0] > 1 && (n[1] == 1 || st[0] < st[1]) ? 0 : 1;     // the inner axis
        if (n[in] > 1 && st[in] < d->D) return DPLR_ERR_INVALID_ARG;
        if (n[1 - in] > 1 && st[1 - in] < (n[in] > 1 ? (n[in] - 1) * st[in] : 0) + d->D) return DPLR_ERR_INVALID_ARG;
    }
    *r = RowsOf{t->data, st[0], st[1]};
    return DPLR_OK;
}

bool map_of(const dplr_gr_desc* d, const RowsOf& r, int dtype, int tile, CUtensorMap* m) {
    return tensor_map_channels(m, r.p, dtype == DPLR_BF16, d->D, d->T, d->B, r.st, r.sb, kCols, box_rows(tile));
}

bool floats_ok(const void* p, bool needed) { return p ? (reinterpret_cast<uintptr_t>(p) & 3u) == 0 : !needed; }
bool state_ok(const void* p, bool needed) { return p ? (reinterpret_cast<uintptr_t>(p) & 15u) == 0 : !needed; }

dplr_status check_workspace(size_t need, const void* ws, size_t bytes) {
    if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0) return DPLR_ERR_WORKSPACE;
    return DPLR_OK;
}

size_t record_bytes(const dplr_gr_desc* d, int tile) { return (size_t)tile_count(d, tile) * kCols * sizeof(Record); }

// Header and records; behind them, for the backward, the states that it forms again. Its two launches follow one another and
// share the records.
struct BackwardPlan { size_t states, total; };
BackwardPlan backward_plan(const dplr_gr_desc* d) {
    const size_t rec = record_bytes(d, back_tile_of(d));     // no forward tile is shorter
    BackwardPlan p;
    p.states = up(kHeader + rec);
    p.total = up(p.states + sizeof(float) * (size_t)d->B * tiles_of(d->T, kStateStep) * d->D);
    return p;
}

Arg arg_of(const dplr_gr_desc* d, int tile, void* workspace) {
    Arg a;
    a.d = Dims{d->B, d->T, d->D, groups_of(d), tiles_of(d->T, tile)};
    a.head = static_cast<Header*>(workspace);
    a.rec = reinterpret_cast<Record*>(static_cast<char*>(workspace) + kHeader);
    const long long at_once = (long long)kCtas * sm_count() / ((long long)a.d.B * a.d.G);      // a channel's tiles are B G apart
    a.far = at_once < kBatch * kBatches - 1 ? (int)at_once : kBatch * kBatches - 1;
    a.wait_cycles = wait_limit();
    return a;
}

cudaError_t copy_state(const dplr_gr_desc* d, float* dst, const float* src, cudaStream_t s) {
    const size_t bytes = sizeof(float) * (size_t)d->B * d->D;
    if (!dst || dst == src) return cudaSuccess;
    return src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, bytes, s);
}

}  // namespace
}  // namespace gr
}  // namespace dplr

using namespace dplr;
using namespace dplr::gr;

#define GR_TRY(x) do { const dplr_status st_ = (x); if (st_ != DPLR_OK) return st_; } while (0)
#define GR_CUDA(x) do { if ((x) != cudaSuccess) return DPLR_ERR_CUDA; } while (0)
#define GR_MAP(x) do { if (!(x)) return DPLR_ERR_CUDA; } while (0)

extern "C" {

dplr_status dplr_gr_check(const dplr_gr_desc* desc) { return check_desc(desc); }

size_t dplr_gr_workspace_size(const dplr_gr_desc* desc) {
    return check_desc(desc) == DPLR_OK ? up(kHeader + record_bytes(desc, tile_of(desc))) : 0;
}

dplr_status dplr_gr_forward(const dplr_gr_desc* desc, const dplr_hd_tensor* x, const dplr_hd_tensor* g, const float* h0,
                            const dplr_hd_tensor* y, float* h_T, float* states, void* workspace, size_t ws_bytes,
                            void* stream) {
    GR_TRY(check_desc(desc));
    RowsOf rx, rg, ry;
    GR_TRY(rows_of(desc, x, desc->in_dtype, false, &rx));
    GR_TRY(rows_of(desc, g, desc->gate_dtype, false, &rg));
    GR_TRY(rows_of(desc, y, desc->in_dtype, true, &ry));
    if (!floats_ok(h0, false) || !floats_ok(h_T, false) || !floats_ok(states, false)) return DPLR_ERR_INVALID_ARG;
    GR_TRY(check_workspace(dplr_gr_workspace_size(desc), workspace, ws_bytes));
    if (hd::taken({ry.p, h_T, states}, {rx.p, rg.p, h_T == h0 ? nullptr : h0, workspace}) || (h0 && (ry.p == h0 || states == h0)))
        return DPLR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) {
        GR_CUDA(copy_state(desc, h_T, h0, s));
        return DPLR_OK;
    }
    const int tile = tile_of(desc);
    CUtensorMap mx, mg, my;
    GR_MAP(map_of(desc, rx, desc->in_dtype, tile, &mx));
    GR_MAP(map_of(desc, rg, desc->gate_dtype, tile, &mg));
    GR_MAP(map_of(desc, ry, desc->in_dtype, tile, &my));
    ForwardArgs a{};
    a.c = arg_of(desc, tile, workspace);
    a.h0 = h0; a.hT = h_T; a.states = states; a.y = Out{ry.p, ry.sb, ry.st};
    GR_CUDA(launch_forward(types_of(desc), mx, mg, my, a, s));
    return DPLR_OK;
}

size_t dplr_gr_backward_workspace_size(const dplr_gr_desc* desc) {
    return check_desc(desc) == DPLR_OK ? backward_plan(desc).total : 0;
}

dplr_status dplr_gr_backward(const dplr_gr_desc* desc, const dplr_hd_tensor* x, const dplr_hd_tensor* g, const float* h0,
                             const float* states, const dplr_hd_tensor* dy, const float* dh_T, const dplr_hd_tensor* dx,
                             const dplr_hd_tensor* dg, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
    GR_TRY(check_desc(desc));
    RowsOf rx, rg, rdy, rdx, rdg;
    GR_TRY(rows_of(desc, x, desc->in_dtype, false, &rx));
    GR_TRY(rows_of(desc, g, desc->gate_dtype, false, &rg));
    GR_TRY(rows_of(desc, dy, desc->in_dtype, false, &rdy));
    GR_TRY(rows_of(desc, dx, desc->in_dtype, true, &rdx));
    GR_TRY(rows_of(desc, dg, desc->gate_dtype, true, &rdg));
    if (!floats_ok(h0, false) || !floats_ok(states, false) || !floats_ok(dh_T, false) || !floats_ok(dh0, false))
        return DPLR_ERR_INVALID_ARG;
    const BackwardPlan pl = backward_plan(desc);
    GR_TRY(check_workspace(pl.total, workspace, ws_bytes));
    if (hd::taken({rdx.p, rdg.p, dh0}, {rx.p, rg.p, rdy.p, h0, states, dh_T, workspace})) return DPLR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) {
        GR_CUDA(copy_state(desc, dh0, dh_T, s));
        return DPLR_OK;
    }
    if (!states) {
        const int tile = tile_of(desc);
        CUtensorMap fx, fg;
        GR_MAP(map_of(desc, rx, desc->in_dtype, tile, &fx));
        GR_MAP(map_of(desc, rg, desc->gate_dtype, tile, &fg));
        float* kept = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.states);
        ForwardArgs f{};
        f.c = arg_of(desc, tile, workspace);
        f.h0 = h0; f.states = kept;
        GR_CUDA(launch_forward(types_of(desc), fx, fg, fx, f, s));       // y is not written: any map stands in for its own
        states = kept;
    }
    CUtensorMap mx, mg, mdy, mdx, mdg;
    GR_MAP(map_of(desc, rx, desc->in_dtype, back_tile_of(desc), &mx));
    GR_MAP(map_of(desc, rg, desc->gate_dtype, back_tile_of(desc), &mg));
    GR_MAP(map_of(desc, rdy, desc->in_dtype, back_tile_of(desc), &mdy));
    GR_MAP(map_of(desc, rdx, desc->in_dtype, back_tile_of(desc), &mdx));
    GR_MAP(map_of(desc, rdg, desc->gate_dtype, back_tile_of(desc), &mdg));
    BackwardArgs a{};
    a.c = arg_of(desc, back_tile_of(desc), workspace);
    a.dhT = dh_T; a.states = states; a.dh0 = dh0;
    GR_CUDA(launch_backward(types_of(desc), mx, mg, mdy, mdx, mdg, a, s));
    return DPLR_OK;
}

dplr_status dplr_gr_forward_packed(const dplr_gr_desc* desc, int32_t R, int32_t n_slots, const int32_t* starts,
                                   const int32_t* token_slot, const int32_t* token_pos, const dplr_hd_tensor* x,
                                   const dplr_hd_tensor* g, float* h, const dplr_hd_tensor* y, void* workspace,
                                   size_t ws_bytes, void* stream) {
    GR_TRY(check_desc(desc));
    if (desc->B != 1 || R < 1 || n_slots < 1) return DPLR_ERR_INVALID_ARG;
    if (n_slots > (1 << 20)) return DPLR_ERR_UNSUPPORTED;
    RowsOf rx, rg, ry;
    GR_TRY(rows_of(desc, x, desc->in_dtype, false, &rx));
    GR_TRY(rows_of(desc, g, desc->gate_dtype, false, &rg));
    GR_TRY(rows_of(desc, y, desc->in_dtype, true, &ry));
    if (!floats_ok(starts, true) || !floats_ok(token_slot, desc->T > 0) || !floats_ok(token_pos, desc->T > 0) ||
        !state_ok(h, true))
        return DPLR_ERR_INVALID_ARG;
    GR_TRY(check_workspace(dplr_gr_workspace_size(desc), workspace, ws_bytes));
    if (hd::taken({ry.p, h}, {rx.p, rg.p, starts, token_slot, token_pos, workspace})) return DPLR_ERR_INVALID_ARG;
    if (desc->T == 0) return DPLR_OK;
    const int tile = tile_of(desc);
    CUtensorMap mx, mg, my;
    GR_MAP(map_of(desc, rx, desc->in_dtype, tile, &mx));
    GR_MAP(map_of(desc, rg, desc->gate_dtype, tile, &mg));
    GR_MAP(map_of(desc, ry, desc->in_dtype, tile, &my));
    ForwardArgs a{};
    a.c = arg_of(desc, tile, workspace);
    a.pool = h; a.starts = starts; a.R = R; a.slot = token_slot; a.pos = token_pos; a.n_slots = n_slots;
    a.y = Out{ry.p, ry.sb, ry.st};
    GR_CUDA(launch_packed(types_of(desc), mx, mg, my, a, static_cast<cudaStream_t>(stream)));
    return DPLR_OK;
}

dplr_status dplr_gr_decode_step(const dplr_gr_desc* desc, int32_t n_slots, const int32_t* slots, const dplr_hd_tensor* x,
                                const dplr_hd_tensor* g, float* h, const dplr_hd_tensor* y, int32_t* status, void* stream) {
    GR_TRY(check_desc(desc));
    if (desc->T != 1 || n_slots < 1) return DPLR_ERR_INVALID_ARG;
    RowsOf rx, rg, ry;
    GR_TRY(rows_of(desc, x, desc->in_dtype, false, &rx));
    GR_TRY(rows_of(desc, g, desc->gate_dtype, false, &rg));
    GR_TRY(rows_of(desc, y, desc->in_dtype, true, &ry));
    if (!floats_ok(slots, true) || !state_ok(h, true) || !floats_ok(status, false)) return DPLR_ERR_INVALID_ARG;
    if (hd::taken({ry.p, h, status}, {rx.p, rg.p, slots})) return DPLR_ERR_INVALID_ARG;
    StepArgs a{};
    a.x = rx.p; a.g = rg.p; a.y = ry.p; a.xs = rx.sb; a.gs = rg.sb; a.ys = ry.sb;
    a.pool = h; a.slots = slots; a.n_slots = n_slots; a.N = desc->B; a.D = desc->D; a.status = status;
    GR_CUDA(launch_step(types_of(desc), a, static_cast<cudaStream_t>(stream)));
    return DPLR_OK;
}

}  // extern "C"
