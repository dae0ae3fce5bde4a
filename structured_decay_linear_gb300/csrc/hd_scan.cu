// The small steps between the passes of the per-head-decay operator: boundary states from segments' own contributions,
// the gradient of the log-gates, and the sums over value heads that share a query/key head. None uses atomics on values,
// so their results do not depend on timing.
//
// Measured: boundary states of B4 H16 T4096, 128 x 128, eight segments a head, both directions: 19 us for 63 MB read (15
// contributions of 4.2 MB) and 71 MB written (17 boundaries, mostly into L2), 7 TB/s; the gates' gradient of the same: 20 us
// for 61 MB, 3 TB/s: a CTA's chain (two states, their product, the sums over its tokens) takes that long, not the memory; a
// ragged batch without a request of two blocks: 3.5 us.
#include <cuda_bf16.h>

#include "hd_internal.h"

namespace dplr {
namespace hd {
namespace {

// ---- boundary states: one thread per four elements of one (sequence, head)'s state, walking its segments. The loads
// of the contributions do not depend on the chain, so kAhead are in flight at a time. (Eight took 4 us off a scan of 16
// segments and put 3 us on one of four, whose larger CTAs started later: chosen by the number of segments.)
template <int kAhead>
__device__ __forceinline__ void scan_row(const Scan& a, int row, int at, bool back) {
    const long long size = (long long)a.dk * a.dv;
    float* W = back ? a.bwd : a.fwd;
    const float* ext = back ? a.bwd_ext : a.fwd_ext;
    long long base, step, eidx;
    int nseg;
    bool fresh = false;
    if (a.geo.blocks) {
        const int r = row / a.geo.H, h = row % a.geo.H;
        const int b0 = a.geo.block_starts[r];
        nseg = a.geo.block_starts[r + 1] - b0;
        if (nseg < 2) return;
        base = (long long)b0 * a.geo.H + h;
        step = a.geo.H;
        const int slot = a.geo.slots[r];
        if (slot < 0 || slot >= a.geo.n_slots) return;
        eidx = (long long)slot * a.geo.H + h;
        fresh = a.geo.context[r] == 0;
    } else {
        nseg = a.geo.nseg;
        base = (long long)row * (nseg + 1);
        step = 1;
        eidx = row;
    }
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ext && !fresh) {
        if (a.turned) {       // element (j, i) of [dv][dk] is (i, j) of [dk][dv]
            const float* e = ext + eidx * size + (at % a.dk) * (long long)a.dv + at / a.dk;
            cur = make_float4(e[0], e[a.dv], e[2 * a.dv], e[3 * a.dv]);
        } else {
            cur = *reinterpret_cast<const float4*>(ext + eidx * size + at);
        }
    }
    // step i (0 ..): the contribution lies at boundary first + i dir, its gates at segment gfirst + i dir
    const int n = back ? nseg - 1 : (a.upto_end ? nseg : nseg - 1);
    const long long dir = back ? -step : step;
    const long long start = base + (back ? (long long)nseg * step : 0);
    const long long gfirst = base + (back ? (long long)(nseg - 1) * step : 0);
    *reinterpret_cast<float4*>(W + start * size + at) = cur;
    for (int i = 0; i < n; i += kAhead) {
        float4 v[kAhead];
        float e[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i + u < n) {
                v[u] = *reinterpret_cast<const float4*>(W + (start + (i + u + 1) * dir) * size + at);
                e[u] = __expf(a.gsum[gfirst + (i + u) * dir]);
            }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i + u < n) {
                cur.x = fmaf(e[u], cur.x, v[u].x);
                cur.y = fmaf(e[u], cur.y, v[u].y);
                cur.z = fmaf(e[u], cur.z, v[u].z);
                cur.w = fmaf(e[u], cur.w, v[u].w);
                *reinterpret_cast<float4*>(W + (start + (i + u + 1) * dir) * size + at) = cur;
            }
    }
}

template <int kAhead>
__global__ void __launch_bounds__(256) hd_scan_kernel(const __grid_constant__ Scan a, int rows) {
    const int at = (blockIdx.y * 256 + threadIdx.x) * 4;
    let_next_kernel_begin();
    wait_for_kernel_before();
    if (a.geo.blocks) {     // a ragged batch may have no request of two blocks: then there is nothing to do
        bool any = false;
        for (int r = threadIdx.x; r < a.R; r += 256) any |= a.geo.block_starts[r + 1] - a.geo.block_starts[r] > 1;
        if (!__syncthreads_or(any)) return;
    }
    if (at >= a.dk * a.dv) return;
    for (int row = blockIdx.x; row < rows; row += gridDim.x) scan_row<kAhead>(a, row, at, a.fwd == nullptr || blockIdx.z == 1);
}

// ---- the order in which CTAs take a ragged batch's blocks: the longest first, so that none starts late. (32 requests of up
// to 2000 tokens: as they came, the last CTA worked alone for 30 of 112 us.) One CTA counts blocks by their chunks and deals
// them out; equal ones come in any order, which decides who computes them and nothing else.
constexpr int kLengths = 256;
__global__ void __launch_bounds__(1024) hd_order_kernel(const __grid_constant__ Geometry g, int most, int* order, int* counter) {
    __shared__ int begin[kLengths];
    let_next_kernel_begin();
    const int tid = threadIdx.x, n = min(g.block_starts[g.R], most);
    const int4* blocks = reinterpret_cast<const int4*>(g.blocks);
    auto bucket = [&](int i) { return min(max(kLengths - (blocks[i].z + kChunk - 1) / kChunk, 0), kLengths - 1); };
    if (tid < kLengths) begin[tid] = 0;
    if (tid == 0) *counter = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 1024) atomicAdd(&begin[bucket(i)], 1);
    __syncthreads();
    if (tid < 32) {      // exclusive sums, eight buckets a lane
        int c[kLengths / 32], sum = 0;
#pragma unroll
        for (int e = 0; e < kLengths / 32; ++e) {
            c[e] = sum;
            sum += begin[kLengths / 32 * tid + e];
        }
        int x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (tid >= off) x += y;
        }
#pragma unroll
        for (int e = 0; e < kLengths / 32; ++e) begin[kLengths / 32 * tid + e] = x - sum + c[e];
    }
    __syncthreads();
    for (int i = tid; i < n; i += 1024) order[atomicAdd(&begin[bucket(i)], 1)] = i;
}

// ---- the gradient of the log-gates: one CTA per segment of one (batch, head)
__global__ void __launch_bounds__(256) hd_gate_grad_kernel(const __grid_constant__ GateGrad a) {
    __shared__ double part[8];
    __shared__ double carry_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    let_next_kernel_begin();
    wait_for_kernel_before();
    const long long bh = blockIdx.x / a.nseg;
    const int seg = blockIdx.x % a.nseg;
    const int t0 = seg * a.L, n = min(a.L, a.T - t0);
    const long long size = (long long)a.dk * a.dv, all = (long long)a.B * a.H * a.T;
    const bool last = seg == a.nseg - 1;
    // <S, dS> at the segment's end: fp32 over a thread's products and a warp, 64 bits across warps (fp64 throughout took
    // three times as long as the bytes)
    float d = 0.f;
    if (!last || a.last_end) {
        const float *S, *R;
        if (a.fwd) {
            S = a.fwd + (bh * (a.nseg + 1) + seg + 1) * size;
            R = a.bwd + (bh * (a.nseg + 1) + seg + 1) * size;
        } else {
            S = a.S_T + bh * size;
            R = a.dST + bh * size;
        }
        float e[4] = {};
#pragma unroll 4
        for (int i = 4 * tid; i < size; i += 1024) {
            const float4 x = *reinterpret_cast<const float4*>(S + i), y = *reinterpret_cast<const float4*>(R + i);
            e[0] = fmaf(x.x, y.x, e[0]); e[1] = fmaf(x.y, y.y, e[1]);
            e[2] = fmaf(x.z, y.z, e[2]); e[3] = fmaf(x.w, y.w, e[3]);
        }
        d = (e[0] + e[1]) + (e[2] + e[3]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) part[warp] = d;
    __syncthreads();
    double carry = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) carry += part[w];
    // suffix sums, 256 tokens at a time from the end
    double total = 0.0;
    for (int hi = n; hi > 0; hi -= 256) {
        const int i = hi - 1 - tid;            // thread 0 takes the last token
        float x = 0.f;
        const long long t = bh * a.T + t0 + i;
        if (i >= 0) {
            for (int z = 0; z < a.nq; ++z) x += a.dq_dots[z * all + t];
            for (int z = 0; z < a.nk; ++z) x -= a.dk_dots[z * all + t];
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        __syncthreads();
        if (lane == 31) part[warp] = x;
        __syncthreads();
        double before = carry;
        for (int w = 0; w < warp; ++w) before += part[w];
        const double sum = before + (double)x;
        if (i >= 0) {
            if (a.dg_token) a.dg_token[t] = (float)sum;
            total += sum;
        }
        if (tid == 255) carry_s = sum;
        __syncthreads();
        carry = carry_s;
    }
    if (a.seg_sum) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        __syncthreads();
        if (lane == 0) part[warp] = total;
        __syncthreads();
        if (tid == 0) {
            double s = 0.0;
            for (int w = 0; w < 8; ++w) s += part[w];
            a.seg_sum[blockIdx.x] = s;
        }
    }
}

// one warp per head: the sum of its segments, batch by batch
__global__ void __launch_bounds__(32) hd_head_grad_kernel(const __grid_constant__ GateGrad a) {
    const int h = blockIdx.x, lane = threadIdx.x;
    let_next_kernel_begin();
    wait_for_kernel_before();
    double s = 0.0;
    for (int i = lane; i < a.B * a.nseg; i += 32)
        s += a.seg_sum[((long long)(i / a.nseg) * a.H + h) * a.nseg + i % a.nseg];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) a.dg_head[h] = (float)s;
}

template <bool BF>
__global__ void __launch_bounds__(256) hd_group_sum_kernel(const __grid_constant__ GroupSum a) {
    const int per = a.D / 4, lg = 31 - __clz(per), group = a.H / a.Hq;      // (per: 8, 16 or 32)
    const GroupSum::One& w = a.one[blockIdx.y];
    let_next_kernel_begin();
    wait_for_kernel_before();
    const long long n = (long long)a.B * a.Hq * a.T * per;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const int c = (int)(i & (per - 1)) * 4;
        const uint32_t row = (uint32_t)(i >> lg), bh = row / a.T;      // rows: below 2^31
        const long long t = row % a.T, hq = bh % a.Hq, b = bh / a.Hq;
        const float* src = w.part + ((b * a.H + hq * group) * a.T + t) * a.D + c;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < group; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(src + (long long)j * a.T * a.D);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        const long long at = b * w.ob + hq * w.oh + t * w.ot + c;
        if (BF) {
            __nv_bfloat162 x = __floats2bfloat162_rn(s.x, s.y), y = __floats2bfloat162_rn(s.z, s.w);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(w.out) + at) =
                make_uint2(*reinterpret_cast<uint32_t*>(&x), *reinterpret_cast<uint32_t*>(&y));
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(w.out) + at) = s;
        }
    }
}

}  // namespace

cudaError_t launch_scan(const Scan& a, cudaStream_t s) {
    const long long rows = a.geo.blocks ? (long long)a.R * a.geo.H : (long long)a.B * a.geo.H;
    if (rows == 0) return cudaSuccess;
    const unsigned gy = (unsigned)((a.dk * a.dv / 4 + 255) / 256), gz = a.fwd && a.bwd ? 2 : 1;
    // a ragged batch's rows are mostly of one block, with nothing to do: as many CTAs as are resident at once walk them (1600
    // rows of which none had anything to do took 16 us as CTAs of their own, 6 us as 256)
    const long long most = a.geo.blocks ? 8 * sm_count() / gy : rows;
    const bool deep = !a.geo.blocks && a.geo.nseg > 8;
    return launch_kernel(deep ? hd_scan_kernel<8> : hd_scan_kernel<4>, dim3((unsigned)(rows < most ? rows : most), gy, gz), 256, 0, s, true, a, (int)rows);
}

cudaError_t launch_order(const Geometry& g, int max_blocks, int* order, int* counter, cudaStream_t s) {
    return launch_kernel(hd_order_kernel, dim3(1), 1024, 0, s, false, g, max_blocks, order, counter);
}

cudaError_t launch_gate_grad(const GateGrad& a, cudaStream_t s) {
    const long long n = (long long)a.B * a.H * a.nseg;
    if (n >= (1LL << 31)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_kernel(hd_gate_grad_kernel, dim3((unsigned)n), 256, 0, s, false, a);
    if (e != cudaSuccess || !a.dg_head) return e;
    return launch_kernel(hd_head_grad_kernel, dim3((unsigned)a.H), 32, 0, s, true, a);
}

cudaError_t launch_group_sum(const GroupSum& a, cudaStream_t s) {
    const long long n = (long long)a.B * a.Hq * a.T * (a.D / 4);
    const long long most = (long long)sm_count() * 4;      // (of each of the two)
    const long long blocks = (n + 255) / 256;
    const unsigned g = (unsigned)(blocks < most ? blocks : most);
    return launch_kernel(a.bf16 ? hd_group_sum_kernel<true> : hd_group_sum_kernel<false>, dim3(g, 2), 256, 0, s, true, a);
}

}  // namespace hd
}  // namespace dplr
