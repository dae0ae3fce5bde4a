// Linear attention with one decay per head in fp32 on the CUDA cores: every type and size, both directions of time,
// dense and ragged batches (hd_internal.h has the operator). It runs what the tensor-core kernel does not take: fp32
// inputs, and bf16 with a head size of 32.
//
// A CTA owns one segment of one (batch, head) and a block of up to 64 columns of the state, which it keeps in shared
// memory, and walks the segment in chunks of 32 tokens (G: inclusive cumulative log-gates of the chunk):
//   forward    P_rc = (x_r . y_c) e^{G_r - G_c}, c <= r;  o_r = P z + e^{G_r} R^T x_r;      R <- e^{G_n} R + sum e^{G_n - G_c} y_c z_c^T
//   backward   P_rc = (x_r . y_c) e^{G_c - G_r}, c >= r;  o_r = P z + e^{G_n - G_r} R^T x_r;  R <- e^{G_n} R + sum e^{G_c} y_c z_c^T
// Columns of the state evolve independently, so the column blocks share nothing but the product x y^T, which each
// forms again. Exponents are differences of cumulative gates and never positive: nothing overflows for any gate.
//
// Bound: by the instructions that two CTAs of eight warps an SM issue (0.4 a cycle and scheduler) and the shared-memory loads
// among them. Chunks of 32 keep P small beside the state's products; 64 columns and 64 features give a thread 4 x 4
// numbers of the state for three loads a token. Measured (fp32, B2 H8 T2001, 64 x 64, 16 segments a head): states 19 us,
// outputs 44 us, 8 TFLOP/s of the recurrence; with scalar products 23 and 50.
#include <cuda_bf16.h>

#include "hd_internal.h"

namespace dplr {
namespace hd {
namespace {

constexpr int TH = 256;   // threads
constexpr int C = 32;     // tokens of a chunk
constexpr int LDP = C + 4;

template <class T> struct Vec;     // 16 bytes of a type
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float* d) {
        d[0] = __uint_as_float(v.x); d[1] = __uint_as_float(v.y); d[2] = __uint_as_float(v.z); d[3] = __uint_as_float(v.w);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float* d) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[2 * i] = __uint_as_float(u[i] << 16);
            d[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Two fp32 numbers in a register pair: one instruction multiplies and adds both. The products below are bound by the
// instructions that a scheduler can issue, of which this takes off a third.
struct F4 { uint64_t a, b; };
__device__ __forceinline__ F4 ld4x2(const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return F4{v.x, v.y};
}
__device__ __forceinline__ uint64_t both(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float2 two(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}

// C rows of a row sequence (D features) on their way through registers: 16 bytes a piece, pieces spread over the threads.
// take() starts the loads of the rows t .. t + n - 1 (the others are zero), put() writes them as fp32 to shared memory.
template <class IT, int D, int LD>
struct Rows {
    static constexpr int N = Vec<IT>::N, PER = D / N, M = (C * PER + TH - 1) / TH;
    uint4 r[M];
    __device__ __forceinline__ void take(const IT* base, long long step, long long t, int n) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = threadIdx.x + m * TH, row = i / PER;
            r[m] = make_uint4(0u, 0u, 0u, 0u);
            if (row < n) r[m] = *reinterpret_cast<const uint4*>(base + (t + row) * step + (i % PER) * N);
        }
    }
    __device__ __forceinline__ void put(float* dst) const {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int i = threadIdx.x + m * TH, row = i / PER, c = (i % PER) * N;
            if (C * PER % TH != 0 && row >= C) break;
            float d[N];
            Vec<IT>::unpack(r[m], d);
#pragma unroll
            for (int e = 0; e < N; e += 4)
                *reinterpret_cast<float4*>(dst + row * LD + c + e) = make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
        }
    }
};

template <class IT>
__device__ __forceinline__ void store4(void* p, long long at, const float (&v)[4], bool f32) {
    if (f32 || sizeof(IT) == 4) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), c = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&c));
    }
}

template <class IT, int DX, int NZ>
__device__ __forceinline__ void segment_pass(const Pass& p, const Geometry& geo, const Segment& sg, int zb, long long bh, float* sm) {
    constexpr int LDX = DX + 4, LDZ = NZ + 4;
    constexpr int CG = NZ / 4, RG = TH / CG;        // column groups of 4, row groups
    constexpr int OR = C / RG, SR = DX / RG;        // rows of o and of the state per thread
    float* X = sm;
    float* Y = X + C * LDX;
    float* Z = Y + C * LDX;
    float* S = Z + C * LDZ;
    float* P = S + DX * LDZ;
    float* G = P + C * LDP;                         // [C] cumulative gates and [C] what their rounding left,
    float* GL = G + C;                              // [C] weights of the update, [C] of the readout
    float* W = GL + C;
    float* CX = W + C;
    float* tot = CX + C;                            // [1] the chunk's total
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, c0 = 4 * cg, z0 = zb * NZ;
    const bool rev = p.reverse;
    const bool so = p.states_only;

    float gsum = 0.f;
    const float* gp = p.g + sg.b * p.gb + sg.h * p.gh;
    const int nchunk = (sg.n + C - 1) / C;
    // the next chunk's rows and gates are on their way while one is computed
    auto head = [&](const View& v) { return static_cast<const IT*>(v.p) + sg.b * v.sb + (sg.h / v.div) * v.sh; };
    const IT *xp = so ? nullptr : head(p.x), *yp = head(p.y), *zp = head(p.z) + z0;
    const long long xs = p.x.st, ys = p.y.st, zs = p.z.st, gs = p.gt;
    Rows<IT, DX, LDX> xr, yr;
    Rows<IT, NZ, LDZ> zr;
    float gr = 0.f;
    auto take = [&](int jj) {
        const int j = rev ? nchunk - 1 - jj : jj;
        const long long t = (long long)sg.t0 + j * C;
        const int n = min(C, sg.n - j * C);
        if (!so) xr.take(xp, xs, t, n);
        yr.take(yp, ys, t, n);
        zr.take(zp, zs, t, n);
        gr = tid < n ? gp[(t + tid) * gs] : 0.f;      // (n <= 32)
    };
    take(0);
    wait_for_kernel_before();
    // ---- the starting state, along its contiguous axis
    {
        const float* src = nullptr;
        bool turned = false;
        if (!so) {
            if (p.bound && !sg.alone) {
                src = p.bound + (rev ? sg.entry + sg.step : sg.entry) * (long long)DX * p.DZ;
                turned = p.bound_turned;
            } else if (p.ext_in && !sg.fresh) {
                src = p.ext_in + sg.ext * (long long)DX * p.DZ;
                turned = p.ext_turned;
            }
        }
        if (src && turned) {
#pragma unroll 8
            for (int i = tid; i < DX * NZ; i += TH) S[(i % DX) * LDZ + i / DX] = src[(z0 + i / DX) * DX + i % DX];
        } else {
#pragma unroll 4
            for (int i = tid; i < DX * CG; i += TH)
                *reinterpret_cast<float4*>(S + i / CG * LDZ + 4 * (i % CG)) =
                    src ? ld4(src + i / CG * p.DZ + z0 + 4 * (i % CG)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    for (int jj = 0; jj < nchunk; ++jj) {
        const int j = rev ? nchunk - 1 - jj : jj;
        const long long t0 = (long long)sg.t0 + j * C;
        const int n = min(C, sg.n - j * C);
        __syncthreads();
        if (!so) xr.put(X);
        yr.put(Y);
        zr.put(Z);
        const float graw = gr;
        if (jj + 1 < nchunk) take(jj + 1);
        if (tid < 32) {
            // Sums in fixed point (40 fractional bits, 64 in all): after a gate of -100 those between later tokens still
            // count. (64-bit floating point has few units here.)
            const bool bad = !(graw <= 1e4f);      // NaN (gates are not positive; one that large is no gate either)
            const uint32_t nan = __ballot_sync(0xffffffffu, bad);
            long long g = __float2ll_rn((bad ? 0.f : graw < kMinGate ? kMinGate : graw) * kGateUnits);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, g, off);
                if (tid >= off) g += y;
            }
            const long long gn = __shfl_sync(0xffffffffu, g, 31);
            const float lost = __int_as_float(0x7fc00000), scale = kGateUnit;
            const float any = nan ? lost : 0.f, upto = nan & (0xffffffffu >> (31 - tid)) ? lost : 0.f;
            const float all = __ll2float_rn(gn) * scale + any, rest = __ll2float_rn(gn - g) * scale + any;
            const float hi = __ll2float_rn(g);
            const float up = hi * scale + upto;
            G[tid] = up;
            GL[tid] = __ll2float_rn(g - __float2ll_rn(hi)) * scale;
            W[tid] = __expf(rev ? up : rest);
            CX[tid] = __expf(rev ? rest : up);
            if (tid == 0) tot[0] = all;
        }
        __syncthreads();
        const float all = tot[0];
        gsum += all;
        if (!so) {
            // ---- P: rows r, r + 16 x columns c, c + 16
            const int r = tid >> 4, c = tid & 15;
            uint64_t a[2][2] = {};      // even and odd features
#pragma unroll 8
            for (int i = 0; i < DX; i += 4) {
                const F4 x0 = ld4x2(X + r * LDX + i), x1 = ld4x2(X + (r + 16) * LDX + i);
                const F4 y0 = ld4x2(Y + c * LDX + i), y1 = ld4x2(Y + (c + 16) * LDX + i);
                a[0][0] = fma2(x0.a, y0.a, fma2(x0.b, y0.b, a[0][0]));
                a[0][1] = fma2(x0.a, y1.a, fma2(x0.b, y1.b, a[0][1]));
                a[1][0] = fma2(x1.a, y0.a, fma2(x1.b, y0.b, a[1][0]));
                a[1][1] = fma2(x1.a, y1.a, fma2(x1.b, y1.b, a[1][1]));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int rr = r + 16 * e, cc = c + 16 * f;
                    const bool in = rev ? cc >= rr : cc <= rr;
                    const float d = (G[rr] - G[cc]) + (GL[rr] - GL[cc]);
                    const float2 v = two(a[e][f]);
                    P[rr * LDP + cc] = in ? (v.x + v.y) * __expf(rev ? -d : d) : 0.f;
                }
            __syncthreads();
            // ---- o: rows OR rg .. of 4 columns
            F4 oo[OR] = {};
#pragma unroll 4
            for (int i = 0; i < DX; i += 4) {
                F4 s[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = ld4x2(S + (i + e) * LDZ + c0);
#pragma unroll
                for (int q = 0; q < OR; ++q) {
                    const float4 x = ld4(X + (OR * rg + q) * LDX + i);
                    const float xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t xx = both(xv[e]);
                        oo[q].a = fma2(xx, s[e].a, oo[q].a);
                        oo[q].b = fma2(xx, s[e].b, oo[q].b);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < OR; ++q) {
                const uint64_t cx = both(CX[OR * rg + q]);
                oo[q].a = mul2(cx, oo[q].a);
                oo[q].b = mul2(cx, oo[q].b);
            }
            // tokens that a row does not see may hold anything: they are left out, not multiplied by zero. First those that
            // all of the thread's rows see, then the few between its rows.
            {
                const int lo = rev ? OR * rg + OR - 1 : 0, hi = rev ? C : OR * rg + 1;
                const float* Pr = P + OR * rg * LDP;
#pragma unroll 4
                for (int u = lo; u < hi; ++u) {
                    const F4 z = ld4x2(Z + u * LDZ + c0);
#pragma unroll
                    for (int q = 0; q < OR; ++q) {
                        const uint64_t w = both(Pr[q * LDP + u]);
                        oo[q].a = fma2(w, z.a, oo[q].a);
                        oo[q].b = fma2(w, z.b, oo[q].b);
                    }
                }
#pragma unroll
                for (int k = 1; k < OR; ++k) {        // forward: token OR rg + k, seen by rows k ..; backward: token
                    const int u = rev ? OR * rg + OR - 1 - k : OR * rg + k;      // OR rg + OR - 1 - k, by rows 0 .. OR - 1 - k
                    const F4 z = ld4x2(Z + u * LDZ + c0);
#pragma unroll
                    for (int q = 0; q < OR; ++q) {
                        const bool in = rev ? q <= OR - 1 - k : q >= k;
                        const uint64_t w = both(Pr[q * LDP + u]);
                        oo[q].a = in ? fma2(w, z.a, oo[q].a) : oo[q].a;
                        oo[q].b = in ? fma2(w, z.b, oo[q].b) : oo[q].b;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < OR; ++q) {
                const int rr = OR * rg + q;
                const long long t = t0 + rr;
                const float2 oa = two(oo[q].a), ob = two(oo[q].b);
                const float o[4] = {oa.x, oa.y, ob.x, ob.y};
                if (rr < n) store4<IT>(p.o, sg.b * p.ob + sg.h * p.oh + t * p.ot + z0 + c0, o, p.o_f32);
                if (p.dots) {
                    float d = 0.f;
                    if (rr < n) {
                        const IT* w = static_cast<const IT*>(p.w.p) + sg.b * p.w.sb + (sg.h / p.w.div) * p.w.sh + t * p.w.st + z0 + c0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) d = fmaf(o[e], static_cast<float>(w[e]), d);
                    }
#pragma unroll
                    for (int off = CG / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                    if (cg == 0 && rr < n)
                        p.dots[(zb * bh + sg.b * geo.H + sg.h) * geo.T + t] = d;
                }
            }
            __syncthreads();   // S was read
        }
        // ---- the state: rows SR rg .. of 4 columns
        {
            F4 a[SR];
            const uint64_t e = both(__expf(all));
#pragma unroll
            for (int q = 0; q < SR; ++q) {
                const F4 s = ld4x2(S + (SR * rg + q) * LDZ + c0);
                a[q].a = mul2(e, s.a);
                a[q].b = mul2(e, s.b);
            }
#pragma unroll 4
            for (int u = 0; u < C; ++u) {      // (rows behind the last token are zero)
                const uint64_t w = both(W[u]);
                F4 z = ld4x2(Z + u * LDZ + c0);
                z.a = mul2(w, z.a);
                z.b = mul2(w, z.b);
                float y[SR];
                if constexpr (SR % 4 == 0) {
#pragma unroll
                    for (int q = 0; q < SR; q += 4) {
                        const float4 v = ld4(Y + u * LDX + SR * rg + q);
                        y[q] = v.x; y[q + 1] = v.y; y[q + 2] = v.z; y[q + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < SR; ++q) y[q] = Y[u * LDX + SR * rg + q];
                }
#pragma unroll
                for (int q = 0; q < SR; ++q) {
                    const uint64_t yy = both(y[q]);
                    a[q].a = fma2(yy, z.a, a[q].a);
                    a[q].b = fma2(yy, z.b, a[q].b);
                }
            }
#pragma unroll
            for (int q = 0; q < SR; ++q)
                *reinterpret_cast<ulonglong2*>(S + (SR * rg + q) * LDZ + c0) = make_ulonglong2(a[q].a, a[q].b);
        }
    }
    __syncthreads();
    // ---- the state it ends with
    float* dst = nullptr;
    if (so) dst = p.bound + (rev ? sg.entry : sg.entry + sg.step) * (long long)DX * p.DZ;
    else if (p.ext_out && (rev ? sg.first : sg.last)) dst = p.ext_out + sg.ext * (long long)DX * p.DZ;
    const bool turned = so ? p.bound_turned : p.ext_turned;
    if (dst)
        for (int i = tid; i < DX * NZ; i += TH) {
            const int r = turned ? i % DX : i / NZ, c = turned ? i / DX : i % NZ;
            dst[turned ? (z0 + c) * DX + r : r * p.DZ + z0 + c] = S[r * LDZ + c];
        }
    if (so && p.gsum && zb == 0 && tid == 0) p.gsum[sg.entry] = gsum;
}

template <class IT, int DX>
__device__ __forceinline__ void pass_nz(const Pass& p, const Geometry& geo, const Segment& sg, int zb, long long bh, float* sm) {
    if (p.DZ == 32) segment_pass<IT, DX, 32>(p, geo, sg, zb, bh, sm);
    else segment_pass<IT, DX, 64>(p, geo, sg, zb, bh, sm);
}

// grid: x = unit * (column blocks of the widest pass) + column block, y = pass
template <class IT>
__global__ void __launch_bounds__(TH) hd_fp32_kernel(const __grid_constant__ Launch a, int zmax, long long bh) {
    extern __shared__ __align__(16) float sm[];
    let_next_kernel_begin();
    const Pass& p = a.pass[blockIdx.y];
    const int zb = blockIdx.x % zmax;
    Segment sg;
    sg.n = 0;
    const bool found = locate(a.geo, blockIdx.x / zmax, sg);
    if (zb * (p.DZ == 32 ? 32 : 64) >= p.DZ || !found || (p.states_only == 1 && (p.reverse ? sg.first : sg.last))) {
        if (!found && sg.n > 0 && threadIdx.x == 0) atomicExch(a.status, (int)DPLR_ERR_INVALID_ARG);   // its request's slot is bad
        wait_for_kernel_before();      // a kernel of which no CTA waited would end before the one before it
        return;
    }
    switch (p.DX) {
        case 32: pass_nz<IT, 32>(p, a.geo, sg, zb, bh, sm); break;
        case 64: pass_nz<IT, 64>(p, a.geo, sg, zb, bh, sm); break;
        default: pass_nz<IT, 128>(p, a.geo, sg, zb, bh, sm); break;
    }
}

std::atomic<uint64_t> g_set_f32{0}, g_set_bf16{0};

}  // namespace

int fp32_zblock(int DZ) { return DZ == 32 ? 32 : 64; }

cudaError_t launch_fp32(const Launch& a, cudaStream_t s) {
    int zmax = 1;
    size_t bytes = 0;
    for (int i = 0; i < a.npass; ++i) {
        const Pass& p = a.pass[i];
        const int nz = fp32_zblock(p.DZ);
        zmax = max(zmax, p.DZ / nz);
        const size_t need = sizeof(float) * ((size_t)2 * C * (p.DX + 4) + (size_t)(C + p.DX) * (nz + 4) + C * LDP + 4 * C + 4);
        bytes = need > bytes ? need : bytes;
    }
    const long long n = units(a.geo, a.B, a.max_blocks) * zmax;
    if (n == 0) return cudaSuccess;
    if (n >= (1LL << 31)) return cudaErrorInvalidValue;
    const void* f = a.bf16 ? (const void*)hd_fp32_kernel<__nv_bfloat16> : (const void*)hd_fp32_kernel<float>;
    const int most = (int)(sizeof(float) * (2 * C * 132 + (C + 128) * 68 + C * LDP + 4 * C + 4));
    cudaError_t e = set_smem_limit_once(f, most, a.bf16 ? g_set_bf16 : g_set_f32);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)n, (unsigned)a.npass);
    const long long bh = (long long)a.B * a.geo.H;
    return launch_kernel(a.bf16 ? hd_fp32_kernel<__nv_bfloat16> : hd_fp32_kernel<float>, grid, TH, bytes, s, a.follows != 0, a, zmax, bh);
}

}  // namespace hd
}  // namespace dplr
