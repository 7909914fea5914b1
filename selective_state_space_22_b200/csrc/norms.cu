// norms.cu -- the norms before and after a mixer block, with the residual, its
// scale and the gate in the same pass, and their gradients.
//
//   before:  r = res + scale x,  out = r rstd(r) w,        rstd(v) = 1/sqrt(mean v^2 + eps)
//   after:   gate first: n = v rstd(v) w with v = y silu(z);  norm first: n = y rstd(y) w silu(z);
//            out = n, or res + scale n;  rstd per group of width/groups channels.
//
// Gradients with m = v rstd and dn the gradient at m:
//   dv = rstd (dn - m mean(dn m)),  dw = sum_rows d(out) m,  dscale = sum_rows dout (what it scales).
//
// Bound by HBM: every row is read once and written once.  A unit (one row, or one
// group of a row) is held in the registers of TPR threads, V neighbouring channels
// (16 bytes of the io type) a vector and VPT vectors a thread; its sums go through
// shuffles and, past one warp, shared memory.  The gradients need both of their
// sums (v^2 and dn v) only after all loads, so one round of sums serves them.
// There a thread keeps its columns over all rows its block takes and sums dw and
// dscale in registers; norm_bwd_sum adds the blocks' parts in a fixed order.
// Measured, bf16: before, 16384 x 2048 with a float32 residual, 59 us (6.8 TB/s) and its
// gradient 112 + 6 us; after, 8192 x 8 groups of 512, 42 us (4.8 TB/s), gradient 80 + 4 us.
#include <type_traits>

#include "mixer.cuh"

namespace ssd {
namespace {

constexpr int BWD_BLOCKS = 296;   // of 256 threads: the two per SM that fit their registers, on 148 SMs
constexpr int MANY_UNITS = 2368;  // 16 per SM

// Sums of (a, b) over the TPR threads of a unit; every thread of the block calls it.
template <int TPR> __device__ __forceinline__ float2 unit_sum(float2 v, float2 *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int wid = threadIdx.x >> 5;
        __syncthreads();  // sh free again
        if ((threadIdx.x & 31) == 0) sh[wid] = v;
        __syncthreads();
        v = sh[wid / W * W];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const float2 u = sh[wid / W * W + i];
            v.x += u.x, v.y += u.y;
        }
    }
    return v;
}

template <int TPR> constexpr int block_threads() { return TPR < 128 ? 128 : TPR; }

template <typename T, typename TR, int V, int VPT, int TPR>
__global__ void __launch_bounds__(block_threads<TPR>()) norm_before_kernel(NormCall c) {
    constexpr bool WIDE = V > 1;
    __shared__ float2 sh[block_threads<TPR>() / 32];
    const int t = threadIdx.x % TPR, row = blockIdx.x * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
    const bool in = row < c.rows;
    const T *x = static_cast<const T *>(c.x) + row * c.ld_x;
    const TR *res = static_cast<const TR *>(c.res) + row * c.ld_res;
    float r[VPT][V];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) r[q][v] = 0.f;
        if (!in || k >= c.width) continue;
        load_v<T, V, WIDE>(x + k, r[q]);
        if (c.scale) {
            float a[V];
            load_v<float, V, WIDE>(c.scale + k, a);
#pragma unroll
            for (int v = 0; v < V; ++v) r[q][v] *= a[v];
        }
        if (c.res) {
            float a[V];
            load_v<TR, V, WIDE>(res + k, a);
#pragma unroll
            for (int v = 0; v < V; ++v) r[q][v] += a[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s.x = fmaf(r[q][v], r[q][v], s.x);
    }
    s = unit_sum<TPR>(s, sh);
    if (!in) return;
    const float rstd = 1.f / sqrtf(s.x / c.width + c.eps);
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
        if (k >= c.width) continue;
        if (c.res_out) store_v<TR, V, WIDE>(static_cast<TR *>(c.res_out) + (size_t)row * c.width + k, r[q]);
        float w[V];
        load_v<float, V, WIDE>(c.w + k, w);
#pragma unroll
        for (int v = 0; v < V; ++v) r[q][v] *= rstd * w[v];
        store_v<T, V, WIDE>(static_cast<T *>(c.out) + (size_t)row * c.width + k, r[q]);
    }
}

// blockIdx.y: the group.
template <typename T, int V, int VPT, int TPR>
__global__ void __launch_bounds__(block_threads<TPR>()) norm_after_kernel(NormCall c) {
    constexpr bool WIDE = V > 1;
    __shared__ float2 sh[block_threads<TPR>() / 32];
    const int t = threadIdx.x % TPR, row = blockIdx.x * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
    const int gw = c.width / c.groups, g0 = blockIdx.y * gw;
    const bool in = row < c.rows;
    const T *y = static_cast<const T *>(c.x) + row * c.ld_x + g0, *z = static_cast<const T *>(c.z) + row * c.ld_z + g0;
    float a[VPT][V], gate[VPT][V];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) a[q][v] = 0.f, gate[q][v] = 1.f;
        if (!in || k >= gw) continue;
        load_v<T, V, WIDE>(y + k, a[q]);
        if (c.z) {
            load_v<T, V, WIDE>(z + k, gate[q]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                gate[q][v] = silu_v(gate[q][v]);
                if (!c.norm_first) a[q][v] *= gate[q][v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s.x = fmaf(a[q][v], a[q][v], s.x);
    }
    s = unit_sum<TPR>(s, sh);
    if (!in) return;
    const float rstd = 1.f / sqrtf(s.x / gw + c.eps);
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
        if (k >= gw) continue;
        float w[V];
        load_v<float, V, WIDE>(c.w + g0 + k, w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[q][v] *= rstd * w[v];
            if (c.norm_first) a[q][v] *= gate[q][v];
        }
        if (c.scale) {
            load_v<float, V, WIDE>(c.scale + g0 + k, w);
#pragma unroll
            for (int v = 0; v < V; ++v) a[q][v] *= w[v];
        }
        if (c.res) {
            load_v<T, V, WIDE>(static_cast<const T *>(c.res) + row * c.ld_res + g0 + k, w);
#pragma unroll
            for (int v = 0; v < V; ++v) a[q][v] += w[v];
        }
        store_v<T, V, WIDE>(static_cast<T *>(c.out) + (size_t)row * c.width + g0 + k, a[q]);
    }
}

// A block's sums over its rows, added over its units, into part[blockIdx.x][width]
// (and the dscale half after all blocks' dw).
template <int V, int VPT, int TPR>
__device__ __forceinline__ void put_parts(const float (&dw)[VPT][V], const float (&ds)[VPT][V], bool scaled, int g0, int gw,
                                          int width, float *part, float *sh) {
    constexpr int U = block_threads<TPR>() / TPR;
    const int t = threadIdx.x % TPR, unit = threadIdx.x / TPR;
    for (int what = 0; what < (scaled ? 2 : 1); ++what) {
        float *o = part + ((size_t)what * gridDim.x + blockIdx.x) * width + g0;
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int k = (q * TPR + t) * V + v;
                float s = what ? ds[q][v] : dw[q][v];
                if constexpr (U > 1) {
                    __syncthreads();
                    sh[threadIdx.x] = s;
                    __syncthreads();
                    if (unit == 0)
#pragma unroll
                        for (int i = 1; i < U; ++i) s += sh[i * TPR + t];
                }
                if (unit == 0 && k < gw) o[k] = s;
            }
    }
}

// V channels of a row as they lie in memory: the next row's are on their way while this
// one is worked on (without, the gradients take 123 us where they
// take 112 us, and 92 us where they take 80 us: 16384 x 2048, and 8192 x 8 groups of 512).
template <typename T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Raw {
    T v[V];
    __device__ __forceinline__ void get(float (&f)[V]) const { load_v<T, V, (V > 1)>(v, f); }
};
template <typename T, int V> __device__ __forceinline__ Raw<T, V> raw_at(const void *p, size_t at) {
    return *reinterpret_cast<const Raw<T, V> *>(static_cast<const T *>(p) + at);
}

template <typename T, typename TR, int V, int VPT, int TPR>
__global__ void __launch_bounds__(block_threads<TPR>()) norm_before_bwd_kernel(NormCall c, float *part) {
    constexpr bool WIDE = V > 1;
    constexpr int U = block_threads<TPR>() / TPR;
    __shared__ float2 sh[block_threads<TPR>() / 32];
    __shared__ float sums[U > 1 ? block_threads<TPR>() : 1];
    const int t = threadIdx.x % TPR, unit = threadIdx.x / TPR;
    float dw[VPT][V], ds[VPT][V], w[VPT][V];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) dw[q][v] = ds[q][v] = w[q][v] = 0.f;
        if (k < c.width) load_v<float, V, WIDE>(c.w + k, w[q]);
    }
    Raw<TR, V> nr[VPT], nu[VPT];  // r and its upstream gradient
    Raw<T, V> nd[VPT], nx[VPT];   // dout and x
    auto fetch = [&](int row) {
        if (row >= c.rows) return;
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
            if (k >= c.width) continue;
            nr[q] = raw_at<TR, V>(c.res, row * c.ld_res + k);
            nd[q] = raw_at<T, V>(c.dout, (size_t)row * c.width + k);
            if (c.dres) nu[q] = raw_at<TR, V>(c.dres, (size_t)row * c.width + k);
            if (c.scale) nx[q] = raw_at<T, V>(c.x, row * c.ld_x + k);
        }
    };
    fetch(blockIdx.x * U + unit);
    for (int row0 = blockIdx.x * U; row0 < c.rows; row0 += gridDim.x * U) {
        const int row = row0 + unit;
        const bool in = row < c.rows;
        float r[VPT][V], d[VPT][V];
        Raw<TR, V> cu[VPT];
        Raw<T, V> cx[VPT];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) r[q][v] = d[q][v] = 0.f;
            if (!in || k >= c.width) continue;
            nr[q].get(r[q]);
            nd[q].get(d[q]);
            cu[q] = nu[q], cx[q] = nx[q];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s.x = fmaf(r[q][v], r[q][v], s.x);
                s.y = fmaf(d[q][v] * w[q][v], r[q][v], s.y);
            }
        }
        fetch(row + gridDim.x * U);
        s = unit_sum<TPR>(s, sh);
        const float rstd = 1.f / sqrtf(s.x / c.width + c.eps), m = s.y * rstd / c.width;
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
            if (!in || k >= c.width) continue;
            float a[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float n = r[q][v] * rstd;
                dw[q][v] = fmaf(d[q][v], n, dw[q][v]);
                d[q][v] = rstd * (d[q][v] * w[q][v] - n * m);
            }
            if (c.dres) {
                cu[q].get(a);
#pragma unroll
                for (int v = 0; v < V; ++v) d[q][v] += a[v];
            }
            if (c.dres_out) store_v<TR, V, WIDE>(static_cast<TR *>(c.dres_out) + (size_t)row * c.width + k, d[q]);
            if (c.scale) {
                cx[q].get(a);
#pragma unroll
                for (int v = 0; v < V; ++v) ds[q][v] = fmaf(d[q][v], a[v], ds[q][v]);
                load_v<float, V, WIDE>(c.scale + k, a);
#pragma unroll
                for (int v = 0; v < V; ++v) d[q][v] *= a[v];
            }
            if (c.dx) store_v<T, V, WIDE>(static_cast<T *>(c.dx) + (size_t)row * c.width + k, d[q]);
        }
    }
    put_parts<V, VPT, TPR>(dw, ds, c.scale != nullptr, 0, c.width, c.width, part, sums);
}

// FIRST: the norm before the gate.  What is there or not (gate, scale) is asked once per
// vector, not per channel: with the questions inside, a channel took 67 instructions and
// 8192 x 8 groups of 512 took 90 us, 80 us so.
template <typename T, int V, int VPT, int TPR, bool FIRST>
__global__ void __launch_bounds__(block_threads<TPR>()) norm_after_bwd_kernel(NormCall c, float *part) {
    constexpr bool WIDE = V > 1;
    constexpr int U = block_threads<TPR>() / TPR;
    __shared__ float2 sh[block_threads<TPR>() / 32];
    __shared__ float sums[U > 1 ? block_threads<TPR>() : 1];
    const int t = threadIdx.x % TPR, unit = threadIdx.x / TPR;
    const int gw = c.width / c.groups, g0 = blockIdx.y * gw;
    float dw[VPT][V], ds[VPT][V], w[VPT][V];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int k = (q * TPR + t) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) dw[q][v] = ds[q][v] = w[q][v] = 0.f;
        if (k < gw) load_v<float, V, WIDE>(c.w + g0 + k, w[q]);
    }
    Raw<T, V> ny[VPT], nz[VPT], nd[VPT];
    auto fetch = [&](int row) {
        if (row >= c.rows) return;
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
            if (k >= gw) continue;
            ny[q] = raw_at<T, V>(c.x, row * c.ld_x + g0 + k);
            if (c.z) nz[q] = raw_at<T, V>(c.z, row * c.ld_z + g0 + k);
            nd[q] = raw_at<T, V>(c.dout, (size_t)row * c.width + g0 + k);
        }
    };
    fetch(blockIdx.x * U + unit);
    for (int row0 = blockIdx.x * U; row0 < c.rows; row0 += gridDim.x * U) {
        const int row = row0 + unit;
        const bool in = row < c.rows;
        float y[VPT][V], gate[VPT][V], sg[VPT][V], d[VPT][V];  // d: the gradient at the norm's (gated) result
        Raw<T, V> cd[VPT];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) y[q][v] = d[q][v] = 0.f, gate[q][v] = sg[q][v] = 1.f;
            if (!in || k >= gw) continue;
            ny[q].get(y[q]);
            nd[q].get(d[q]);
            cd[q] = nd[q];
            if (c.z) {
                nz[q].get(gate[q]);
#pragma unroll
                for (int v = 0; v < V; ++v) sg[q][v] = sigmoid_f(gate[q][v]), gate[q][v] *= sg[q][v];
            }
            if (c.scale) {
                float a[V];
                load_v<float, V, WIDE>(c.scale + g0 + k, a);
#pragma unroll
                for (int v = 0; v < V; ++v) d[q][v] *= a[v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float vv = FIRST ? y[q][v] : y[q][v] * gate[q][v], dm = FIRST ? d[q][v] * gate[q][v] : d[q][v];
                s.x = fmaf(vv, vv, s.x);
                s.y = fmaf(dm * w[q][v], vv, s.y);
            }
        }
        fetch(row + gridDim.x * U);
        s = unit_sum<TPR>(s, sh);
        const float rstd = 1.f / sqrtf(s.x / gw + c.eps), m = s.y * rstd / gw;
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int k = (q * TPR + t) * V;
            if (!in || k >= gw) continue;
            float dy[V], dz[V];
            if (c.scale) {
                float a[V];
                cd[q].get(a);
#pragma unroll
                for (int v = 0; v < V; ++v) ds[q][v] = fmaf(a[v], y[q][v] * gate[q][v] * (rstd * w[q][v]), ds[q][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float dgate = fmaf(gate[q][v], 1.f - sg[q][v], sg[q][v]);  // silu'(z)
                if (FIRST) {
                    const float n = y[q][v] * rstd, dm = d[q][v] * gate[q][v];
                    dw[q][v] = fmaf(dm, n, dw[q][v]);
                    dy[v] = rstd * fmaf(dm, w[q][v], -n * m);
                    dz[v] = d[q][v] * n * (w[q][v] * dgate);
                } else {
                    const float n = y[q][v] * gate[q][v] * rstd;
                    dw[q][v] = fmaf(d[q][v], n, dw[q][v]);
                    const float dv = rstd * fmaf(d[q][v], w[q][v], -n * m);
                    dy[v] = dv * gate[q][v];
                    dz[v] = dv * y[q][v] * dgate;
                }
            }
            const size_t o = (size_t)row * c.width + g0 + k;
            store_v<T, V, WIDE>(static_cast<T *>(c.dx) + o, dy);
            if (c.z) store_v<T, V, WIDE>(static_cast<T *>(c.dz) + o, dz);
        }
    }
    put_parts<V, VPT, TPR>(dw, ds, c.scale != nullptr, g0, gw, c.width, part, sums);
}

// dw (blockIdx.y 0) or dscale (1) from the blocks' parts: 32 warps take every 32nd.
__global__ void __launch_bounds__(1024) norm_bwd_sum(const float *__restrict__ part, int parts, int width,
                                                    float *__restrict__ dw, float *__restrict__ ds) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
    const float *p = part + (size_t)blockIdx.y * parts * width;
    float a = 0.f;
    if (k < width)
#pragma unroll 8
        for (int i = q; i < parts; i += 32) a += p[(size_t)i * width + k];
    s[q][lane] = a;
    __syncthreads();
    a = s[lane][q];  // column q of the block
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0 && blockIdx.x * 32 + q < width) (blockIdx.y ? ds : dw)[blockIdx.x * 32 + q] = a;
}

// Calls f with the unit's split: TPR threads (a power of two, MIN .. 512) of VPT
// vectors of V channels.  Forwards a thread takes two vectors of 16 bytes once there are
// enough units (up to 512 bf16 channels then stay in one warp: 8192 x 8 groups of 512 take
// 42.3 us, 49.6 us with one vector; eight rows of 2048 4.6 us, 4.0 us with one), and eight
// single channels where four would take more than a warp (5175 x 1333 24.5 us, 30.7 us with
// four; 20000 x 90 14.3 us, 10.2 us with four).  Backwards it takes one vector of 16 bytes
// where 512 threads reach (with two the same groups took 118 us, 101 us with one).
template <int VPT, int MIN, typename F> cudaError_t with_tpr(int vectors, F &&f) {
    const int need = (vectors + VPT - 1) / VPT;
    constexpr std::integral_constant<int, VPT> vpt{};
    if constexpr (MIN <= 32)
        if (need <= 32) return f(vpt, std::integral_constant<int, 32>{});
    if constexpr (MIN <= 64)
        if (need <= 64) return f(vpt, std::integral_constant<int, 64>{});
    if constexpr (MIN <= 128)
        if (need <= 128) return f(vpt, std::integral_constant<int, 128>{});
    if constexpr (MIN <= 256)
        if (need <= 256) return f(vpt, std::integral_constant<int, 256>{});
    return f(vpt, std::integral_constant<int, 512>{});
}
template <int V, typename F> cudaError_t with_split(int width, bool two, F &&f) {
    static_assert(NORM_MAX_WIDTH == 8192, "the splits below end there");
    const int vectors = (width + V - 1) / V;
    if constexpr (V <= 2) {
        if constexpr (V == 1) {
            if (vectors > 4096) return with_tpr<16, 512>(vectors, f);
            if (two && vectors > 128 && vectors <= 2048) return with_tpr<8, 32>(vectors, f);
        }
        if (vectors <= 2048) return with_tpr<4, 32>(vectors, f);
        return with_tpr<8, 512>(vectors, f);
    } else {
        if (vectors <= (two ? 32 : 512)) return with_tpr<1, 32>(vectors, f);
        if constexpr (V == 4)
            if (vectors > 1024) return with_tpr<4, 512>(vectors, f);
        return with_tpr<2, 32>(vectors, f);
    }
}

template <typename T, typename TR, int V> cudaError_t run_before(const NormCall &c, cudaStream_t st) {
    return with_split<V>(c.width, c.rows >= MANY_UNITS, [&](auto vpt, auto tpr) {
        constexpr int TH = block_threads<tpr()>(), U = TH / tpr();
        norm_before_kernel<T, TR, V, vpt(), tpr()><<<(c.rows + U - 1) / U, TH, 0, st>>>(c);
        return cudaGetLastError();
    });
}
template <typename T, int V> cudaError_t run_after(const NormCall &c, cudaStream_t st) {
    return with_split<V>(c.width / c.groups, (long long)c.rows * c.groups >= MANY_UNITS, [&](auto vpt, auto tpr) {
        constexpr int TH = block_threads<tpr()>(), U = TH / tpr();
        norm_after_kernel<T, V, vpt(), tpr()><<<dim3((c.rows + U - 1) / U, c.groups), TH, 0, st>>>(c);
        return cudaGetLastError();
    });
}
int bwd_blocks(int rows, int units, int threads, int groups) {
    return min((rows + units - 1) / units, max(1, BWD_BLOCKS * 256 / threads / groups));
}
cudaError_t run_sum(const NormCall &c, const float *ws, int parts, cudaStream_t st) {
    norm_bwd_sum<<<dim3((c.width + 31) / 32, c.scale ? 2 : 1), 1024, 0, st>>>(ws, parts, c.width, c.dw, c.dscale);
    return cudaGetLastError();
}
template <typename T, typename TR, int V> cudaError_t run_before_bwd(const NormCall &c, float *ws, cudaStream_t st) {
    return with_split<V>(c.width, false, [&](auto vpt, auto tpr) {
        constexpr int TH = block_threads<tpr()>(), U = TH / tpr();
        const int blocks = bwd_blocks(c.rows, U, TH, 1);
        if (blocks > 0) norm_before_bwd_kernel<T, TR, V, vpt(), tpr()><<<blocks, TH, 0, st>>>(c, ws);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? run_sum(c, ws, blocks, st) : e;
    });
}
template <typename T, int V> cudaError_t run_after_bwd(const NormCall &c, float *ws, cudaStream_t st) {
    return with_split<V>(c.width / c.groups, false, [&](auto vpt, auto tpr) {
        constexpr int TH = block_threads<tpr()>(), U = TH / tpr();
        const int blocks = bwd_blocks(c.rows, U, TH, c.groups);
        if (blocks > 0 && c.norm_first) norm_after_bwd_kernel<T, V, vpt(), tpr(), true><<<dim3(blocks, c.groups), TH, 0, st>>>(c, ws);
        if (blocks > 0 && !c.norm_first) norm_after_bwd_kernel<T, V, vpt(), tpr(), false><<<dim3(blocks, c.groups), TH, 0, st>>>(c, ws);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? run_sum(c, ws, blocks, st) : e;
    });
}

// Whether every row (and group) can be read as vectors of V channels, at most 16 bytes an
// access.
bool wide_rows(const NormCall &c, int V) {
    const size_t e = c.bf16 ? 2 : 4, er = c.res_bf16 ? 2 : 4;
    return c.width % V == 0 && (c.width / c.groups) % V == 0 && (!c.x || rows_aligned(c.x, c.ld_x, e, min(16, V * (int)e))) &&
           (!c.z || rows_aligned(c.z, c.ld_z, e, min(16, V * (int)e))) && (!c.res || rows_aligned(c.res, c.ld_res, er, min(16, V * (int)er)));
}

// Calls f with the channels of a vector: 16 bytes of the io type, pairs, or single ones
// (bf16, norm after: 5175 x 1332 channels in pairs 20 us and 42 us backwards, single 31 and
// 66; 8192 x 4004 82 and 212, single 170 and 647).  Backwards up to 512 channels stay single:
// 8192 x 8 groups of 500 take 166 us so and 199 us in pairs.
template <typename F> cudaError_t with_vectors(const NormCall &c, bool backward, F &&f) {
    if (wide_rows(c, c.bf16 ? 8 : 4)) return f(std::integral_constant<int, 8>{});
    if (wide_rows(c, 2) && (!backward || c.width / c.groups > 512)) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}
// .. and with the types of the io and the residual.
template <typename F> cudaError_t with_types(const NormCall &c, bool backward, F &&f) {
    using H = __nv_bfloat16;
    return with_vectors(c, backward, [&](auto v) {
        constexpr std::integral_constant<int, (v() > 4 ? 4 : v())> v4{};
        if (!c.bf16) return f(float(), float(), v4);
        return c.res_bf16 ? f(H(), H(), v) : f(H(), float(), v);
    });
}

}  // namespace

cudaError_t launch_norm_before(const NormCall &c, cudaStream_t st) {
    return with_types(c, false, [&](auto t, auto r, auto v) { return run_before<decltype(t), decltype(r), v()>(c, st); });
}
cudaError_t launch_norm_after(const NormCall &c, cudaStream_t st) {
    return with_types(c, false, [&](auto t, auto r, auto v) {
        return std::is_same<decltype(t), decltype(r)>::value ? run_after<decltype(t), v()>(c, st) : cudaErrorInvalidValue;
    });
}
size_t norm_bwd_workspace(int rows, int width) {  // blocks have 128 threads at least
    return 2 * (size_t)min(rows, 2 * BWD_BLOCKS) * width * sizeof(float);
}
cudaError_t launch_norm_before_bwd(const NormCall &c, float *ws, cudaStream_t st) {
    return with_types(c, true, [&](auto t, auto r, auto v) { return run_before_bwd<decltype(t), decltype(r), v()>(c, ws, st); });
}
cudaError_t launch_norm_after_bwd(const NormCall &c, float *ws, cudaStream_t st) {
    return with_types(c, true, [&](auto t, auto r, auto v) {
        return std::is_same<decltype(t), decltype(r)>::value ? run_after_bwd<decltype(t), v()>(c, ws, st) : cudaErrorInvalidValue;
    });
}

}  // namespace ssd
