// selscan.cu -- the Mamba-1 selective scan on packed sequences and on single tokens.
//
//   delta_t = softplus(dt_t + bias) (or dt_t + bias),
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)          per channel.
//
// A block takes one sequence and SEL_WARPS * 32 / TL channels of one B/C group and
// walks the sequence in chunks; inside a chunk the tokens of a channel are split
// over TL lanes (selscan_tile.cuh).  The split over time inside the warp keeps the
// exponentials at one per state and token, where a second pass over chunks would
// double them, and gives a single prompt enough warps.  Bound by the exponential
// unit (N per channel and token at 16 per SM and clock) and by issue, then HBM.
#include "selscan_tile.cuh"

namespace ssd {
namespace {

template <typename T, int TL, int K> struct FwdShape {
    static constexpr int SEG = TL * K, CL = 32 / TL, CB = SEL_WARPS * CL;
    using Rows = RowTile<T, SEG, CB, TL>;
    using BC = BCTile<T, SEG, TL>;
    static size_t smem(int N) { return 3 * (size_t)Rows::BYTES + (size_t)N * BC::STATE_WORDS * 4 + 2 * (size_t)CB * N * 4; }
};

// One chunk: the lane's tokens (4 Q slots, `mine` of them real) of channel ch, over
// all states.  Q is a compile-time number so that the arrays stay in registers and
// the state loop has no branches.
template <typename T, int TL, int K, int Q>
__device__ __forceinline__ void fwd_chunk(const SelCall &c, unsigned char *xs, unsigned char *ds, unsigned char *zs,
                                          const uint32_t *bc, const float *As, float *hs, int l, int ch, int mine, float bias,
                                          float Dv) {
    using S = FwdShape<T, TL, K>;
    using Rows = typename S::Rows;
    using BC = typename S::BC;
    constexpr int CB = S::CB, LEN = 4 * Q;
    const int N = c.dstate;
    float2 dl[LEN / 2], u2[LEN / 2], y2[LEN / 2];
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        float d = 0.f, u = 0.f;
        if (k < mine) {
            d = ld_f32<T>(Rows::row(ds, l * LEN + k, l) + ch) + bias;
            if (c.softplus) d = softplus_f(d);
            u = d * ld_f32<T>(Rows::row(xs, l * LEN + k, l) + ch);
        }
        total += d;
        if (k & 1)
            dl[k / 2].y = d, u2[k / 2].y = u;
        else
            dl[k / 2].x = d, u2[k / 2].x = u;
    }
#pragma unroll
    for (int k = 0; k < LEN / 2; ++k) y2[k] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int s = 0; s < N; ++s) {
        const float A2 = As[s * CB + ch], hc = hs[s * CB + ch];
        const float2 A22 = splat(A2);
        float2 a2[LEN / 2], b2[LEN / 2], c2[LEN / 2];
        float S_ = 0.f, P = ex2a(A2 * total);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            BC::quad(bc, s, q, l, b2 + 2 * q, c2 + 2 * q);
#pragma unroll
            for (int k = 2 * q; k < 2 * q + 2; ++k) {
                const float2 arg = mul2(dl[k], A22);
                a2[k] = make_float2(ex2a(arg.x), ex2a(arg.y));
                b2[k] = mul2(u2[k], b2[k]);
                S_ = fmaf(a2[k].x, S_, b2[k].x);
                S_ = fmaf(a2[k].y, S_, b2[k].y);
            }
        }
        if (l == 0) S_ = fmaf(P, hc, S_);
#pragma unroll
        for (int o = 1; o < TL; o *= 2) {
            const float Sp = __shfl_up_sync(0xffffffffu, S_, o, TL), Pp = __shfl_up_sync(0xffffffffu, P, o, TL);
            if (l >= o) S_ = fmaf(P, Sp, S_), P *= Pp;
        }
        float h = __shfl_up_sync(0xffffffffu, S_, 1, TL);
        if (l == 0) h = hc;
        if (l == TL - 1) hs[s * CB + ch] = S_;
#pragma unroll
        for (int k = 0; k < LEN / 2; ++k) {
            float2 hh;
            hh.x = h = fmaf(a2[k].x, h, b2[k].x);
            hh.y = h = fmaf(a2[k].y, h, b2[k].y);
            y2[k] = fma2(c2[k], hh, y2[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        if (k < mine) {
            T *px = Rows::row(xs, l * LEN + k, l) + ch;
            float o = fmaf(Dv, ld_f32<T>(px), k & 1 ? y2[k / 2].y : y2[k / 2].x);
            if (c.z) o *= silu_v(ld_f32<T>(Rows::row(zs, l * LEN + k, l) + ch));
            st_f32<T>(px, o);
        }
    }
}

template <typename T, int TL, int K>
__global__ void __launch_bounds__(SEL_WARPS * 32, 2) sel_fwd_kernel(SelCall c, bool wide, bool wide_bc) {
    using S = FwdShape<T, TL, K>;
    using Rows = typename S::Rows;
    using BC = typename S::BC;
    constexpr int SEG = S::SEG, CB = S::CB;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char *xs = smem, *ds = xs + Rows::BYTES, *zs = ds + Rows::BYTES;
    uint32_t *bc = reinterpret_cast<uint32_t *>(zs + Rows::BYTES);
    const int N = c.dstate;
    float *As = reinterpret_cast<float *>(bc + N * BC::STATE_WORDS), *hs = As + CB * N;  // [n][channel]

    const int i = blockIdx.x;
    int lo, hi;
    if (!seq_rows(c.seq, i, lo, hi) || lo == hi) return;  // the same for the whole block
    const int per_group = c.channels / c.groups, tiles = (per_group + CB - 1) / CB;
    const int g = blockIdx.y / tiles, c0 = g * per_group + (blockIdx.y % tiles) * CB;
    const int cols = min(CB, (g + 1) * per_group - c0);
    const int slot = c.state ? slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error) : -1;
    const bool init = slot >= 0 && c.seq.has_init && c.seq.has_init[i];
    float *st = c.state + (slot >= 0 ? ((size_t)slot * c.channels + c0) * N : 0);
    for (int u = threadIdx.x; u < CB * N; u += SEL_WARPS * 32) {
        const int ch = u / N, n = u - ch * N;
        const bool in = ch < cols;
        As[n * CB + ch] = in ? c.A[(size_t)c0 * N + u] * LOG2E : 0.f;
        hs[n * CB + ch] = in && init ? st[u] : 0.f;
    }
    const int lane = threadIdx.x & 31, l = lane % TL, ch = (threadIdx.x >> 5) * S::CL + lane / TL;
    const int chc = min(ch, cols - 1);
    const float bias = c.dt_bias ? c.dt_bias[c0 + chc] : 0.f, Dv = c.D ? c.D[c0 + chc] : 0.f;
    const T *x = static_cast<const T *>(c.x) + c0, *dt = static_cast<const T *>(c.dt) + c0,
            *z = static_cast<const T *>(c.z) + c0;
    const T *B = static_cast<const T *>(c.B) + g * N, *C = static_cast<const T *>(c.C) + g * N;
    T *y = static_cast<T *>(c.y) + c0;

    for (int t0 = lo, chunk = 0; t0 < hi; t0 += SEG, ++chunk) {
        const int n = min(SEG, hi - t0), len = ((n + TL - 1) / TL + 3) & ~3;
        Rows::fetch(xs, x + t0 * c.ld_x, c.ld_x, n, cols, len, wide);
        Rows::fetch(ds, dt + t0 * c.ld_dt, c.ld_dt, n, cols, len, wide);
        if (c.z) Rows::fetch(zs, z + t0 * c.ld_z, c.ld_z, n, cols, len, wide);
        cp_commit();
        BC::fetch(bc, B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, n, N, len, wide_bc);
        cp_wait<0>();
        __syncthreads();
        if (c.chunk_states) {  // SEG == SEL_CHUNK then
            float *o = c.chunk_states + ((size_t)(lo / SEL_CHUNK + i + chunk) * c.channels + c0) * N;
            for (int u = threadIdx.x; u < cols * N; u += SEL_WARPS * 32) o[u] = hs[(u % N) * CB + u / N];
            __syncthreads();  // before hs moves on
        }
        const int mine = ch < cols ? max(0, min(len, n - l * len)) : 0;  // tokens of this lane
        switch (len / 4) {
        case 1: fwd_chunk<T, TL, K, 1>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv); break;
        case 2: fwd_chunk<T, TL, K, 2>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv); break;
        case 3: fwd_chunk<T, TL, K, 3>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv); break;
        default: fwd_chunk<T, TL, K, 4>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv); break;
        }
        __syncthreads();
        Rows::flush(xs, y + (size_t)t0 * c.channels, c.channels, n, cols, len, wide);
        __syncthreads();  // before the next chunk's copies
    }
    if (slot >= 0)
        for (int u = threadIdx.x; u < cols * N; u += SEL_WARPS * 32) st[u] = hs[(u % N) * CB + u / N];
}

// One token per sequence, in place on the state.  LP lanes share a channel, four
// states each (dstate = 4 LP), so a warp reads and writes whole lines of the state; a
// thread takes U channels, a block's stride apart, with all its loads first.
// LP = 0: any dstate, a lane per channel.  Bound by HBM: the state in and out.
constexpr int UPD_THREADS = 256;
template <typename T, int LP, int U>
__global__ void __launch_bounds__(UPD_THREADS) sel_update_kernel(SelCall c, bool wide_bc) {
    constexpr int L = LP ? LP : 1, CH = UPD_THREADS / L;  // channels per block and step
    const int i = blockIdx.y, N = c.dstate, q = threadIdx.x % L, per_group = c.channels / c.groups;
    const int d0 = blockIdx.x * CH * U + threadIdx.x / L;
    // everything that does not depend on the slot is on its way while the slot is looked up
    float xv[U], dt[U], zv[U], bias[U], Dv[U];
    float4 a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int d = min(d0 + u * CH, c.channels - 1);
        xv[u] = ld_f32<T>(static_cast<const T *>(c.x) + i * c.ld_x + d);
        dt[u] = ld_f32<T>(static_cast<const T *>(c.dt) + i * c.ld_dt + d);
        zv[u] = c.z ? ld_f32<T>(static_cast<const T *>(c.z) + i * c.ld_z + d) : 0.f;
        bias[u] = c.dt_bias ? c.dt_bias[d] : 0.f;
        Dv[u] = c.D ? c.D[d] : 0.f;
        if constexpr (LP > 0) a[u] = __ldg(reinterpret_cast<const float4 *>(c.A + (size_t)d * N) + q);
    }
    const int slot = slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error);
    if (slot < 0) return;
    float *st = c.state + (size_t)slot * c.channels * N;
    float4 h[U];
    if constexpr (LP > 0)
#pragma unroll
        for (int u = 0; u < U; ++u)
            h[u] = __ldcs(reinterpret_cast<const float4 *>(st + (size_t)min(d0 + u * CH, c.channels - 1) * N) + q);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int d = d0 + u * CH;
        const bool in = d < c.channels;
        const int g = min(d, c.channels - 1) / per_group;
        const T *B = static_cast<const T *>(c.B) + i * c.ld_b + g * N, *C = static_cast<const T *>(c.C) + i * c.ld_c + g * N;
        float delta = dt[u] + bias[u], acc = 0.f;
        if (c.softplus) delta = softplus_f(delta);
        const float du = delta * xv[u], d2 = delta * LOG2E;
        if constexpr (LP > 0) {
            float b[4], cv[4];
            if (wide_bc) {
                load_v<T, 4, true>(B + 4 * q, b), load_v<T, 4, true>(C + 4 * q, cv);
            } else {
                load_v<T, 4, false>(B + 4 * q, b), load_v<T, 4, false>(C + 4 * q, cv);
            }
            h[u].x = fmaf(ex2a(d2 * a[u].x), h[u].x, du * b[0]);
            h[u].y = fmaf(ex2a(d2 * a[u].y), h[u].y, du * b[1]);
            h[u].z = fmaf(ex2a(d2 * a[u].z), h[u].z, du * b[2]);
            h[u].w = fmaf(ex2a(d2 * a[u].w), h[u].w, du * b[3]);
            acc = fmaf(cv[0], h[u].x, fmaf(cv[1], h[u].y, fmaf(cv[2], h[u].z, cv[3] * h[u].w)));
            if (in) __stcs(reinterpret_cast<float4 *>(st + (size_t)d * N) + q, h[u]);
#pragma unroll
            for (int o = 1; o < L; o *= 2) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        } else if (in) {
            for (int n = 0; n < N; ++n) {
                float *hn = st + (size_t)d * N + n;
                *hn = fmaf(ex2a(d2 * c.A[(size_t)d * N + n]), *hn, du * ld_f32<T>(B + n));
                acc = fmaf(ld_f32<T>(C + n), *hn, acc);
            }
        }
        if (in && q == 0) {
            float o = fmaf(Dv[u], xv[u], acc);
            if (c.z) o *= silu_v(zv[u]);
            st_f32<T>(static_cast<T *>(c.y) + (size_t)i * c.channels + d, o);
        }
    }
}

template <typename T, int TL, int K> cudaError_t run_fwd(const SelCall &c, cudaStream_t st) {
    using S = FwdShape<T, TL, K>;
    const size_t smem = S::smem(c.dstate), e = sizeof(T);
    const int per_group = c.channels / c.groups;
    const bool wide = rows_aligned(c.x, c.ld_x, e, 16) && rows_aligned(c.dt, c.ld_dt, e, 16) &&
                      (!c.z || rows_aligned(c.z, c.ld_z, e, 16)) && rows_aligned(c.y, c.channels, e, 16) &&
                      per_group * e % 16 == 0;
    const bool wide_bc = c.dstate % 4 == 0 && rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
    cudaError_t err = cudaFuncSetAttribute(sel_fwd_kernel<T, TL, K>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    const dim3 grid(c.seq.nseq, c.groups * ((per_group + S::CB - 1) / S::CB));
    sel_fwd_kernel<T, TL, K><<<grid, SEL_WARPS * 32, smem, st>>>(c, wide, wide_bc);
    return cudaGetLastError();
}

template <typename T> cudaError_t pick_fwd(const SelCall &c, cudaStream_t st) {
    const long long blocks = (long long)c.seq.nseq * ((c.channels + 31) / 32);
    if (!c.chunk_states && c.dstate <= 16 && blocks < 148) return run_fwd<T, 32, 16>(c, st);
    return run_fwd<T, 8, 16>(c, st);
}

template <typename T, int LP, int U> cudaError_t run_update(const SelCall &c, int batch, bool wide_bc, cudaStream_t st) {
    const int per = UPD_THREADS / (LP ? LP : 1) * U;
    sel_update_kernel<T, LP, U><<<dim3((c.channels + per - 1) / per, batch), UPD_THREADS, 0, st>>>(c, wide_bc);
    return cudaGetLastError();
}
// Four channels per thread once that still leaves every SM eight blocks.
template <typename T, int LP> cudaError_t run_update(const SelCall &c, int batch, cudaStream_t st) {
    const size_t e = sizeof(T);
    const bool wide_bc = rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
    const long long blocks = (long long)batch * c.channels * (LP ? LP : 1) / (UPD_THREADS * 4);
    return blocks >= 148 * 8 ? run_update<T, LP, 4>(c, batch, wide_bc, st) : run_update<T, LP, 1>(c, batch, wide_bc, st);
}
template <typename T> cudaError_t pick_update(const SelCall &c, int batch, cudaStream_t st) {
    switch (c.dstate) {
    case 4: return run_update<T, 1>(c, batch, st);
    case 8: return run_update<T, 2>(c, batch, st);
    case 16: return run_update<T, 4>(c, batch, st);
    case 32: return run_update<T, 8>(c, batch, st);
    case 64: return run_update<T, 16>(c, batch, st);
    default: return run_update<T, 0>(c, batch, st);
    }
}

}  // namespace

cudaError_t launch_sel_varlen(const SelCall &c, cudaStream_t st) {
    return c.bf16 ? pick_fwd<__nv_bfloat16>(c, st) : pick_fwd<float>(c, st);
}
cudaError_t launch_sel_update(const SelCall &c, int batch, cudaStream_t st) {
    return c.bf16 ? pick_update<__nv_bfloat16>(c, batch, st) : pick_update<float>(c, batch, st);
}

}  // namespace ssd
