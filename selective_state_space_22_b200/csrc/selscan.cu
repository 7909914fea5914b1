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
    T *const px = Rows::row(xs, l * LEN, l) + ch;
    const T *const pd = Rows::row(ds, l * LEN, l) + ch, *const pz = Rows::row(zs, l * LEN, l) + ch;
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        const bool in = k < mine;
        float d = ld_f32<T>(pd + k * CB) + bias;
        if (c.softplus) d = softplus_f(d);
        d = in ? d : 0.f;
        const float u = in ? d * ld_f32<T>(px + k * CB) : 0.f;
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
        float o = fmaf(Dv, ld_f32<T>(px + k * CB), k & 1 ? y2[k / 2].y : y2[k / 2].x);
        if (c.z) o *= silu_v(ld_f32<T>(pz + k * CB));
        if (k < mine) st_f32<T>(px + k * CB, o);
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
        const int n = min(SEG, hi - t0), per_lane = (n + TL - 1) / TL, len = per_lane <= 4 ? 4 : per_lane <= 8 ? 8 : K;
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
        if (len == 4)
            fwd_chunk<T, TL, K, 1>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv);
        else if (len == 8)
            fwd_chunk<T, TL, K, 2>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv);
        else
            fwd_chunk<T, TL, K, 4>(c, xs, ds, zs, bc, As, hs, l, ch, mine, bias, Dv);
        __syncthreads();
        Rows::flush(xs, y + (size_t)t0 * c.channels, c.channels, n, cols, len, wide);
        __syncthreads();  // before the next chunk's copies
    }
    if (slot >= 0)
        for (int u = threadIdx.x; u < cols * N; u += SEL_WARPS * 32) st[u] = hs[(u % N) * CB + u / N];
}

// One token per sequence, in place on the state.  A warp takes 32 channels.  Each lane
// does the scalar work (step size, gate) of one; for the states, the LP lanes of a
// group go through their LP channels together, four states a lane (dstate = 4 LP), so
// that a group reads and writes whole rows of the state, all loads first, and a lane
// ends with its own channel's readout.  (LP lanes doing the scalar work of each of
// their channels together measured 43.6 us against KERNEL us for 256 x 4096 channels
// of 16 states: five times the instructions.)  LP = 0: any dstate, a lane per channel.
// SAME: the warp's channels lie in one B/C group.  Bound by HBM: the state in and out.
constexpr int UPD_THREADS = 128;
template <typename T, int LP, bool SAME>
__global__ void __launch_bounds__(UPD_THREADS) sel_update_kernel(SelCall c, bool wide_bc) {
    constexpr int L = LP ? LP : 1;
    const int i = blockIdx.y, N = c.dstate, lane = threadIdx.x & 31, q = lane % L, per_group = c.channels / c.groups;
    const int d = blockIdx.x * UPD_THREADS + threadIdx.x, d0 = d - q;  // own channel, first of the lane's group
    const int last = c.channels - 1, dc = min(d, last);
    // what does not depend on the slot is on its way while the slot is looked up
    const float xv = ld_f32<T>(static_cast<const T *>(c.x) + i * c.ld_x + dc);
    float delta = ld_f32<T>(static_cast<const T *>(c.dt) + i * c.ld_dt + dc) + (c.dt_bias ? c.dt_bias[dc] : 0.f);
    const float zv = c.z ? ld_f32<T>(static_cast<const T *>(c.z) + i * c.ld_z + dc) : 0.f;
    const float Dv = c.D ? c.D[dc] : 0.f;
    const T *B = static_cast<const T *>(c.B) + i * c.ld_b, *C = static_cast<const T *>(c.C) + i * c.ld_c;
    float4 a[L];
    if constexpr (LP > 0 && LP <= 4)  // registers allow it
#pragma unroll
        for (int u = 0; u < L; ++u) a[u] = __ldg(reinterpret_cast<const float4 *>(c.A + (size_t)min(d0 + u, last) * N) + q);
    const int slot = slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error);
    if (slot < 0) return;
    float *st = c.state + (size_t)slot * c.channels * N;
    float y = 0.f;
    if constexpr (LP > 0) {
        float4 h[L];
#pragma unroll
        for (int u = 0; u < L; ++u) h[u] = __ldcs(reinterpret_cast<const float4 *>(st + (size_t)min(d0 + u, last) * N) + q);
        if (c.softplus) delta = softplus_f(delta);
        const float du = delta * xv, d2 = delta * LOG2E;
        float b[4], cv[4], acc[L];
        auto load_bc = [&](int g) {
            if (wide_bc) {
                load_v<T, 4, true>(B + g * N + 4 * q, b), load_v<T, 4, true>(C + g * N + 4 * q, cv);
            } else {
                load_v<T, 4, false>(B + g * N + 4 * q, b), load_v<T, 4, false>(C + g * N + 4 * q, cv);
            }
        };
        if (SAME) load_bc(min(d - lane, last) / per_group);
#pragma unroll
        for (int u = 0; u < L; ++u) {
            const int du_ = min(d0 + u, last);
            if (!SAME) load_bc(du_ / per_group);
            if (LP > 4) a[u] = __ldg(reinterpret_cast<const float4 *>(c.A + (size_t)du_ * N) + q);
            const float s2 = __shfl_sync(0xffffffffu, d2, u, L), su = __shfl_sync(0xffffffffu, du, u, L);
            h[u].x = fmaf(ex2a(s2 * a[u].x), h[u].x, su * b[0]);
            h[u].y = fmaf(ex2a(s2 * a[u].y), h[u].y, su * b[1]);
            h[u].z = fmaf(ex2a(s2 * a[u].z), h[u].z, su * b[2]);
            h[u].w = fmaf(ex2a(s2 * a[u].w), h[u].w, su * b[3]);
            acc[u] = fmaf(cv[0], h[u].x, fmaf(cv[1], h[u].y, fmaf(cv[2], h[u].z, cv[3] * h[u].w)));
            if (d0 + u <= last) __stcs(reinterpret_cast<float4 *>(st + (size_t)du_ * N) + q, h[u]);
        }
        // each step halves the channels a lane still sums: lane q ends with channel q
#pragma unroll
        for (int n = L / 2; n > 0; n /= 2)
#pragma unroll
            for (int u = 0; u < n; ++u) {
                const float keep = q & n ? acc[u + n] : acc[u], give = q & n ? acc[u] : acc[u + n];
                acc[u] = keep + __shfl_xor_sync(0xffffffffu, give, n);
            }
        y = acc[0];
    } else if (d <= last) {
        if (c.softplus) delta = softplus_f(delta);
        const float du = delta * xv, d2 = delta * LOG2E;
        const int g = d / per_group;
        for (int n = 0; n < N; ++n) {
            float *hn = st + (size_t)d * N + n;
            *hn = fmaf(ex2a(d2 * c.A[(size_t)d * N + n]), *hn, du * ld_f32<T>(B + g * N + n));
            y = fmaf(ld_f32<T>(C + g * N + n), *hn, y);
        }
    }
    if (d <= last) {
        y = fmaf(Dv, xv, y);
        if (c.z) y *= silu_v(zv);
        st_f32<T>(static_cast<T *>(c.y) + (size_t)i * c.channels + d, y);
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

template <typename T, int LP> cudaError_t run_update(const SelCall &c, int batch, cudaStream_t st) {
    const size_t e = sizeof(T);
    const bool wide_bc = rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
    const dim3 grid((c.channels + UPD_THREADS - 1) / UPD_THREADS, batch);
    if (c.groups == 1 || c.channels / c.groups % 32 == 0)
        sel_update_kernel<T, LP, true><<<grid, UPD_THREADS, 0, st>>>(c, wide_bc);
    else
        sel_update_kernel<T, LP, false><<<grid, UPD_THREADS, 0, st>>>(c, wide_bc);
    return cudaGetLastError();
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
