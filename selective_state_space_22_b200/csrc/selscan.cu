// selscan.cu -- the Mamba-1 selective scan on packed sequences and on single tokens.
//
//   delta_t = softplus(dt_t + bias) (or dt_t + bias),
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)          per channel.
//
// A thread per channel, its states in registers, along a sequence or a segment of one
// (selscan_seg.cuh): three packed operations and an exponential per state and token,
// some forty more per token.  x, dt, z and y go straight between global memory and
// registers (neighbouring lanes, neighbouring channels), four tokens ahead; B and C,
// which a block's channels share, through shared memory.  Bound by the exponential
// unit (N + 4 operations per channel and token at 16 per SM and clock), then by issue.
// A first form split the tokens of a chunk over the lanes of a warp, with one
// exponential per state and token at any length; its scans over lanes and the second
// walk they need left it at 352 us where this one takes KERNEL_TIME (64 x 512 tokens,
// 1024 channels, 16 states).
#include "selscan_seg.cuh"

namespace ssd {
namespace {

constexpr int FWD_THREADS = 64, AHEAD = 4;

// FULL: y, kept states and the end state; else only what sel_join needs.
template <typename T, int NP, bool FULL>
__global__ void __launch_bounds__(FWD_THREADS) sel_fwd_kernel(SelCall c, Segments sg, bool wide) {
    constexpr int P = NP / 2, TT = NP <= 16 ? 32 : 16;
    using Stage = StageBC<T, NP, TT, FWD_THREADS>;
    __shared__ __align__(16) float4 bc[2][Stage::BYTES / 16];
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end)) return;  // the same for the whole block
    if (!FULL && hi == end) return;  // nothing follows
    const Mine me = my_channel<FWD_THREADS>(c, blockIdx.y);
    const int N = c.dstate, d = me.channel, slot = FULL && c.state ? slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error) : -1;
    const T *B = static_cast<const T *>(c.B) + me.group * N + lo * c.ld_b, *C = static_cast<const T *>(c.C) + me.group * N + lo * c.ld_c;
    Stage stage;
    stage.load(B, c.ld_b, C, c.ld_c, min(TT, hi - lo), N, wide);
    float2 A2[P], h[P];
    float *const state = c.state + (slot >= 0 ? ((size_t)slot * c.channels + d) * N : 0);
    const bool init = slot >= 0 && c.seq.has_init && c.seq.has_init[i] && sg.seg == WHOLE;
    float *const carried = sg.state + ((size_t)blockIdx.x * N) * c.channels + d;
    auto load_h = [&](int n) {
        if (n >= N) return 0.f;
        if (FULL && sg.seg != WHOLE) return carried[(size_t)n * c.channels];
        return init ? state[n] : 0.f;
    };
#pragma unroll
    for (int p = 0; p < P; ++p) {
        A2[p] = make_float2(2 * p < N ? c.A[(size_t)d * N + 2 * p] * LOG2E : 0.f, 2 * p + 1 < N ? c.A[(size_t)d * N + 2 * p + 1] * LOG2E : 0.f);
        h[p] = make_float2(load_h(2 * p), load_h(2 * p + 1));
    }
    const float bias = c.dt_bias ? c.dt_bias[d] : 0.f, Dv = c.D ? c.D[d] : 0.f;
    const T *px = static_cast<const T *>(c.x) + lo * c.ld_x + d, *pd = static_cast<const T *>(c.dt) + lo * c.ld_dt + d;
    const T *pz = static_cast<const T *>(c.z) + (c.z ? lo * c.ld_z + d : 0);
    T *py = static_cast<T *>(c.y) + (size_t)lo * c.channels + d;
    T nx[AHEAD], nd[AHEAD], nz[AHEAD];
    int left = hi - lo;  // tokens not yet fetched
    auto fetch = [&] {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (k < left) {
                nx[k] = *px, nd[k] = *pd;
                if (FULL && c.z) nz[k] = *pz, pz += c.ld_z;
                px += c.ld_x, pd += c.ld_dt;
            }
        }
        left -= AHEAD;
    };
    fetch();
    stage.put(bc[0]);
    float steps = 0.f;
    float *kept = nullptr;
    if (FULL && c.chunk_states) kept = c.chunk_states + ((size_t)(first / SEL_CHUNK + i + (lo - first) / SEL_CHUNK) * N) * c.channels + d;
    for (int t0 = lo, buf = 0; t0 < hi; t0 += TT, buf ^= 1) {
        const int nt = min(TT, hi - t0);
        B += TT * c.ld_b, C += TT * c.ld_c;
        if (t0 + TT < hi) stage.load(B, c.ld_b, C, c.ld_c, min(TT, hi - t0 - TT), N, wide);
        __syncthreads();  // bc[buf] is written, and nobody reads bc[buf ^ 1] any more
#pragma unroll 1
        for (int t = 0; t < nt; t += AHEAD) {
            float dl[AHEAD], xv[AHEAD], gate[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                xv[k] = ld_f32<T>(&nx[k]);
                dl[k] = ld_f32<T>(&nd[k]) + bias;
                if (c.softplus) dl[k] = softplus_f(dl[k]);
                if (FULL) gate[k] = c.z ? silu_v(ld_f32<T>(&nz[k])) : 1.f;
            }
            fetch();
            if (FULL && kept && (t0 - first + t) % SEL_CHUNK == 0) {
                if (me.in)
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        if (n < N) kept[(size_t)n * c.channels] = n & 1 ? h[n / 2].y : h[n / 2].x;
                kept += (size_t)N * c.channels;
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (t + k >= nt) break;
                const float2 d2 = splat(dl[k]), u2 = splat(dl[k] * xv[k]);
                float2 y2 = make_float2(0.f, 0.f);
                const float4 *q = bc[buf] + (t + k) * P;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float4 v = q[p];
                    const float2 arg = mul2(d2, A2[p]);
                    h[p] = fma2(make_float2(ex2a(arg.x), ex2a(arg.y)), h[p], mul2(u2, make_float2(v.x, v.y)));
                    if (FULL) y2 = fma2(make_float2(v.z, v.w), h[p], y2);
                }
                if (FULL) {
                    if (me.in) st_f32<T>(py, fmaf(Dv, xv[k], y2.x + y2.y) * gate[k]);
                    py += c.channels;
                } else {
                    steps += dl[k];
                }
            }
        }
        if (t0 + TT < hi) stage.put(bc[buf ^ 1]);
    }
    if (!me.in) return;
    if (FULL) {
        if (slot >= 0 && hi == end)
#pragma unroll
            for (int n = 0; n < NP; ++n)
                if (n < N) state[n] = n & 1 ? h[n / 2].y : h[n / 2].x;
    } else {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < N) carried[(size_t)n * c.channels] = n & 1 ? h[n / 2].y : h[n / 2].x;
        sg.steps[(size_t)blockIdx.x * c.channels + d] = steps;
    }
}

// A thread per (sequence, state, channel) goes through the sequence's segments.
__global__ void __launch_bounds__(128) sel_join_kernel(SelCall c, Segments sg, bool backwards) {
    const int i = blockIdx.x, n = blockIdx.z, d = blockIdx.y * 128 + threadIdx.x, N = c.dstate;
    int lo, hi;
    if (!seq_rows(c.seq, i, lo, hi) || lo == hi) return;
    const int slot = !backwards && c.state ? slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error) : -1;
    if (d >= c.channels) return;
    const float A2 = c.A[(size_t)d * N + n] * LOG2E;
    float h = slot >= 0 && c.seq.has_init && c.seq.has_init[i] ? c.state[((size_t)slot * c.channels + d) * N + n] : 0.f;
    const int count = (hi - lo + sg.seg - 1) / sg.seg, s0 = lo / sg.seg + i;
    const size_t step = (size_t)N * c.channels;
    float *at = sg.state + (size_t)s0 * step + (size_t)n * c.channels + d;
    const float *steps = sg.steps + (size_t)s0 * c.channels + d;
    // the segment at the far end has neither an end state nor steps: nothing needs them
#pragma unroll 4
    for (int j = 0; j < count; ++j) {
        const int k = backwards ? count - 1 - j : j;
        const bool more = j + 1 < count;
        const float S = more ? at[k * step] : 0.f, w = more ? steps[(size_t)k * c.channels] : 0.f;
        at[k * step] = h;
        h = fmaf(ex2a(A2 * w), h, S);
    }
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

constexpr int FWD_WARPS_PER_SM = 16;

template <typename T> cudaError_t run_fwd(const SelCall &c, const Segments &sg, cudaStream_t st) {
    const dim3 grid(sg.slots, channel_tiles<FWD_THREADS>(c));
    const bool wide = wide_bc(c);
    return with_states(c.dstate, [&](auto np) {
        if (sg.seg != WHOLE) {
            sel_fwd_kernel<T, np(), false><<<grid, FWD_THREADS, 0, st>>>(c, sg, wide);
            cudaError_t e = cudaGetLastError();
            if (e == cudaSuccess) e = launch_sel_join(c, sg, false, st);
            if (e != cudaSuccess) return e;
        }
        sel_fwd_kernel<T, np(), true><<<grid, FWD_THREADS, 0, st>>>(c, sg, wide);
        return cudaGetLastError();
    });
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

cudaError_t launch_sel_join(const SelCall &c, const Segments &s, bool backwards, cudaStream_t st) {
    sel_join_kernel<<<dim3(c.seq.nseq, (c.channels + 127) / 128, c.dstate), 128, 0, st>>>(c, s, backwards);
    return cudaGetLastError();
}

size_t sel_fwd_workspace(int tokens, int nseq, int channels, int dstate) {
    const int seg = choose_seg(tokens, nseq, channels, FWD_WARPS_PER_SM);
    return seg == WHOLE ? 0 : (size_t)seg_slots(tokens, nseq, seg) * channels * (dstate + 1) * sizeof(float);
}

cudaError_t launch_sel_varlen(const SelCall &c, float *ws, cudaStream_t st) {
    Segments sg;
    sg.seg = choose_seg(c.seq.tokens, c.seq.nseq, c.channels, FWD_WARPS_PER_SM);
    sg.slots = seg_slots(c.seq.tokens, c.seq.nseq, sg.seg);
    sg.state = ws, sg.steps = ws + (sg.seg == WHOLE ? 0 : (size_t)sg.slots * c.dstate * c.channels);
    return c.bf16 ? run_fwd<__nv_bfloat16>(c, sg, st) : run_fwd<float>(c, sg, st);
}
cudaError_t launch_sel_update(const SelCall &c, int batch, cudaStream_t st) {
    return c.bf16 ? pick_update<__nv_bfloat16>(c, batch, st) : pick_update<float>(c, batch, st);
}

}  // namespace ssd
