// selscan.cu -- the Mamba-1 selective scan on packed sequences and on single tokens.
//
//   delta_t = softplus(dt_t + bias) (or dt_t + bias),
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)          per channel.
//
// A thread per channel and 8 states, along a sequence or a segment of one
// (selscan_seg.cuh): per state and token three packed operations to two states and an
// exponential.  x, dt, z and y go straight between global memory and
// registers (neighbouring lanes, neighbouring channels), eight tokens ahead; B and C,
// which a block's channels share, through shared memory.  Bound by the exponential
// unit (N + 4 operations per channel and token at 16 per SM and clock), then by issue.
// Measured at 64 x 512 tokens, 1024 channels, 16 states, bf16, states kept: 258 us, 2.1 TB/s
// and 58 % of the exponential unit.  A form that split the tokens of a chunk over the lanes
// of a warp (one exponential per state and token at any length, but scans over lanes and a
// second walk) took 352 us, all states in one thread 318 us, two channels to a packed
// operation 290 us.
#include "selscan_seg.cuh"

namespace ssd {
namespace {

constexpr int AHEAD = 8;  // tokens at a time, and fetched ahead
constexpr int FWD_BLOCKS_PER_SM = 4;

template <int NP> struct FwdLanes {
    static constexpr int NS = NP < 8 ? NP : 8, P = NS / 2, SPLIT = NP / NS, CHANS = 32 / SPLIT, OWN = AHEAD / SPLIT;
    static constexpr int CH = SCAN_THREADS / SPLIT;  // channels of a block
    static constexpr int TT = NP <= 16 ? 32 : 16;    // tokens of B and C at a time
};

// v[k] summed over the SPLIT lanes of a channel: a lane of part s ends with token
// j SPLIT + s in v[j].
template <int SPLIT, int K> __device__ __forceinline__ void sum_lanes(float (&v)[K], int part) {
    constexpr int CHANS = 32 / SPLIT;
#pragma unroll
    for (int j = 0; j < K / SPLIT; ++j) {
        float t[SPLIT];
#pragma unroll
        for (int u = 0; u < SPLIT; ++u) t[u] = v[j * SPLIT + u];
#pragma unroll
        for (int n = SPLIT / 2; n > 0; n /= 2)
#pragma unroll
            for (int u = 0; u < n; ++u)
                t[u] = (part & n ? t[u + n] : t[u]) + __shfl_xor_sync(0xffffffffu, part & n ? t[u] : t[u + n], n * CHANS);
        v[j] = t[0];
    }
}

// FULL: y, kept states and the end state; else only what sel_join needs.
template <typename T, int NP, bool FULL>
__global__ void __launch_bounds__(SCAN_THREADS, FWD_BLOCKS_PER_SM) sel_fwd_kernel(SelCall c, Segments sg, bool wide) {
    using L = FwdLanes<NP>;
    constexpr int P = L::P, SPLIT = L::SPLIT, CHANS = L::CHANS, OWN = L::OWN, TT = L::TT;
    using Stage = StageBC<T, NP, TT, false>;
    __shared__ __align__(16) float4 bc[2][TT * NP / 2];
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end)) return;  // the same for the whole block
    if (!FULL && hi == end) return;  // nothing follows
    const int N = c.dstate, lane = threadIdx.x & 31, part = lane / CHANS, n0 = part * L::NS;
    const int per_group = c.channels / c.groups, tiles = (per_group + L::CH - 1) / L::CH, group = blockIdx.y / tiles;
    const int at = blockIdx.y % tiles * L::CH + (threadIdx.x >> 5) * CHANS + lane % CHANS;
    const bool mine = at < per_group;
    const int d = group * per_group + min(at, per_group - 1);  // threads past the group follow along on its last channel
    const T *B = static_cast<const T *>(c.B) + group * N + lo * c.ld_b, *C = static_cast<const T *>(c.C) + group * N + lo * c.ld_c;
    Stage stage;
    stage.load(B, c.ld_b, C, c.ld_c, min(TT, hi - lo), N, wide);
    // the lane's next tokens: part, part + SPLIT, ..
    int row = lo + part;
    const T *px = static_cast<const T *>(c.x) + row * c.ld_x + d, *pd = static_cast<const T *>(c.dt) + row * c.ld_dt + d;
    const T *pz = static_cast<const T *>(c.z) + (c.z ? row * c.ld_z + d : 0);
    T *py = static_cast<T *>(c.y) + (size_t)row * c.channels + d;
    T nx[OWN], nd[OWN], nz[OWN];
    auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (row < hi) {
                nx[j] = *px, nd[j] = *pd;
                if (FULL && c.z) nz[j] = *pz;
            }
            row += SPLIT, px += SPLIT * c.ld_x, pd += SPLIT * c.ld_dt;
            if (FULL) pz += SPLIT * c.ld_z;
        }
    };
    fetch();
    const int slot = FULL && c.state ? slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error) : -1;
    float *const state = c.state + (slot >= 0 ? ((size_t)slot * c.channels + d) * N : 0);
    const bool init = slot >= 0 && c.seq.has_init && c.seq.has_init[i] && sg.seg == WHOLE;
    float *const carried = sg.state + (size_t)blockIdx.x * N * c.channels + d;  // [state][channel]
    auto load_h = [&](int n) {
        if (n >= N) return 0.f;
        if (FULL && sg.seg != WHOLE) return carried[(size_t)n * c.channels];
        return init ? state[n] : 0.f;
    };
    auto load_A = [&](int n) { return n < N ? rate(c.A[(size_t)d * N + n]) : 0.f; };
    float2 A2[P], h[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        A2[p] = make_float2(load_A(n0 + 2 * p), load_A(n0 + 2 * p + 1));
        h[p] = make_float2(load_h(n0 + 2 * p), load_h(n0 + 2 * p + 1));
    }
    const float bias = c.dt_bias ? c.dt_bias[d] : 0.f, D = c.D ? c.D[d] : 0.f;
    float steps = 0.f;
    float *kept = nullptr;
    if (FULL && c.chunk_states)
        kept = c.chunk_states + ((size_t)(first / SEL_CHUNK + i + (lo - first) / SEL_CHUNK) * N + n0) * c.channels + d;
    stage.put(bc[0]);
    for (int t0 = lo, buf = 0; t0 < hi; t0 += TT, buf ^= 1) {
        const int nt = min(TT, hi - t0);
        B += TT * c.ld_b, C += TT * c.ld_c;
        if (t0 + TT < hi) stage.load(B, c.ld_b, C, c.ld_c, min(TT, hi - t0 - TT), N, wide);
        __syncthreads();  // bc[buf] is written, and nobody reads bc[buf ^ 1] any more
#pragma unroll 1
        for (int t = 0; t < nt; t += AHEAD) {
            // the lane's tokens; one past the end is a step of nothing
            float dl[OWN], u[OWN], xv[OWN], gate[OWN];
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const bool in = t + j * SPLIT + part < nt;
                xv[j] = ld_f32<T>(&nx[j]);
                dl[j] = ld_f32<T>(&nd[j]) + bias;
                if (c.softplus) dl[j] = softplus_f(dl[j]);
                if (FULL && c.z) gate[j] = silu_v(ld_f32<T>(&nz[j]));
                u[j] = in ? dl[j] * xv[j] : 0.f, dl[j] = in ? dl[j] : 0.f;
                if (!FULL) steps += dl[j];
            }
            fetch();
            if (FULL && kept) {
                static_assert(SEL_CHUNK == AHEAD, "a state is kept before every step of this loop");
                if (mine)
#pragma unroll
                    for (int k = 0; k < L::NS; ++k)
                        if (n0 + k < N) kept[(size_t)k * c.channels] = k & 1 ? h[k / 2].y : h[k / 2].x;
                kept += (size_t)N * c.channels;
            }
            float y[AHEAD];
            const float4 *q = bc[buf] + (t * NP + n0) / 2;
            auto token = [&](int k) {
                const float ds = SPLIT == 1 ? dl[k / SPLIT] : __shfl_sync(0xffffffffu, dl[k / SPLIT], lane % CHANS + k % SPLIT * CHANS);
                const float us = SPLIT == 1 ? u[k / SPLIT] : __shfl_sync(0xffffffffu, u[k / SPLIT], lane % CHANS + k % SPLIT * CHANS);
                float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float4 v = q[k * (NP / 2) + p];
                    const float2 arg = mul2(splat(ds), A2[p]);
                    h[p] = fma2(make_float2(ex2a(arg.x), ex2a(arg.y)), h[p], mul2(splat(us), make_float2(v.x, v.y)));
                    if (FULL) y2 = fma2(make_float2(v.z, v.w), h[p], y2);
                }
                y[k] = y2.x + y2.y;
            };
#pragma unroll
            for (int k = 0; k < AHEAD / 2; ++k) token(k);
            if (t + AHEAD / 2 < nt) {
#pragma unroll
                for (int k = AHEAD / 2; k < AHEAD; ++k) token(k);
            } else {
#pragma unroll
                for (int k = AHEAD / 2; k < AHEAD; ++k) y[k] = 0.f;
            }
            if (FULL) {
                sum_lanes<SPLIT>(y, part);
#pragma unroll
                for (int j = 0; j < OWN; ++j) {
                    float o = fmaf(D, xv[j], y[j]);
                    if (c.z) o *= gate[j];
                    if (mine && t + j * SPLIT + part < nt) st_f32<T>(py, o);
                    py += (size_t)SPLIT * c.channels;
                }
            }
        }
        if (t0 + TT < hi) stage.put(bc[buf ^ 1]);
    }
    if (FULL) {
        if (slot >= 0 && hi == end && mine)
#pragma unroll
            for (int k = 0; k < L::NS; ++k)
                if (n0 + k < N) state[n0 + k] = k & 1 ? h[k / 2].y : h[k / 2].x;
    } else {
        if (mine)
#pragma unroll
            for (int k = 0; k < L::NS; ++k)
                if (n0 + k < N) carried[(size_t)(n0 + k) * c.channels] = k & 1 ? h[k / 2].y : h[k / 2].x;
#pragma unroll
        for (int o = CHANS; o < 32; o *= 2) steps += __shfl_xor_sync(0xffffffffu, steps, o);
        if (mine && part == 0) sg.steps[(size_t)blockIdx.x * c.channels + d] = steps;
    }
}

// 2^x h + S for a whole segment's x.  The factor alone may leave float32 where the product
// does not (a state that grew, or grows), so it goes in as two that do not: past 2^254 every
// normal float32 overflows, and past 2^-252 the second factor is zero.  From -126 to 127 the
// first is all of it.
__device__ __forceinline__ float carry(float x, float h, float S) {
    const float part = fminf(fmaxf(x, -126.f), 127.f);
    return fmaf(ex2a(part), ex2a(fminf(x - part, 127.f)) * h, S);
}

// A thread per (sequence, state, channel) goes through the sequence's segments.
__global__ void __launch_bounds__(128) sel_join_kernel(SelCall c, Segments sg, bool backwards) {
    const int i = blockIdx.x, n = blockIdx.z, d = blockIdx.y * 128 + threadIdx.x, N = c.dstate;
    int lo, hi;
    if (!seq_rows(c.seq, i, lo, hi) || lo == hi) return;
    const int slot = !backwards && c.state ? slot_of(c.seq.slots, c.seq.nslots, i, c.seq.dev_error) : -1;
    if (d >= c.channels) return;
    const float A2 = rate(c.A[(size_t)d * N + n]);
    float h = slot >= 0 && c.seq.has_init && c.seq.has_init[i] ? c.state[((size_t)slot * c.channels + d) * N + n] : 0.f;
    const int count = (hi - lo + sg.seg - 1) / sg.seg, s0 = lo / sg.seg + i;
    const size_t step = (size_t)N * c.channels;
    float *at = sg.state + (size_t)s0 * step + (size_t)n * c.channels + d;
    const float *steps = sg.steps + (size_t)s0 * c.channels + d;
    // the segment at the far end has neither an end state nor steps: nothing needs them
    constexpr int BATCH = 8;  // loads in flight
    for (int j0 = 0; j0 < count; j0 += BATCH) {
        float S[BATCH], w[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int j = j0 + u, k = backwards ? count - 1 - j : j;
            const bool more = j + 1 < count;
            S[u] = more ? at[k * step] : 0.f, w[u] = more ? steps[(size_t)k * c.channels] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int j = j0 + u, k = backwards ? count - 1 - j : j;
            if (j < count) at[k * step] = h;
            h = carry(A2 * w[u], h, S[u]);
        }
    }
}

// One token per sequence, in place on the state.  A warp takes 32 channels.  Each lane
// does the scalar work (step size, gate) of one; for the states, the LP lanes of a
// group go through their LP channels together, four states a lane (dstate = 4 LP), so
// that a group reads and writes whole rows of the state, all loads first, and a lane
// ends with its own channel's readout.  (LP lanes doing the scalar work of each of
// their channels together measured 43.6 us against 27.5 us for 256 x 4096 channels
// of 16 states: five times the instructions; 64 registers, so that eight blocks are on an
// SM, 26.1 us, 48 31.7 us.)  LP = 0: any dstate, a lane per channel.
// As in the scan, a step of nothing is a decay of one, also where A is -infinity: A is kept
// from -1e38 on, where a step above 1e-36 leaves nothing.
// SAME: the warp's channels lie in one B/C group.  Bound by HBM: the state in and out
// (26.1 us is 5.5 TB/s of the bytes that have to move).
constexpr int UPD_THREADS = 128;
__device__ __forceinline__ float finite_rate(float A) { return A < -1e38f ? -1e38f : A; }
__device__ __forceinline__ float4 finite_rates(float4 a) {
    return make_float4(finite_rate(a.x), finite_rate(a.y), finite_rate(a.z), finite_rate(a.w));
}
template <typename T, int LP, bool SAME>
__global__ void __launch_bounds__(UPD_THREADS, LP > 4 ? 1 : 8) sel_update_kernel(SelCall c, bool wide_bc) {
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
        for (int u = 0; u < L; ++u) a[u] = finite_rates(__ldg(reinterpret_cast<const float4 *>(c.A + (size_t)min(d0 + u, last) * N) + q));
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
            if (LP > 4) a[u] = finite_rates(__ldg(reinterpret_cast<const float4 *>(c.A + (size_t)du_ * N) + q));
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
            *hn = fmaf(ex2a(d2 * finite_rate(c.A[(size_t)d * N + n])), *hn, du * ld_f32<T>(B + g * N + n));
            y = fmaf(ld_f32<T>(C + g * N + n), *hn, y);
        }
    }
    if (d <= last) {
        y = fmaf(Dv, xv, y);
        if (c.z) y *= silu_v(zv);
        st_f32<T>(static_cast<T *>(c.y) + (size_t)i * c.channels + d, y);
    }
}

constexpr int FWD_WARPS_PER_SM = 32;
inline int fwd_seg(int tokens, int nseq, int channels, int N) {
    return choose_seg(tokens, nseq, channels, N <= 8 ? 32 : N <= 16 ? 16 : N <= 32 ? 8 : 4, FWD_WARPS_PER_SM);  // as FwdLanes
}

template <typename T, int NP, bool FULL> cudaError_t run_pass(const SelCall &c, const Segments &sg, cudaStream_t st) {
    constexpr int CH = FwdLanes<NP>::CH;
    const dim3 grid(sg.slots, c.groups * ((c.channels / c.groups + CH - 1) / CH));
    sel_fwd_kernel<T, NP, FULL><<<grid, SCAN_THREADS, 0, st>>>(c, sg, Access(c).bc);
    return cudaGetLastError();
}
template <typename T> cudaError_t run_fwd(const SelCall &c, const Segments &sg, cudaStream_t st) {
    return with_states(c.dstate, [&](auto np) {
        if (sg.seg != WHOLE) {
            cudaError_t e = run_pass<T, np(), false>(c, sg, st);
            if (e == cudaSuccess) e = launch_sel_join(c, sg, false, st);
            if (e != cudaSuccess) return e;
        }
        return run_pass<T, np(), true>(c, sg, st);
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
    const int seg = fwd_seg(tokens, nseq, channels, dstate);
    return seg == WHOLE ? 0 : (size_t)seg_slots(tokens, nseq, seg) * channels * (dstate + 1) * sizeof(float);
}

cudaError_t launch_sel_varlen(const SelCall &c, float *ws, cudaStream_t st) {
    Segments sg;
    sg.seg = fwd_seg(c.seq.tokens, c.seq.nseq, c.channels, c.dstate);
    sg.slots = seg_slots(c.seq.tokens, c.seq.nseq, sg.seg);
    sg.state = ws, sg.steps = ws + (sg.seg == WHOLE ? 0 : (size_t)sg.slots * c.dstate * c.channels);
    return c.bf16 ? run_fwd<__nv_bfloat16>(c, sg, st) : run_fwd<float>(c, sg, st);
}
cudaError_t launch_sel_update(const SelCall &c, int batch, cudaStream_t st) {
    return c.bf16 ? pick_update<__nv_bfloat16>(c, batch, st) : pick_update<float>(c, batch, st);
}

}  // namespace ssd
