// conv_varlen.cu -- the short causal depthwise convolution on packed sequences
// and on single tokens, and its gradient.
//
//   pre[t][c] = bias[c] + sum_{j<K} w[c][K-1-j] in[t-j][c],   out = silu(pre) or pre
//
// with t-j before the sequence's first row read from the slot's state (its last
// K-1 inputs) or zero.  Gradient, with dpre = dout silu'(pre):
//   din[t] = sum_j w[K-1-j] dpre[t+j]  (rows of the same sequence),
//   dw[K-1-j] = sum_t dpre[t] in[t-j],  dbias = sum_t dpre[t].
//
// Bound by HBM: each input read once, each output written once (K multiply-adds
// and one sigmoid per element).  A thread owns V neighbouring channels (16 bytes)
// and slides down a run of RUN tokens with the window in registers, so that no
// shared memory and no barrier is needed; the K-1 rows before a run are read
// again (an L2 hit).  Where a run meets sequence boundaries is worked out by the
// warp, one row per lane, as bit masks; four rows with no boundary among them
// take a straight path.
#include "mixer.cuh"

namespace ssd {
namespace {

constexpr int RUN = 32;    // tokens per warp
constexpr int WARPS = 4;   // runs per block

// Largest i in [0, n) with cu[i] <= t, or -1.  Ends after ceil(log2 n) steps
// whatever cu holds.
__device__ __forceinline__ int find_seq(const int *cu, int n, int t) {
    int lo = -1, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// A lane's row t: its sequence and the sequence's rows; false when no sequence holds it.
__device__ __forceinline__ bool row_seq(const Packed &p, int t, int &i, int &lo, int &hi) {
    i = -1, lo = hi = 0;
    if (t >= p.tokens) return false;
    i = find_seq(p.cu, p.nseq, t);
    if (i < 0) return false;
    lo = p.cu[i], hi = p.cu[i + 1];
    return lo >= 0 && t < hi && hi <= p.tokens;
}

// The bounds as a whole must not decrease or leave the tensor.
__device__ void check_bounds(const Packed &p) {
    for (int i = threadIdx.x; i < p.nseq; i += blockDim.x) {
        int lo, hi;
        seq_rows(p, i, lo, hi);
    }
}

template <typename T, int V> struct Dst {  // a thread's channels in the x, B or C output
    T *p;
    long long ld;
};
template <typename T, int V>
__device__ __forceinline__ Dst<T, V> out_of(T *xo, T *bo, T *co, int c, int cx, int cb) {
    if (c < cx) return {xo + c, cx};
    if (c < cx + cb) return {bo + (c - cx), cb};
    return {co + (c - cx - cb), cb};
}

// V channels (c .. c+V-1, in one output), KT taps of which the first KT - K are
// zero.  V > 1: rows and outputs are 16-byte aligned vectors.
template <typename T, int V, int KT>
__global__ void __launch_bounds__(32 * WARPS) conv_varlen_kernel(const T *__restrict__ in, long long ld,
                                                                const float *__restrict__ w,
                                                                const float *__restrict__ bias, T *__restrict__ xo,
                                                                T *__restrict__ bo, T *__restrict__ co,
                                                                T *__restrict__ state, int cx, int cb, int K, int silu,
                                                                Packed p) {
    constexpr bool WIDE = V > 1;
    const int ctot = cx + 2 * cb, lane = threadIdx.x & 31;
    const int c = (blockIdx.y * 32 + lane) * V;
    const bool mine = c < ctot;
    const int cc = mine ? c : 0;  // lanes past the channels follow along on channel 0, without storing
    if (blockIdx.x == 0 && blockIdx.y == 0) check_bounds(p);
    const int r0 = (blockIdx.x * WARPS + (threadIdx.x >> 5)) * RUN;
    if (r0 >= p.tokens) return;
    // one row per lane
    int seq, lo, hi;
    bool live = row_seq(p, r0 + lane, seq, lo, hi);
    const bool start = live && r0 + lane == lo;
    // the first K-1 rows of a sequence belong to the run that holds its first row
    if (live && lo < r0 && r0 + lane - lo < K - 1) live = false;
    const unsigned livem = __ballot_sync(0xffffffffu, live), startm = __ballot_sync(0xffffffffu, start);
    if (livem == 0) return;

    float wk[KT][V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < KT; ++k) wk[k][v] = k >= KT - K ? w[(size_t)(cc + v) * K + k - (KT - K)] : 0.f;
        b[v] = bias ? bias[cc + v] : 0.f;
    }
    const Dst<T, V> dst = out_of<T, V>(xo, bo, co, cc, cx, cb);
    const T *src = in + cc;
    float win[KT - 1][V];  // win[KT-1-j] = in[t-j]
#pragma unroll
    for (int k = 0; k < KT - 1; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) win[k][v] = 0.f;

    auto conv = [&](auto &&tap, int t) {  // tap(k): the input under w[k]
        float o[V];
        if constexpr (V > 1) {
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                float2 s = make_float2(b[v], b[v + 1]);
#pragma unroll
                for (int k = 0; k < KT; ++k)
                    s = fma2(make_float2(wk[k][v], wk[k][v + 1]), make_float2(tap(k)[v], tap(k)[v + 1]), s);
                o[v] = s.x, o[v + 1] = s.y;
            }
        } else {
            o[0] = b[0];
#pragma unroll
            for (int k = 0; k < KT; ++k) o[0] = fmaf(wk[k][0], tap(k)[0], o[0]);
        }
        if (silu)
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = silu_v(o[v]);
        if (mine) store_v<T, V, WIDE>(dst.p + t * dst.ld, o);
    };
    // The first row of a sequence: the window from its slot's state, and the state
    // after the sequence (known from its last rows) written back.
    auto enter = [&](int i, int first, int end) {
#pragma unroll
        for (int k = 0; k < KT - 1; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = 0.f;
        if (!state || K == 1) return;
        const int slot = slot_of(p.slots, p.nslots, i, p.dev_error);
        if (slot < 0 || !mine) return;
        T *st = state + ((size_t)slot * ctot + cc) * (K - 1);
        if (p.has_init && p.has_init[i]) {
#pragma unroll
            for (int k = 0; k < KT - 1; ++k)
                if (k >= KT - K)
#pragma unroll
                    for (int v = 0; v < V; ++v) win[k][v] = ld_f32<T>(st + v * (K - 1) + k - (KT - K));
        }
#pragma unroll
        for (int k = 0; k < KT - 1; ++k) {
            if (k < KT - K) continue;
            const int row = end - (KT - 1) + k;  // the last K-1 inputs, or what is left of the old ones
            float f[V];
            if (row >= first) {
                load_v<T, V, WIDE>(src + row * ld, f);
            } else {
                const int o = row - first + KT - 1;  // > k: entries not yet overwritten in registers
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    f[v] = 0.f;
#pragma unroll
                    for (int q = 0; q < KT - 1; ++q)
                        if (q == o) f[v] = win[q][v];
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) st_f32<T>(st + v * (K - 1) + k - (KT - K), f[v]);
        }
    };
    auto slide = [&](const float (&cur)[V]) {
#pragma unroll
        for (int k = 0; k < KT - 2; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
#pragma unroll
        for (int v = 0; v < V; ++v) win[KT - 2][v] = cur[v];
    };

    bool primed = false;  // the window holds the rows before the next one
    for (int r = 0; r < RUN; r += 4) {
        const unsigned lv = (livem >> r) & 15u, sm = (startm >> r) & 15u;
        if (lv == 0) {
            primed = false;
            continue;
        }
        const int t0 = r0 + r;
        float x[4][V];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (t0 + q < p.tokens) load_v<T, V, WIDE>(src + (t0 + q) * ld, x[q]);
        if (lv == 15u && sm == 0u && primed) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                conv([&](int k) -> const float(&)[V] { return q + k < KT - 1 ? win[q + k < KT - 1 ? q + k : 0] : x[q + k >= KT - 1 ? q + k - (KT - 1) : 0]; }, t0 + q);
            // rows t0+4-(KT-1) .. t0+3
#pragma unroll
            for (int k = 0; k < KT - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = k + 4 < KT - 1 ? win[k + 4 < KT - 1 ? k + 4 : 0][v] : x[k + 4 >= KT - 1 ? k + 4 - (KT - 1) : 0][v];
            continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (!((lv >> q) & 1u)) {
                primed = false;
                continue;
            }
            const int t = t0 + q, at = r + q;
            if ((sm >> q) & 1u) {
                enter(__shfl_sync(0xffffffffu, seq, at), t, __shfl_sync(0xffffffffu, hi, at));
            } else if (!primed) {  // at least K-1 rows of the sequence lie before t
#pragma unroll
                for (int k = 0; k < KT - 1; ++k)
                    if (k >= KT - K && t - (KT - 1) + k >= 0) load_v<T, V, WIDE>(src + (t - (KT - 1) + k) * ld, win[k]);
            }
            primed = true;
            conv([&](int k) -> const float(&)[V] { return k < KT - 1 ? win[k < KT - 1 ? k : 0] : x[q]; }, t);
            slide(x[q]);
        }
    }
    // first rows, past the run, of a sequence that started in its last K-2 rows
    const int lo31 = __shfl_sync(0xffffffffu, lo, 31), hi31 = __shfl_sync(0xffffffffu, hi, 31);
    if ((livem >> 31) && lo31 >= r0)
        for (int t = r0 + RUN; t < min(hi31, lo31 + K - 1); ++t) {
            float x[V];
            load_v<T, V, WIDE>(src + t * ld, x);
            conv([&](int k) -> const float(&)[V] { return k < KT - 1 ? win[k < KT - 1 ? k : 0] : x; }, t);
            slide(x);
        }
}

// One token per sequence: a thread per channel.  A few bytes per channel: bound by
// latency, and at large batches by HBM.
template <typename T>
__global__ void __launch_bounds__(128) conv_update_kernel(const T *__restrict__ in, long long ld,
                                                         const float *__restrict__ w, const float *__restrict__ bias,
                                                         T *__restrict__ xo, T *__restrict__ bo, T *__restrict__ co,
                                                         T *__restrict__ state, int cx, int cb, int K, int silu,
                                                         Packed p) {
    const int ctot = cx + 2 * cb, c = blockIdx.x * 128 + threadIdx.x, i = blockIdx.y;
    const int slot = slot_of(p.slots, p.nslots, i, p.dev_error);
    if (slot < 0 || c >= ctot) return;
    T *st = state + ((size_t)slot * ctot + c) * (K - 1);
    const T xv = in[i * ld + c];
    float acc = bias ? bias[c] : 0.f;
    acc = fmaf(w[(size_t)c * K + K - 1], ld_f32<T>(&xv), acc);
    for (int k = 0; k < K - 1; ++k) {
        const T old = st[k];
        acc = fmaf(w[(size_t)c * K + k], ld_f32<T>(&old), acc);
        if (k > 0) st[k - 1] = old;
    }
    if (K > 1) st[K - 2] = xv;
    const Dst<T, 1> dst = out_of<T, 1>(xo, bo, co, c, cx, cb);
    st_f32<T>(dst.p + i * dst.ld, silu ? silu_v(acc) : acc);
}

// Gradient.  A warp walks its run from the last row to the first with the inputs
// in[t .. t-K+1] and the later rows' dpre in registers; the K-1 rows after the run
// are computed again for their dpre.  dw and dbias are summed per thread over the
// run, over the block's runs in shared memory and then, by conv_bwd_sum, over
// blocks in a fixed order.
template <typename T, int V, int KT>
__global__ void __launch_bounds__(32 * WARPS) conv_bwd_kernel(const T *__restrict__ in, long long ld,
                                                             const float *__restrict__ w,
                                                             const float *__restrict__ bias, const T *__restrict__ dxo,
                                                             const T *__restrict__ dbo, const T *__restrict__ dco,
                                                             T *__restrict__ dx, float *__restrict__ part, int cx,
                                                             int cb, int K, int silu, Packed p) {
    constexpr bool WIDE = V > 1;
    __shared__ float red[WARPS - 1][32][(KT + 1) * V + 1];
    const int ctot = cx + 2 * cb, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * V;
    const bool mine = c < ctot;
    const int cc = mine ? c : 0;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_bounds(p);
    const int r0 = (blockIdx.x * WARPS + wid) * RUN;
    float wk[KT][V], b[V], dw[KT][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            wk[k][v] = k >= KT - K ? w[(size_t)(cc + v) * K + k - (KT - K)] : 0.f;
            dw[k][v] = 0.f;
        }
        b[v] = bias ? bias[cc + v] : 0.f;
        db[v] = 0.f;
    }
    const Dst<const T, V> src = out_of<const T, V>(dxo, dbo, dco, cc, cx, cb);
    int seq, lo, hi;
    const bool live = row_seq(p, r0 + lane, seq, lo, hi);
    const unsigned livem = __ballot_sync(0xffffffffu, live);
    float xw[KT][V], dp[KT][V];  // xw[j] = in[t-j], dp[j] = dpre[t+j]
    // dpre of row t of a sequence with first row `first` into dp[0]; the taps before
    // `first` read as zero
    auto dpre_of = [&](int t, int first, bool primed) {
        if (primed) {
#pragma unroll
            for (int j = 0; j < KT - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) xw[j][v] = xw[j + 1][v];
        }
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            if (primed && j != K - 1) continue;  // the one row that is new (taps past K-1 stay zero)
            if (j < K && t - j >= first) {
                load_v<T, V, WIDE>(in + cc + (t - j) * ld, xw[j]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) xw[j][v] = 0.f;
            }
        }
        float d[V];
        load_v<T, V, WIDE>(src.p + t * src.ld, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (silu) {
                float s = b[v];
#pragma unroll
                for (int j = 0; j < KT; ++j) s = fmaf(wk[KT - 1 - j][v], xw[j][v], s);
                const float g = sigmoid_f(s);
                d[v] *= g * fmaf(s, 1.f - g, 1.f);
            }
            dp[0][v] = d[v];
        }
    };
    auto later = [&] {  // one row up: dp[j] becomes dpre[(t-1)+j]
#pragma unroll
        for (int j = KT - 1; j > 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) dp[j][v] = dp[j - 1][v];
    };
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) dp[j][v] = 0.f;
    };
    clear();
    bool primed = false;
    const int lo31 = __shfl_sync(0xffffffffu, lo, 31), hi31 = __shfl_sync(0xffffffffu, hi, 31);
    if (livem >> 31)
        for (int t = min(hi31, r0 + RUN + K - 1) - 1; t >= r0 + RUN; --t) {
            dpre_of(t, lo31, primed);
            later();
            primed = true;
        }
    for (int r = RUN - 1; r >= 0; --r) {
        const int t = r0 + r;
        float o[V];
        if ((livem >> r) & 1u) {
            const int first = __shfl_sync(0xffffffffu, lo, r), end = __shfl_sync(0xffffffffu, hi, r);
            if (t == end - 1) clear(), primed = false;  // nothing of this sequence lies later
            dpre_of(t, first, primed);
            primed = true;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    s = fmaf(wk[KT - 1 - j][v], dp[j][v], s);
                    dw[KT - 1 - j][v] = fmaf(dp[0][v], xw[j][v], dw[KT - 1 - j][v]);
                }
                db[v] += dp[0][v];
                o[v] = s;
            }
            later();
        } else {  // rows of no sequence have no gradient
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = 0.f;
        }
        if (mine && t < p.tokens) store_v<T, V, WIDE>(dx + (size_t)t * ctot + cc, o);
    }
    if (wid > 0)
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < KT; ++k) red[wid - 1][lane][v * (KT + 1) + k] = dw[k][v];
            red[wid - 1][lane][v * (KT + 1) + KT] = db[v];
        }
    __syncthreads();
    if (wid == 0 && mine)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float *o = part + ((size_t)blockIdx.x * ctot + cc + v) * (K + 1);
#pragma unroll
            for (int k = 0; k <= KT; ++k) {
                float s = k < KT ? dw[k < KT ? k : 0][v] : db[v];
#pragma unroll
                for (int q = 0; q < WARPS - 1; ++q) s += red[q][lane][v * (KT + 1) + k];
                if (k == KT)
                    o[K] = s;
                else if (k >= KT - K)
                    o[k - (KT - K)] = s;
            }
        }
}

// dw[c][k] and dbias[c] from the blocks' parts [parts][channels][K+1]: 32 lanes
// take every 32nd part, then a butterfly.
__global__ void __launch_bounds__(256) conv_bwd_sum(const float *__restrict__ part, int parts, int channels, int K,
                                                   float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float s[8][33];
    const int o = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5, n = channels * (K + 1);
    float a = 0.f;
    if (o < n)
        for (int i = q; i < parts; i += 8) a += part[(size_t)i * n + o];
    s[q][threadIdx.x & 31] = a;
    __syncthreads();
    if (q || o >= n) return;
    for (int i = 1; i < 8; ++i) a += s[i][threadIdx.x];
    const int c = o / (K + 1), k = o % (K + 1);
    if (k < K)
        dw[(size_t)c * K + k] = a;
    else if (db)
        db[c] = a;
}

// Whether rows of V channels can be read and written as V * sizeof(T) byte vectors.
bool wide_rows(const ConvCall &c, int V) {
    const size_t e = c.bf16 ? 2 : 4;
    return c.cx % V == 0 && c.cb % V == 0 && rows_aligned(c.in, c.ld, e, V * e);
}

template <typename T, int V, int KT> cudaError_t run_fwd(const ConvCall &c, cudaStream_t st) {
    const int ctot = c.cx + 2 * c.cb;
    const dim3 grid((c.seq.tokens + RUN * WARPS - 1) / (RUN * WARPS), (ctot + 32 * V - 1) / (32 * V));
    conv_varlen_kernel<T, V, KT><<<grid, 32 * WARPS, 0, st>>>(
        static_cast<const T *>(c.in), c.ld, c.w, c.bias, static_cast<T *>(c.xo), static_cast<T *>(c.bo),
        static_cast<T *>(c.co), static_cast<T *>(c.state), c.cx, c.cb, c.width, c.silu, c.seq);
    return cudaGetLastError();
}
template <typename T, int V> cudaError_t pick_fwd(const ConvCall &c, cudaStream_t st) {
    if (c.width > 4) return run_fwd<T, 1, 8>(c, st);
    return wide_rows(c, V) ? run_fwd<T, V, 4>(c, st) : run_fwd<T, 1, 4>(c, st);
}

template <typename T, int V, int KT> cudaError_t run_bwd(const ConvCall &c, float *ws, cudaStream_t st) {
    const int ctot = c.cx + 2 * c.cb, parts = (c.seq.tokens + RUN * WARPS - 1) / (RUN * WARPS);
    if (parts > 0) {
        const dim3 grid(parts, (ctot + 32 * V - 1) / (32 * V));
        conv_bwd_kernel<T, V, KT><<<grid, 32 * WARPS, 0, st>>>(
            static_cast<const T *>(c.in), c.ld, c.w, c.bias, static_cast<const T *>(c.xo),
            static_cast<const T *>(c.bo), static_cast<const T *>(c.co), static_cast<T *>(c.dx), ws, c.cx, c.cb,
            c.width, c.silu, c.seq);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    conv_bwd_sum<<<(ctot * (c.width + 1) + 31) / 32, 256, 0, st>>>(ws, parts, ctot, c.width, c.dw, c.db);
    return cudaGetLastError();
}
template <typename T, int V> cudaError_t pick_bwd(const ConvCall &c, float *ws, cudaStream_t st) {
    if (c.width > 4) return run_bwd<T, 1, 8>(c, ws, st);
    return wide_rows(c, V) ? run_bwd<T, V, 4>(c, ws, st) : run_bwd<T, 1, 4>(c, ws, st);
}

}  // namespace

cudaError_t launch_conv_varlen(const ConvCall &c, cudaStream_t st) {
    return c.bf16 ? pick_fwd<__nv_bfloat16, 8>(c, st) : pick_fwd<float, 4>(c, st);
}

cudaError_t launch_conv_update(const ConvCall &c, int batch, cudaStream_t st) {
    const dim3 grid((c.cx + 2 * c.cb + 127) / 128, batch);
    if (c.bf16) {
        using T = __nv_bfloat16;
        conv_update_kernel<T><<<grid, 128, 0, st>>>(static_cast<const T *>(c.in), c.ld, c.w, c.bias,
                                                    static_cast<T *>(c.xo), static_cast<T *>(c.bo),
                                                    static_cast<T *>(c.co), static_cast<T *>(c.state), c.cx, c.cb,
                                                    c.width, c.silu, c.seq);
    } else {
        conv_update_kernel<float><<<grid, 128, 0, st>>>(static_cast<const float *>(c.in), c.ld, c.w, c.bias,
                                                        static_cast<float *>(c.xo), static_cast<float *>(c.bo),
                                                        static_cast<float *>(c.co), static_cast<float *>(c.state), c.cx,
                                                        c.cb, c.width, c.silu, c.seq);
    }
    return cudaGetLastError();
}

size_t conv_bwd_workspace(int tokens, int channels, int width) {
    return (size_t)((tokens + RUN * WARPS - 1) / (RUN * WARPS)) * channels * (width + 1) * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvCall &c, float *ws, cudaStream_t st) {
    return c.bf16 ? pick_bwd<__nv_bfloat16, 4>(c, ws, st) : pick_bwd<float, 4>(c, ws, st);
}

}  // namespace ssd
