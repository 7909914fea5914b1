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
#include <type_traits>

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

// A run's next BATCH rows, fetched ahead as they lie in memory.  (All 35 rows copied
// into shared memory at once instead measured 44.5 us for 9408 x 4352 bf16 where this
// form took 39.8 us, 34 us since: the rows were not late, and 16 KB more per block cost
// occupancy.)
template <typename T, int V> struct Ahead {
    static constexpr int BATCH = sizeof(T) * V == 16 ? 4 : 8;
    using Vec = typename std::conditional<V == 1, T, typename std::conditional<sizeof(T) * V == 16, uint4, uint2>::type>::type;
    Vec cur[BATCH], nxt[BATCH];
    __device__ __forceinline__ void load(const T *src, long long ld, int t, int tokens) {
        const T *row = src + t * ld;
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            nxt[q] = *reinterpret_cast<const Vec *>(row);
            if (t + q < tokens - 1) row += ld;  // past the end the last row again
        }
    }
    __device__ __forceinline__ void next(const T *src, long long ld, int t, int tokens, bool more) {
#pragma unroll
        for (int q = 0; q < BATCH; ++q) cur[q] = nxt[q];
        if (more) load(src, ld, t, tokens);
    }
    __device__ __forceinline__ void get(int q, float (&f)[V]) { load_v<T, V, (V > 1)>(reinterpret_cast<const T *>(&cur[q]), f); }
};

// V channels (c .. c+V-1, in one output), KT taps of which the first KT - K are not
// there (EXACT: K == KT).  V > 1: rows and outputs are aligned vectors.
template <typename T, int V, int KT, bool EXACT>
__global__ void __launch_bounds__(32 * WARPS, V > 1 ? 5 : 8) conv_varlen_kernel(const T *__restrict__ in, long long ld,
                                                                const float *__restrict__ w,
                                                                const float *__restrict__ bias, T *__restrict__ xo,
                                                                T *__restrict__ bo, T *__restrict__ co,
                                                                T *__restrict__ state, int cx, int cb, int K, int silu,
                                                                Packed p) {
    constexpr bool WIDE = V > 1;
    constexpr int BATCH = Ahead<T, V>::BATCH;
    const int ctot = cx + 2 * cb, lane = threadIdx.x & 31;
    const int tiles = (ctot + 32 * V - 1) / (32 * V), rows_at = blockIdx.x / tiles;  // a block's neighbours share its rows
    const int c = ((blockIdx.x % tiles) * 32 + lane) * V;
    const bool mine = c < ctot;
    const int cc = mine ? c : 0;  // lanes past the channels follow along on channel 0, without storing
    if (blockIdx.x == 0) check_bounds(p);
    const int r0 = (rows_at * WARPS + (threadIdx.x >> 5)) * RUN;
    if (r0 >= p.tokens) return;
    const T *src = in + cc;
    Ahead<T, V> rows;
    rows.load(src, ld, r0, p.tokens);  // on their way while the boundaries are looked up
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
        if (KT == 4 && EXACT) {  // whole 16-byte rows of weights
            const float4 q = *reinterpret_cast<const float4 *>(w + (size_t)(cc + v) * 4);
            wk[0][v] = q.x, wk[1][v] = q.y, wk[2][v] = q.z, wk[3][v] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < KT; ++k) wk[k][v] = k >= KT - K ? w[(size_t)(cc + v) * K + k - (KT - K)] : 0.f;
        }
        b[v] = bias ? bias[cc + v] : 0.f;
    }
    const Dst<T, V> dst = out_of<T, V>(xo, bo, co, cc, cx, cb);
    float win[KT - 1][V];  // win[KT-1-j] = in[t-j]
#pragma unroll
    for (int k = 0; k < KT - 1; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) win[k][v] = 0.f;

    auto conv = [&](auto &&tap, T *to) {  // tap(k): the input under w[k]
        float o[V];
        if constexpr (V > 1) {
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                float2 s = make_float2(b[v], b[v + 1]);
#pragma unroll
                for (int k = 0; k < KT; ++k)
                    if (EXACT || k >= KT - K)  // a missing tap does not see its input (which may be infinite)
                        s = fma2(make_float2(wk[k][v], wk[k][v + 1]), make_float2(tap(k)[v], tap(k)[v + 1]), s);
                if (silu) s = silu2(s);
                o[v] = s.x, o[v + 1] = s.y;
            }
        } else {
            o[0] = b[0];
#pragma unroll
            for (int k = 0; k < KT; ++k)
                if (EXACT || k >= KT - K) o[0] = fmaf(wk[k][0], tap(k)[0], o[0]);
            if (silu) o[0] = silu_v(o[0]);
        }
        if (mine) store_v<T, V, WIDE>(to, o);
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

    auto prime = [&](int t) {  // at least K-1 rows of the sequence lie before t
#pragma unroll
        for (int k = 0; k < KT - 1; ++k)
            if (k >= KT - K && t - (KT - 1) + k >= 0) load_v<T, V, WIDE>(src + (t - (KT - 1) + k) * ld, win[k]);
    };
    bool primed = (livem & 1u) && !(startm & 1u);  // the window holds the rows before the next one
    if (primed) prime(r0);
#pragma unroll 1
    for (int r = 0; r < RUN; r += BATCH) {
        constexpr unsigned ALL = (1u << BATCH) - 1;
        const unsigned lv = (livem >> r) & ALL, sm = (startm >> r) & ALL;
        const int t0 = r0 + r;
        rows.next(src, ld, t0 + BATCH, p.tokens, r + BATCH < RUN && t0 + BATCH < p.tokens);
        if (lv == ALL && sm == 0u && primed) {
            float x[BATCH][V];  // each row is unpacked once; the window is the rows before
            T *to = dst.p + t0 * dst.ld;
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                rows.get(q, x[q]);
                conv([&](int k) -> const float(&)[V] {
                    return q + k < KT - 1 ? win[q + k < KT - 1 ? q + k : 0] : x[q + k >= KT - 1 ? q + k - (KT - 1) : 0];
                }, to);
                to += dst.ld;
            }
#pragma unroll
            for (int k = 0; k < KT - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = x[BATCH - (KT - 1) + k][v];
            continue;
        }
#pragma unroll 1  // boundaries are rare: a short loop that reads its rows again
        for (int q = 0; q < BATCH; ++q) {
            if (!((lv >> q) & 1u)) {
                primed = false;
                continue;
            }
            const int t = t0 + q, at = r + q;
            if ((sm >> q) & 1u) {
                enter(__shfl_sync(0xffffffffu, seq, at), t, __shfl_sync(0xffffffffu, hi, at));
            } else if (!primed) {
                prime(t);
            }
            primed = true;
            float x[V];
            load_v<T, V, WIDE>(src + t * ld, x);
            conv([&](int k) -> const float(&)[V] { return k < KT - 1 ? win[k < KT - 1 ? k : 0] : x; }, dst.p + t * dst.ld);
            slide(x);
        }
    }
    // first rows, past the run, of a sequence that started in its last K-2 rows
    const int lo31 = __shfl_sync(0xffffffffu, lo, 31), hi31 = __shfl_sync(0xffffffffu, hi, 31);
    if ((livem >> 31) && lo31 >= r0)
        for (int t = r0 + RUN; t < min(hi31, lo31 + K - 1); ++t) {
            float x[V];
            load_v<T, V, WIDE>(src + t * ld, x);
            conv([&](int k) -> const float(&)[V] { return k < KT - 1 ? win[k < KT - 1 ? k : 0] : x; }, dst.p + t * dst.ld);
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
    // one tap has no state to find: only a padding entry is skipped then
    const int slot = K > 1 ? slot_of(p.slots, p.nslots, i, p.dev_error) : p.slots ? min(p.slots[i], 0) : 0;
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
template <typename T, int V, int KT, bool EXACT>
__global__ void __launch_bounds__(32 * WARPS, V == 2 ? 5 : 4) conv_bwd_kernel(const T *__restrict__ in, long long ld,
                                                             const float *__restrict__ w,
                                                             const float *__restrict__ bias, const T *__restrict__ dxo,
                                                             const T *__restrict__ dbo, const T *__restrict__ dco,
                                                             T *__restrict__ dx, float *__restrict__ part, int cx,
                                                             int cb, int K, int silu, Packed p) {
    constexpr bool WIDE = V > 1;
    __shared__ float red[WARPS - 1][32][(KT + 1) * V + 1];
    const int ctot = cx + 2 * cb, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int tiles = (ctot + 32 * V - 1) / (32 * V), rows_at = blockIdx.x / tiles;  // a block's neighbours share its rows
    const int c = ((blockIdx.x % tiles) * 32 + lane) * V;
    const bool mine = c < ctot;
    const int cc = mine ? c : 0;
    if (blockIdx.x == 0) check_bounds(p);
    const int r0 = (rows_at * WARPS + wid) * RUN;
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
    // The batch below: inputs KT-1 rows back and upstream gradients, on their way.
    constexpr int BATCH = 4;
    using Vec = typename Ahead<T, V>::Vec;
    Vec nx[BATCH], ng[BATCH];
    auto fetch = [&](int t) {  // rows t, t-1, .. (clamped: rows outside are not used)
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int at = min(max(t - q, 0), p.tokens - 1);
            nx[q] = *reinterpret_cast<const Vec *>(in + cc + max(at - (KT - 1), 0) * ld);
            ng[q] = *reinterpret_cast<const Vec *>(src.p + at * src.ld);
        }
    };
    if (EXACT) fetch(r0 + RUN - 1);
    int seq, lo, hi;
    const bool live = row_seq(p, r0 + lane, seq, lo, hi);
    const int t_lane = r0 + lane;
    // rows that a batch cannot take straight: not live, the last of their sequence, or
    // with fewer than KT-1 rows of it before them
    const unsigned livem = __ballot_sync(0xffffffffu, live);
    const unsigned oddm = __ballot_sync(0xffffffffu, !live || t_lane == hi - 1 || t_lane - lo < KT - 1);
    float xw[KT][V], dp[KT][V];  // after row t: xw[j] = in[t-j]; dp[j] = dpre[t-1+j] (j > 0)
    // dout silu'(pre) for the inputs x(j) = in[t-j]
    auto dpre = [&](auto &&x, float (&d)[V]) {
        if (!silu) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = b[v];
#pragma unroll
            for (int j = 0; j < KT; ++j)
                if (EXACT || j < K) s = fmaf(wk[KT - 1 - j][v], x(j)[v], s);
            const float g = sigmoid_f(s);
            d[v] *= g * fmaf(s, 1.f - g, 1.f);
        }
    };
    // Row t of a sequence with first row `first`: its inputs into xw, its dpre into
    // dp[0]; taps before `first` read as zero.
    auto row_in = [&](int t, int first, bool primed) {
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
        load_v<T, V, WIDE>(src.p + t * src.ld, dp[0]);
        dpre([&](int j) -> const float(&)[V] { return xw[j]; }, dp[0]);
    };
    auto later = [&] {  // one row up: dp[j] becomes dpre[(t-1)+j]
#pragma unroll
        for (int j = KT - 1; j > 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) dp[j][v] = dp[j - 1][v];
    };
    // din of a row from d(j) = dpre[t+j], and the row's share of dw and dbias
    auto row_out = [&](auto &&x, auto &&d, float (&o)[V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = 0.f;
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                if (!EXACT && j >= K) continue;
                o[v] = fmaf(wk[KT - 1 - j][v], d(j)[v], o[v]);
                dw[KT - 1 - j][v] = fmaf(d(0)[v], x(j)[v], dw[KT - 1 - j][v]);
            }
            db[v] += d(0)[v];
        }
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
#pragma unroll 1
        for (int t = min(hi31, r0 + RUN + K - 1) - 1; t >= r0 + RUN; --t) {
            row_in(t, lo31, primed);
            later();
            primed = true;
        }
#pragma unroll 1
    for (int r = RUN - BATCH; r >= 0; r -= BATCH) {  // rows r0 + r + 3 down to r0 + r
        const int top = r0 + r + BATCH - 1;
        Vec cx_[BATCH], cg[BATCH];
        if (EXACT) {
#pragma unroll
            for (int q = 0; q < BATCH; ++q) cx_[q] = nx[q], cg[q] = ng[q];
            if (r >= BATCH) fetch(top - BATCH);
        }
        if (EXACT && primed && ((oddm >> r) & ((1u << BATCH) - 1)) == 0) {
            float x[KT - 1 + BATCH][V], d[KT - 1 + BATCH][V];  // x[i] = in[top-i], d[i] = dpre[top+KT-1-i]
#pragma unroll
            for (int j = 0; j < KT - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) x[j][v] = xw[j + 1][v], d[j][v] = dp[KT - 1 - j][v];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                load_v<T, V, WIDE>(reinterpret_cast<const T *>(&cx_[q]), x[KT - 1 + q]);
                load_v<T, V, WIDE>(reinterpret_cast<const T *>(&cg[q]), d[KT - 1 + q]);
                auto xq = [&](int j) -> const float(&)[V] { return x[q + j]; };
                dpre(xq, d[KT - 1 + q]);
                float o[V];
                row_out(xq, [&](int j) -> const float(&)[V] { return d[KT - 1 + q - j]; }, o);
                if (mine) store_v<T, V, WIDE>(dx + (size_t)(top - q) * ctot + cc, o);
            }
#pragma unroll
            for (int j = 0; j < KT - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) xw[j + 1][v] = x[BATCH + j][v], dp[KT - 1 - j][v] = d[BATCH + j][v];
            continue;
        }
#pragma unroll 1
        for (int t = top; t > top - BATCH; --t) {
            float o[V];
            if ((livem >> (t - r0)) & 1u) {
                const int first = __shfl_sync(0xffffffffu, lo, t - r0), end = __shfl_sync(0xffffffffu, hi, t - r0);
                if (t == end - 1) clear(), primed = false;  // nothing of this sequence lies later
                row_in(t, first, primed);
                primed = true;
                row_out([&](int j) -> const float(&)[V] { return xw[j]; }, [&](int j) -> const float(&)[V] { return dp[j]; }, o);
                later();
            } else {  // rows of no sequence have no gradient
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = 0.f;
                primed = false;
            }
            if (mine && t < p.tokens) store_v<T, V, WIDE>(dx + (size_t)t * ctot + cc, o);
        }
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
            float *o = part + ((size_t)rows_at * ctot + cc + v) * (K + 1);
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

// dw[c][k] and dbias[c] from the blocks' parts [parts][channels][K+1]: 32 warps take
// every 32nd.
__global__ void __launch_bounds__(1024) conv_bwd_sum(const float *__restrict__ part, int parts, int channels, int K,
                                                    float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5, n = channels * (K + 1), at = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (at < n)
#pragma unroll 4
        for (int i = q; i < parts; i += 32) a += part[(size_t)i * n + at];
    s[q][lane] = a;
    __syncthreads();
    a = s[lane][q];  // element q of the block
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const int e = blockIdx.x * 32 + q, c = e / (K + 1), k = e % (K + 1);
    if (lane || e >= n) return;
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

template <typename T, int V, int KT, bool EXACT> cudaError_t run_fwd(const ConvCall &c, cudaStream_t st) {
    const int ctot = c.cx + 2 * c.cb;
    const unsigned grid = (unsigned)((c.seq.tokens + RUN * WARPS - 1) / (RUN * WARPS) * ((ctot + 32 * V - 1) / (32 * V)));
    conv_varlen_kernel<T, V, KT, EXACT><<<grid, 32 * WARPS, 0, st>>>(
        static_cast<const T *>(c.in), c.ld, c.w, c.bias, static_cast<T *>(c.xo), static_cast<T *>(c.bo),
        static_cast<T *>(c.co), static_cast<T *>(c.state), c.cx, c.cb, c.width, c.silu, c.seq);
    return cudaGetLastError();
}
template <typename T, int V> cudaError_t pick_fwd(const ConvCall &c, cudaStream_t st) {
    if (c.width > 4) return run_fwd<T, 1, 8, false>(c, st);
    if (c.width < 4) return wide_rows(c, V) ? run_fwd<T, V, 4, false>(c, st) : run_fwd<T, 1, 4, false>(c, st);
    return wide_rows(c, V) ? run_fwd<T, V, 4, true>(c, st) : run_fwd<T, 1, 4, true>(c, st);
}

template <typename T, int V, int KT, bool EXACT> cudaError_t run_bwd(const ConvCall &c, float *ws, cudaStream_t st) {
    const int ctot = c.cx + 2 * c.cb, parts = (c.seq.tokens + RUN * WARPS - 1) / (RUN * WARPS);
    if (parts > 0) {
        const unsigned grid = (unsigned)(parts * ((ctot + 32 * V - 1) / (32 * V)));
        conv_bwd_kernel<T, V, KT, EXACT><<<grid, 32 * WARPS, 0, st>>>(
            static_cast<const T *>(c.in), c.ld, c.w, c.bias, static_cast<const T *>(c.xo),
            static_cast<const T *>(c.bo), static_cast<const T *>(c.co), static_cast<T *>(c.dx), ws, c.cx, c.cb,
            c.width, c.silu, c.seq);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    conv_bwd_sum<<<(ctot * (c.width + 1) + 31) / 32, 1024, 0, st>>>(ws, parts, ctot, c.width, c.dw, c.db);
    return cudaGetLastError();
}
template <typename T, int V> cudaError_t pick_bwd(const ConvCall &c, float *ws, cudaStream_t st) {
    if (c.width > 4) return run_bwd<T, 1, 8, false>(c, ws, st);
    if (c.width < 4) return wide_rows(c, V) ? run_bwd<T, V, 4, false>(c, ws, st) : run_bwd<T, 1, 4, false>(c, ws, st);
    return wide_rows(c, V) ? run_bwd<T, V, 4, true>(c, ws, st) : run_bwd<T, 1, 4, true>(c, ws, st);
}

}  // namespace

cudaError_t launch_conv_varlen(const ConvCall &c, cudaStream_t st) {
    return c.bf16 ? pick_fwd<__nv_bfloat16, 4>(c, st) : pick_fwd<float, 4>(c, st);
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
    return c.bf16 ? pick_bwd<__nv_bfloat16, 4>(c, ws, st) : pick_bwd<float, 2>(c, ws, st);
}

}  // namespace ssd
