// selscan_bwd.cu -- the gradient of the gated Mamba-1 scan on packed sequences.
//
// With a_t = exp(delta_t A), y = p silu(z), p = sum_n C h + D x and dp = dy silu(z):
//   g_t = dp_t C_t + a_{t+1} g_{t+1}            (the gradient at h_t, per state)
//   dC_t = sum_d dp_t h_t,  dB_t = sum_d delta_t x_t g_t          (over a group's channels)
//   du_t = sum_n g_t B_t,   q_t = g_t a_t h_{t-1},  dA = sum_t delta_t q_t
//   ddelta_t = x_t du_t + sum_n A q_t,  dx_t = delta_t du_t + D dp_t,  dD = sum_t dp_t x_t
//   dz_t = dy_t p_t silu'(z_t),  ddt_t = ddelta_t softplus'(dt_t + bias),  dbias = sum_t ddt_t.
//
// A block takes one sequence and CB channels and walks the chunks backwards.  In a
// chunk each state is run forwards from the kept chunk state (a and h_{t-1} stay in
// registers, so the exponentials are taken once) and then backwards, both split
// over the lanes of a channel as in the forward.  dB and dC are summed over a
// warp's channels by shuffles that halve the values with each step, over the
// block's warps in shared memory (each step of the state loop gives every warp
// another state, so there are no atomics and one fixed order), and over blocks by
// sel_bwd_sum.  Bound by issue: some 20 operations per state and token.
#include "selscan_tile.cuh"

namespace ssd {
namespace {

constexpr int TL = 8, K = SEL_CHUNK / TL, SEG = SEL_CHUNK, CL = 32 / TL, CB = SEL_WARPS * CL;
static_assert(CL == 4 && (K == 8 || K == 16), "the matrix instructions below sum 4 lanes, 8 or 16 tokens each");

// Sums over the four channels of a warp by matrix instructions: D[token][lane run] +=
// A[token][k] B[k][lane run], where B holds the lanes' values as they are (k: the four
// lanes of a run, times two registers) and A is ones for the k of one token and zero
// elsewhere.  One instruction sums two values of every lane over its run's channels,
// where shuffles that halve the values took twelve (32 of the 43 instructions per state
// and token were not the recurrence; the kernel took 1428 us against KERNEL_TIME at
// 64 x 512 tokens of 1024 channels and 16 states).
//   float32: each value goes in as two tf32 parts, its first 11 bits and the next 11, so
//   that it keeps 2^-22; the sums are float32.
//   bf16: the first part alone.  A product then loses what lies past 11 bits (below
//   2^-10 of it, a quarter of a step of the bf16 gradient it goes into); the sums are
//   float32 all the same.
template <typename T> struct ChannelSum {
    uint32_t one[8];  // row lane/4 of A has ones in its places for token i (mod 8)
    __device__ __forceinline__ explicit ChannelSum(int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) one[i] = (lane >> 2) == i ? 0x3f800000u : 0u;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, float b0, float b1) {
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
    }
    // d[0], d[1]: token lane/4 (d[2], d[3]: + 8) of lane runs 2 (lane%4) and + 1
    template <int H> __device__ __forceinline__ void operator()(const float2 (&v)[H], float (&d)[4]) const {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const uint32_t p = one[(2 * i) & 7], q = one[(2 * i + 1) & 7];
            const uint32_t a0 = i < 4 ? p : 0u, a1 = i < 4 ? 0u : p, a2 = i < 4 ? q : 0u, a3 = i < 4 ? 0u : q;
            if constexpr (sizeof(T) == 4) {
                const float x = __uint_as_float(__float_as_uint(v[i].x) & 0xffffe000u), y = __uint_as_float(__float_as_uint(v[i].y) & 0xffffe000u);
                mma(d, a0, a1, a2, a3, x, y);
                mma(d, a0, a1, a2, a3, v[i].x - x, v[i].y - y);
            } else {
                mma(d, a0, a1, a2, a3, v[i].x, v[i].y);
            }
        }
    }
};

template <typename T> struct BwdShape {
    using Rows = RowTile<T, SEG, CB, TL>;
    using BC = BCTile<T, SEG, TL>;
    static size_t smem(int N) {
        return 4 * (size_t)Rows::BYTES + (size_t)N * BC::STATE_WORDS * 4 + 2 * (size_t)N * SEG * 4 + 4 * (size_t)CB * N * 4;
    }
};

struct Parts {      // workspace
    float *bc;      // [groups * tiles][tokens][2][dstate]
    float *a;       // [nseq][channels][dstate]
    float *d;       // [nseq][2][channels]: dD, dbias
};

// Where a lane stands and what its block holds in shared memory.
struct Lane {
    int l, ch, w;        // lane run, channel of the block, warp
    int mine;            // real tokens of the run
    float bias, D;
    unsigned char *xs, *ds, *zs, *ys;
    const uint32_t *bc;
    const float *As, *hs;
    float *gs, *dAs, *sB, *sC;
};

// One chunk of 4 Q token slots per lane run: on return the tiles x, dt, z hold dx,
// ddt, dz.  dD and dbias go on in the lane's registers.
template <typename T, int Q>
__device__ __forceinline__ void bwd_chunk(const SelCall &c, const Lane &a, float &dD, float &dbias) {
    using Rows = typename BwdShape<T>::Rows;
    using BC = typename BwdShape<T>::BC;
    constexpr int LEN = 4 * Q, H = LEN / 2;
    const int N = c.dstate, M = max(N, SEL_WARPS), l = a.l, ch = a.ch;
    float2 dl[H], u2[H], dp[H], du[H], sd[H], p2[H];
    float total = 0.f;
    T *const px = Rows::row(a.xs, l * LEN, l) + ch, *const pd = Rows::row(a.ds, l * LEN, l) + ch;
    T *const pz = Rows::row(a.zs, l * LEN, l) + ch, *const py = Rows::row(a.ys, l * LEN, l) + ch;
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        const bool in = k < a.mine;
        float d = ld_f32<T>(pd + k * CB) + a.bias, e = ld_f32<T>(py + k * CB);
        if (c.softplus) d = softplus_f(d);
        if (c.z) e *= silu_v(ld_f32<T>(pz + k * CB));
        d = in ? d : 0.f, e = in ? e : 0.f;
        const float u = in ? d * ld_f32<T>(px + k * CB) : 0.f;
        total += d;
        if (k & 1)
            dl[k / 2].y = d, u2[k / 2].y = u, dp[k / 2].y = e;
        else
            dl[k / 2].x = d, u2[k / 2].x = u, dp[k / 2].x = e;
    }
#pragma unroll
    for (int k = 0; k < H; ++k) du[k] = sd[k] = p2[k] = make_float2(0.f, 0.f);
    const ChannelSum<T> channel_sum(threadIdx.x & 31);
    // The sum of v over the warp's channels into the block's sums, [token][lane run].
    auto reduce = [&](const float2 (&v)[H], float *acc) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        channel_sum(v, d);
        float2 *o = reinterpret_cast<float2 *>(acc) + (threadIdx.x & 31);
        *o = add2(*o, make_float2(d[0], d[1]));
        if (LEN > 8) o[32] = add2(o[32], make_float2(d[2], d[3]));
    };
#pragma unroll 1
    for (int it = 0; it < M; ++it) {
        const int s = it + a.w < M ? it + a.w : it + a.w - M;
        if (s < N) {
            const float A2 = a.As[s * CB + ch], hc = a.hs[s * CB + ch], gc = a.gs[s * CB + ch];
            const float2 A22 = splat(A2);
            float2 a2[H], hp[H], v2[H], b2[H], c2[H];
            // forwards: v2 holds the inputs, then dp h
            float S_ = 0.f, P = ex2a(A2 * total);
            const float P0 = P;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                BC::quad(a.bc, s, q, l, b2 + 2 * q, c2 + 2 * q);
#pragma unroll
                for (int k = 2 * q; k < 2 * q + 2; ++k) {
                    const float2 arg = mul2(dl[k], A22);
                    a2[k] = make_float2(ex2a(arg.x), ex2a(arg.y));
                    v2[k] = mul2(u2[k], b2[k]);
                    S_ = fmaf(a2[k].x, S_, v2[k].x);
                    S_ = fmaf(a2[k].y, S_, v2[k].y);
                }
            }
            if (l == 0) S_ = fmaf(P, hc, S_);
#pragma unroll
            for (int o = 1; o < TL; o *= 2) {
                const float Sp = __shfl_up_sync(0xffffffffu, S_, o * CL), Pp = __shfl_up_sync(0xffffffffu, P, o * CL);
                if (l >= o) S_ = fmaf(P, Sp, S_), P *= Pp;
            }
            float h = __shfl_up_sync(0xffffffffu, S_, CL);
            if (l == 0) h = hc;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                float2 hh;
                hp[k].x = h;
                hh.x = h = fmaf(a2[k].x, h, v2[k].x);
                hp[k].y = h;
                hh.y = h = fmaf(a2[k].y, h, v2[k].y);
                p2[k] = fma2(c2[k], hh, p2[k]);
                v2[k] = mul2(dp[k], hh);
            }
            reduce(v2, a.sC + s * SEG);
            // backwards: G = a g, what a token hands to the one before it
            float R = 0.f;
            P = P0;
#pragma unroll
            for (int k = H - 1; k >= 0; --k) {
                v2[k] = mul2(dp[k], c2[k]);
                R = a2[k].y * (R + v2[k].y);
                R = a2[k].x * (R + v2[k].x);
            }
            if (l == TL - 1) R = fmaf(P, gc, R);
#pragma unroll
            for (int o = 1; o < TL; o *= 2) {
                const float Rn = __shfl_down_sync(0xffffffffu, R, o * CL), Pn = __shfl_down_sync(0xffffffffu, P, o * CL);
                if (l + o < TL) R = fmaf(P, Rn, R), P *= Pn;
            }
            float G = __shfl_down_sync(0xffffffffu, R, CL);
            if (l == TL - 1) G = gc;
            if (l == 0) a.gs[s * CB + ch] = R;
            float2 dA2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = H - 1; k >= 0; --k) {
                float2 gg, GG;
                gg.y = G + v2[k].y, GG.y = G = a2[k].y * gg.y;
                gg.x = G + v2[k].x, GG.x = G = a2[k].x * gg.x;
                const float2 qq = mul2(GG, hp[k]);
                du[k] = fma2(gg, b2[k], du[k]);
                sd[k] = fma2(A22, qq, sd[k]);
                dA2 = fma2(dl[k], qq, dA2);
                v2[k] = mul2(u2[k], gg);
            }
            reduce(v2, a.sB + s * SEG);
            float dA = dA2.x + dA2.y;
#pragma unroll
            for (int o = CL; o < 32; o *= 2) dA += __shfl_xor_sync(0xffffffffu, dA, o);
            if (l == 0) a.dAs[s * CB + ch] += dA;
        }
        __syncthreads();  // the next state's sums
    }
#pragma unroll
    for (int k = 0; k < LEN; ++k) {
        const bool in = k < a.mine;
        const float d = k & 1 ? dl[k / 2].y : dl[k / 2].x, e = k & 1 ? dp[k / 2].y : dp[k / 2].x;
        const float duk = k & 1 ? du[k / 2].y : du[k / 2].x;
        const float sdk = (k & 1 ? sd[k / 2].y : sd[k / 2].x) * 0.6931471805599453f;  // A was scaled by log2 e
        const float xv = ld_f32<T>(px + k * CB);
        float ddt = fmaf(xv, duk, sdk);
        if (c.softplus) ddt *= sigmoid_f(ld_f32<T>(pd + k * CB) + a.bias);
        dD += in ? e * xv : 0.f;
        dbias += in ? ddt : 0.f;
        if (c.z) {
            const float zv = ld_f32<T>(pz + k * CB), sg = sigmoid_f(zv);
            const float pre = fmaf(a.D, xv, k & 1 ? p2[k / 2].y : p2[k / 2].x);
            const float dz = ld_f32<T>(py + k * CB) * pre * sg * fmaf(zv, 1.f - sg, 1.f);
            if (in) st_f32<T>(pz + k * CB, dz);
        }
        if (in) {
            st_f32<T>(px + k * CB, fmaf(d, duk, a.D * e));
            st_f32<T>(pd + k * CB, ddt);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(SEL_WARPS * 32, 1) sel_bwd_kernel(SelCall c, Parts parts, bool wide, bool wide_bc) {
    using S = BwdShape<T>;
    using Rows = typename S::Rows;
    using BC = typename S::BC;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char *xs = smem, *ds = xs + Rows::BYTES, *zs = ds + Rows::BYTES, *ys = zs + Rows::BYTES;
    uint32_t *bc = reinterpret_cast<uint32_t *>(ys + Rows::BYTES);
    const int N = c.dstate;
    float *sB = reinterpret_cast<float *>(bc + N * BC::STATE_WORDS), *sC = sB + N * SEG;  // sums over the block's channels
    float *As = sC + N * SEG, *hs = As + CB * N, *gs = hs + CB * N, *dAs = gs + CB * N;   // [n][channel]

    const int i = blockIdx.x;
    const int per_group = c.channels / c.groups, tiles = (per_group + CB - 1) / CB;
    const int g = blockIdx.y / tiles, c0 = g * per_group + (blockIdx.y % tiles) * CB;
    const int cols = min(CB, (g + 1) * per_group - c0);
    int lo, hi;
    if (!seq_rows(c.seq, i, lo, hi)) lo = hi = 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, l = lane / CL, ch = w * CL + lane % CL;
    const int chc = min(ch, cols - 1);
    const float bias = c.dt_bias ? c.dt_bias[c0 + chc] : 0.f, Dv = c.D ? c.D[c0 + chc] : 0.f;
    const T *x = static_cast<const T *>(c.x) + c0, *dt = static_cast<const T *>(c.dt) + c0,
            *z = static_cast<const T *>(c.z) + c0, *dy = static_cast<const T *>(c.dy) + c0;
    const T *B = static_cast<const T *>(c.B) + g * N, *C = static_cast<const T *>(c.C) + g * N;
    for (int u = threadIdx.x; u < CB * N; u += SEL_WARPS * 32) {
        const int cc = u / N, n = u - cc * N;
        As[n * CB + cc] = cc < cols ? c.A[(size_t)c0 * N + u] * LOG2E : 0.f;
        gs[n * CB + cc] = dAs[n * CB + cc] = 0.f;
    }
    float dD = 0.f, dbias = 0.f;
    Lane at{l, ch, w, 0, bias, Dv, xs, ds, zs, ys, bc, As, hs, gs, dAs, sB, sC};
    const int chunks = (hi - lo + SEG - 1) / SEG;
    for (int chunk = chunks - 1; chunk >= 0; --chunk) {
        const int t0 = lo + chunk * SEG, n = min(SEG, hi - t0), per_lane = (n + TL - 1) / TL, len = per_lane <= 4 ? 4 : per_lane <= 8 ? 8 : K;
        __syncthreads();  // the tiles are free again
        Rows::fetch(xs, x + t0 * c.ld_x, c.ld_x, n, cols, len, wide);
        Rows::fetch(ds, dt + t0 * c.ld_dt, c.ld_dt, n, cols, len, wide);
        if (c.z) Rows::fetch(zs, z + t0 * c.ld_z, c.ld_z, n, cols, len, wide);
        Rows::fetch(ys, dy + (size_t)t0 * c.channels, c.channels, n, cols, len, wide);
        cp_commit();
        BC::fetch(bc, B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, n, N, len, wide_bc);
        const float *kept = c.chunk_states + ((size_t)(lo / SEL_CHUNK + i + chunk) * c.channels + c0) * N;
        for (int u = threadIdx.x; u < CB * N; u += SEL_WARPS * 32)
            hs[(u % N) * CB + u / N] = u < cols * N ? kept[u] : 0.f;
        for (int u = threadIdx.x; u < N * SEG; u += SEL_WARPS * 32) sB[u] = sC[u] = 0.f;
        cp_wait<0>();
        __syncthreads();
        at.mine = ch < cols ? max(0, min(len, n - l * len)) : 0;
        if (len == 4)
            bwd_chunk<T, 1>(c, at, dD, dbias);
        else if (K == 8 || len == 8)
            bwd_chunk<T, 2>(c, at, dD, dbias);
        else if (K == 16)
            bwd_chunk<T, K / 4>(c, at, dD, dbias);
        __syncthreads();
        const size_t row0 = (size_t)t0 * c.channels + c0;
        Rows::flush(xs, static_cast<T *>(c.dx) + row0, c.channels, n, cols, len, wide);
        Rows::flush(ds, static_cast<T *>(c.ddt) + row0, c.channels, n, cols, len, wide);
        if (c.z) Rows::flush(zs, static_cast<T *>(c.dz) + row0, c.channels, n, cols, len, wide);
        float *pb = parts.bc + ((size_t)blockIdx.y * c.seq.tokens + t0) * 2 * N;
        for (int u = threadIdx.x; u < n * N; u += SEL_WARPS * 32) {
            const int r = u / N, s = u - r * N, run = r / len, o = s * SEG + (r - run * len) * TL + run;
            pb[r * 2 * N + s] = sB[o];
            pb[r * 2 * N + N + s] = sC[o];
        }
    }
    __syncthreads();
    float *pa = parts.a + ((size_t)i * c.channels + c0) * N;
    for (int u = threadIdx.x; u < cols * N; u += SEL_WARPS * 32) pa[u] = dAs[(u % N) * CB + u / N];
#pragma unroll
    for (int o = CL; o < 32; o *= 2) {
        dD += __shfl_xor_sync(0xffffffffu, dD, o);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
    }
    if (l == 0 && ch < cols) {
        float *pd = parts.d + (size_t)i * 2 * c.channels + c0 + ch;
        pd[0] = dD;
        pd[c.channels] = dbias;
    }
}

// The sums over blocks.  The first row_blocks blocks: dB and dC, a warp per token,
// from the channel tiles of each group; a token of no sequence gets zero gradients.
// The others: dA, dD and dbias over the sequences, a thread per element.
template <typename T>
__global__ void __launch_bounds__(256) sel_bwd_sum(SelCall c, Parts parts, int row_blocks) {
    const int N = c.dstate, G = c.groups, per_group = c.channels / G, tiles = (per_group + CB - 1) / CB;
    if ((int)blockIdx.x < row_blocks) {
        const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        if (t >= c.seq.tokens) return;
        int a = -1, b = c.seq.nseq;  // the last sequence that starts at or before t
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (c.seq.cu[m] <= t) a = m; else b = m;
        }
        const bool held = a >= 0 && c.seq.cu[a] >= 0 && t < c.seq.cu[a + 1] && c.seq.cu[a + 1] <= c.seq.tokens;
        T *dB = static_cast<T *>(c.dB) + (size_t)t * G * N, *dC = static_cast<T *>(c.dC) + (size_t)t * G * N;
        for (int u = lane; u < G * 2 * N; u += 32) {
            const int g = u / (2 * N), k = u - g * 2 * N;
            float s = 0.f;
            if (held)
                for (int j = 0; j < tiles; ++j) s += parts.bc[((size_t)(g * tiles + j) * c.seq.tokens + t) * 2 * N + k];
            st_f32<T>(k < N ? dB + g * N + k : dC + g * N + k - N, s);
        }
        if (!held)
            for (int d = lane; d < c.channels; d += 32) {
                const size_t o = (size_t)t * c.channels + d;
                st_f32<T>(static_cast<T *>(c.dx) + o, 0.f);
                st_f32<T>(static_cast<T *>(c.ddt) + o, 0.f);
                if (c.z) st_f32<T>(static_cast<T *>(c.dz) + o, 0.f);
            }
        return;
    }
    const long long u = (long long)(blockIdx.x - row_blocks) * 256 + threadIdx.x, na = (long long)c.channels * N;
    if (u < na) {
        float s = 0.f;
        for (int i = 0; i < c.seq.nseq; ++i) s += parts.a[(size_t)i * na + u];
        c.dA[u] = s;
    } else if (u < na + 2 * c.channels) {
        const long long v = u - na;
        float s = 0.f;
        for (int i = 0; i < c.seq.nseq; ++i) s += parts.d[(size_t)i * 2 * c.channels + v];
        float *o = v < c.channels ? c.dD : c.dbias;
        if (o) o[v < c.channels ? v : v - c.channels] = s;
    }
}

size_t bc_floats(int tokens, int channels, int groups, int dstate) {
    return (size_t)groups * ((channels / groups + CB - 1) / CB) * tokens * 2 * dstate;
}

template <typename T> cudaError_t run(const SelCall &c, float *ws, cudaStream_t st) {
    using S = BwdShape<T>;
    const size_t e = sizeof(T), smem = S::smem(c.dstate);
    const int per_group = c.channels / c.groups;
    const bool wide = rows_aligned(c.x, c.ld_x, e, 16) && rows_aligned(c.dt, c.ld_dt, e, 16) &&
                      (!c.z || rows_aligned(c.z, c.ld_z, e, 16)) && c.channels * e % 16 == 0 && per_group * e % 16 == 0;
    const bool wide_bc = c.dstate % 4 == 0 && rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
    Parts p;
    p.bc = ws;
    p.a = p.bc + bc_floats(c.seq.tokens, c.channels, c.groups, c.dstate);
    p.d = p.a + (size_t)c.seq.nseq * c.channels * c.dstate;
    if (c.seq.nseq > 0 && c.seq.tokens > 0) {
        cudaError_t err = cudaFuncSetAttribute(sel_bwd_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        const dim3 grid(c.seq.nseq, c.groups * ((per_group + CB - 1) / CB));
        sel_bwd_kernel<T><<<grid, SEL_WARPS * 32, smem, st>>>(c, p, wide, wide_bc);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    SelCall s = c;
    if (c.seq.tokens == 0) s.seq.nseq = 0;  // nothing was summed
    const int row_blocks = (c.seq.tokens + 7) / 8;
    const long long rest = ((long long)c.channels * (c.dstate + 2) + 255) / 256;
    sel_bwd_sum<T><<<(unsigned)(row_blocks + rest), 256, 0, st>>>(s, p, row_blocks);
    return cudaGetLastError();
}

}  // namespace

size_t sel_bwd_workspace(int tokens, int nseq, int channels, int groups, int dstate) {
    return (bc_floats(tokens, channels, groups, dstate) + (size_t)nseq * channels * (dstate + 2)) * sizeof(float);
}

cudaError_t launch_sel_bwd(const SelCall &c, void *ws, cudaStream_t st) {
    return c.bf16 ? run<__nv_bfloat16>(c, static_cast<float *>(ws), st) : run<float>(c, static_cast<float *>(ws), st);
}

}  // namespace ssd
