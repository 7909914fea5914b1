// selscan_bwd.cu -- the gradient of the gated Mamba-1 scan on packed sequences.
//
// With a_t = exp(delta_t A), y = p silu(z), p = sum_n C h + D x and dp = dy silu(z):
//   g_t = dp_t C_t + G_{t+1},  G_t = a_t g_t     (the gradient at h_t, and what it hands back)
//   dC_t = sum_d dp_t h_t,  dB_t = sum_d delta_t x_t g_t          (over a group's channels)
//   du_t = sum_n g_t B_t,   q_t = G_t h_{t-1},  dA = sum_t delta_t q_t
//   ddelta_t = x_t du_t + sum_n A q_t,  dx_t = delta_t du_t + D dp_t,  dD = sum_t dp_t x_t
//   dz_t = dy_t p_t silu'(z_t),  ddt_t = ddelta_t softplus'(dt_t + bias),  dbias = sum_t ddt_t.
//
// A thread per channel walks its sequence (or segment, selscan_seg.cuh) backwards, in
// chunks of SEL_CHUNK tokens that start where the forward kept the states, and a chunk
// in two halves of SUB tokens.  For each half and pair of states it runs the
// recurrence forwards (a_t and h_{t-1} stay in registers, so the backward walk takes no
// exponential) and then backwards, two states to a packed operation; the second half
// starts from a state formed again from the first half's tokens, which costs half an
// exponential per state and token and halves the states to keep.  Per state and token:
// 7 operations, half of an extra forward step, 2 for the sums over channels.
// dB and dC are summed over a warp's channels by matrix instructions (ChannelSum), over
// the block's warps in shared memory, and over blocks by sel_bwd_sum, all in a fixed
// order.  Bound by issue.  A first form split a chunk's tokens over the lanes of a warp
// like the forward's; its scans, its scalar chains and one barrier per state left it at
// 1428 us where this one takes KERNEL_TIME (64 x 512 tokens, 1024 channels, 16 states).
#include "selscan_seg.cuh"

namespace ssd {
namespace {

constexpr int SUB = 8;
static_assert(SEL_CHUNK == 2 * SUB, "a chunk is two halves");

// Sums over the 32 channels of a warp by matrix instructions: D[value][lane/4] +=
// A[value][k] B[k][lane/4], where B holds the lanes' values as they are (k: the four
// lanes of a group, times two registers) and A is ones for the k of one value and zero
// elsewhere; two shuffles and three additions are left for the eight groups.  Sixteen
// values take 8 instructions and those, where shuffles that halve the values took 124.
//   float32: each value goes in as two tf32 parts, its first 11 bits and the next 11, so
//   that it keeps 2^-22; the sums are float32.
//   bf16: the first part alone.  A product then loses what lies past 11 bits (below
//   2^-10 of it, a quarter of a step of the bf16 gradient it goes into); the sums are
//   float32 all the same.
template <typename T> struct ChannelSum {
    uint32_t one[8];  // row lane/4 of A is all ones for value i (mod 8)
    __device__ __forceinline__ explicit ChannelSum(int lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) one[i] = (lane >> 2) == i ? 0x3f800000u : 0u;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, float b0, float b1) {
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
    }
    // Lanes 0 and 1 of each group of four end with the warp's sum of value lane/4 and
    // lane/4 + 8, where value 2 i is v[i].x and value 2 i + 1 is v[i].y.
    __device__ __forceinline__ float operator()(const float2 (&v)[8], int lane) const {
        float d[4] = {0.f, 0.f, 0.f, 0.f};  // rows lane/4 and lane/4 + 8, columns 2 (lane%4) and + 1
#pragma unroll
        for (int i = 0; i < 8; ++i) {
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
        const float s0 = d[0] + d[1], s1 = d[2] + d[3];
        const float s = (lane & 1 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, lane & 1 ? s0 : s1, 1);
        return s + __shfl_xor_sync(0xffffffffu, s, 2);
    }
};

__device__ __forceinline__ void cp16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp4(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int NP> constexpr int bwd_threads() { return NP <= 32 ? 128 : 64; }

template <typename T, int NP> struct BwdShared {
    static constexpr int THREADS = bwd_threads<NP>(), P = NP / 2, WARPS = THREADS / 32;
    T x[SEL_CHUNK][THREADS], dt[SEL_CHUNK][THREADS], z[SEL_CHUNK][THREADS], dy[SEL_CHUNK][THREADS];
    float4 bc[SEL_CHUNK * P];
    float2 A2[P][THREADS], G[P][THREADS], dA[P][THREADS], hm[P][THREADS];  // hm: the state before the second half
    float h0[NP][THREADS];                                                // the state before the chunk
    float part[WARPS][SUB][2][NP];                                        // a warp's sums: [token][dB, dC][state]
};

struct Parts {   // workspace
    float *bc;   // [channel tiles][tokens][2][dstate]
    float *a;    // [slots][dstate][channels]
    float *d;    // [slots][2][channels]: dD, dbias
};

// n rows of `cols` channels into [SEL_CHUNK][THREADS]; wide: aligned 16-byte pieces
template <typename T, int THREADS>
__device__ __forceinline__ void fetch_rows(T (*to)[THREADS], const T *src, long long ld, int n, int cols, bool wide) {
    if (wide) {
        constexpr int E = 16 / (int)sizeof(T), PER = THREADS / E;
        for (int u = threadIdx.x; u < n * PER; u += THREADS) {
            const int r = u / PER, k = u % PER * E;
            if (k < cols) cp16(&to[r][k], src + r * ld + k);
        }
    } else if ((int)threadIdx.x < cols) {
        for (int r = 0; r < n; ++r) to[r][threadIdx.x] = src[r * ld + threadIdx.x];
    }
}

template <typename T, int NP>
__global__ void __launch_bounds__(bwd_threads<NP>(), NP <= 16 ? 3 : 1) sel_bwd_kernel(SelCall c, Segments sg, Parts parts, bool wide,
                                                                             bool wide_states) {
    using Sh = BwdShared<T, NP>;
    constexpr int P = NP / 2, THREADS = Sh::THREADS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sh &sh = *reinterpret_cast<Sh *>(smem_raw);
    const Mine me = my_channel<THREADS>(c, blockIdx.y);
    const int N = c.dstate, d = me.channel, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t step = (size_t)N * c.channels;
    float *const pa = parts.a + blockIdx.x * step + d, *const pd_ = parts.d + (size_t)blockIdx.x * 2 * c.channels + d;
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end)) {  // the same for the whole block
        if (me.in) {
            for (int n = 0; n < N; ++n) pa[(size_t)n * c.channels] = 0.f;
            pd_[0] = pd_[c.channels] = 0.f;
        }
        return;
    }
    const int per_group = c.channels / c.groups, tiles = (per_group + THREADS - 1) / THREADS;
    const int t_first = me.group * per_group + blockIdx.y % tiles * THREADS, t_cols = min(THREADS, (me.group + 1) * per_group - t_first);
    const float bias = c.dt_bias ? c.dt_bias[d] : 0.f, Dv = c.D ? c.D[d] : 0.f;
    const ChannelSum<T> channel_sum(lane);
    for (int p = 0; p < P; ++p) {
        const int n = 2 * p;
        sh.A2[p][tid] = make_float2(n < N ? c.A[(size_t)d * N + n] * LOG2E : 0.f, n + 1 < N ? c.A[(size_t)d * N + n + 1] * LOG2E : 0.f);
        sh.dA[p][tid] = make_float2(0.f, 0.f);
        float2 G = make_float2(0.f, 0.f);
        if (sg.seg != WHOLE) {
            const float *from = sg.state + blockIdx.x * step + d;
            if (n < N) G.x = from[(size_t)n * c.channels];
            if (n + 1 < N) G.y = from[(size_t)(n + 1) * c.channels];
        }
        sh.G[p][tid] = G;
    }
    for (int n = N; n < NP; ++n) sh.h0[n][tid] = 0.f;
    float dD = 0.f, dbias = 0.f;
    StageBC<T, NP, SEL_CHUNK, THREADS> stage;
    const T *B = static_cast<const T *>(c.B) + me.group * N, *C = static_cast<const T *>(c.C) + me.group * N;
    const int c_first = (lo - first) / SEL_CHUNK, c_last = (hi - 1 - first) / SEL_CHUNK;
    const float *kept = c.chunk_states + (size_t)(first / SEL_CHUNK + i) * step + d;
    {
        const int t0 = first + c_last * SEL_CHUNK;
        stage.load(B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, min(SEL_CHUNK, hi - t0), N, wide_states);
    }
    for (int chunk = c_last; chunk >= c_first; --chunk) {
        const int t0 = first + chunk * SEL_CHUNK, n = min(SEL_CHUNK, hi - t0);
        __syncthreads();  // the chunk before has been read
        fetch_rows<T, THREADS>(sh.x, static_cast<const T *>(c.x) + t0 * c.ld_x + t_first, c.ld_x, n, t_cols, wide);
        fetch_rows<T, THREADS>(sh.dt, static_cast<const T *>(c.dt) + t0 * c.ld_dt + t_first, c.ld_dt, n, t_cols, wide);
        if (c.z) fetch_rows<T, THREADS>(sh.z, static_cast<const T *>(c.z) + t0 * c.ld_z + t_first, c.ld_z, n, t_cols, wide);
        fetch_rows<T, THREADS>(sh.dy, static_cast<const T *>(c.dy) + (size_t)t0 * c.channels + t_first, c.channels, n, t_cols, wide);
        for (int s = 0; s < N; ++s) cp4(&sh.h0[s][tid], kept + chunk * step + (size_t)s * c.channels);
        stage.put(sh.bc);
        if (chunk > c_first) {
            const int tp = t0 - SEL_CHUNK;
            stage.load(B + tp * c.ld_b, c.ld_b, C + tp * c.ld_c, c.ld_c, SEL_CHUNK, N, wide_states);
        }
        cp_wait_all();
        __syncthreads();

        // step size of row r; tokens past the end, and threads without a channel, take steps
        // of nothing (their rows of the tiles were never written)
        auto step_of = [&](int r) {
            const float v = ld_f32<T>(&sh.dt[r][tid]) + bias;
            const float s = c.softplus ? softplus_f(v) : v;
            return r < n && me.in ? s : 0.f;
        };
        if (n > SUB) {  // the state before the second half
            float2 dl[SUB], u2[SUB];
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
                const float s = step_of(k);
                dl[k] = splat(s), u2[k] = splat(me.in ? s * ld_f32<T>(&sh.x[k][tid]) : 0.f);
            }
#pragma unroll 2
            for (int p = 0; p < P; ++p) {
                const float2 A2 = sh.A2[p][tid];
                float2 h = make_float2(sh.h0[2 * p][tid], sh.h0[2 * p + 1][tid]);
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const float2 b = *reinterpret_cast<const float2 *>(sh.bc + k * P + p), arg = mul2(dl[k], A2);
                    h = fma2(make_float2(ex2a(arg.x), ex2a(arg.y)), h, mul2(u2[k], b));
                }
                sh.hm[p][tid] = h;
            }
        }
        for (int half = n > SUB ? 1 : 0; half >= 0; --half) {
            const int k0 = half * SUB;
            float2 dl[SUB], u2[SUB], dp[SUB], du[SUB], sd[SUB], pre[SUB];
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
                const bool in = k0 + k < n && me.in;
                const float s = step_of(k0 + k);
                float e = ld_f32<T>(&sh.dy[k0 + k][tid]);
                if (c.z) e *= silu_v(ld_f32<T>(&sh.z[k0 + k][tid]));
                dl[k] = splat(s), u2[k] = splat(in ? s * ld_f32<T>(&sh.x[k0 + k][tid]) : 0.f), dp[k] = splat(in ? e : 0.f);
                du[k] = sd[k] = pre[k] = make_float2(0.f, 0.f);
            }
#pragma unroll 1
            for (int p = 0; p < P; ++p) {
                const float2 A2 = sh.A2[p][tid];
                float2 h = half ? sh.hm[p][tid] : make_float2(sh.h0[2 * p][tid], sh.h0[2 * p + 1][tid]);
                float2 a[SUB], hp[SUB], v[SUB];
                const float4 *q = sh.bc + k0 * P + p;
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const float4 bc = q[k * P];
                    const float2 arg = mul2(dl[k], A2);
                    a[k] = make_float2(ex2a(arg.x), ex2a(arg.y));
                    hp[k] = h;
                    h = fma2(a[k], h, mul2(u2[k], make_float2(bc.x, bc.y)));
                    pre[k] = fma2(make_float2(bc.z, bc.w), h, pre[k]);
                    v[k] = mul2(dp[k], h);
                }
                const float sC = channel_sum(v, lane);
                float2 G = sh.G[p][tid], dA = sh.dA[p][tid];
#pragma unroll
                for (int k = SUB - 1; k >= 0; --k) {
                    const float4 bc = q[k * P];
                    const float2 g = fma2(dp[k], make_float2(bc.z, bc.w), G);
                    G = mul2(a[k], g);
                    const float2 qq = mul2(G, hp[k]);
                    du[k] = fma2(g, make_float2(bc.x, bc.y), du[k]);
                    sd[k] = fma2(A2, qq, sd[k]);
                    dA = fma2(dl[k], qq, dA);
                    v[k] = mul2(u2[k], g);
                }
                sh.G[p][tid] = G, sh.dA[p][tid] = dA;
                const float sB = channel_sum(v, lane);
                if ((lane & 3) < 2) {  // value lane/4 (+ 8): token value/2, state 2 p + value%2
                    const int value = (lane >> 2) + 8 * (lane & 1);
                    float *o = &sh.part[warp][value >> 1][0][2 * p + (value & 1)];
                    o[0] = sB, o[NP] = sC;
                }
            }
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
                const int r = k0 + k;
                const bool in = r < n && me.in;
                const float xv = ld_f32<T>(&sh.x[r][tid]), duk = du[k].x + du[k].y;
                float ddt = fmaf(xv, duk, (sd[k].x + sd[k].y) * 0.6931471805599453f);  // A was scaled by log2 e
                if (c.softplus) ddt *= sigmoid_f(ld_f32<T>(&sh.dt[r][tid]) + bias);
                const size_t o = (size_t)(t0 + r) * c.channels + d;
                if (in) {
                    st_f32<T>(static_cast<T *>(c.dx) + o, fmaf(dl[k].x, duk, Dv * dp[k].x));
                    st_f32<T>(static_cast<T *>(c.ddt) + o, ddt);
                    dD = fmaf(dp[k].x, xv, dD);
                    dbias += ddt;
                    if (c.z) {
                        const float zv = ld_f32<T>(&sh.z[r][tid]), s = sigmoid_f(zv), p = fmaf(Dv, xv, pre[k].x + pre[k].y);
                        st_f32<T>(static_cast<T *>(c.dz) + o, ld_f32<T>(&sh.dy[r][tid]) * p * s * fmaf(zv, 1.f - s, 1.f));
                    }
                }
            }
            __syncthreads();  // every warp's sums are there
            for (int u = tid; u < SUB * 2 * NP; u += THREADS) {
                const int t = u / (2 * NP), k = u % (2 * NP), s = k % NP;
                float v = (&sh.part[0][0][0][0])[u];
#pragma unroll
                for (int w = 1; w < Sh::WARPS; ++w) v += (&sh.part[w][0][0][0])[u];
                if (s < N && k0 + t < n) parts.bc[((size_t)blockIdx.y * c.seq.tokens + t0 + k0 + t) * 2 * N + (k / NP) * N + s] = v;
            }
            __syncthreads();  // before the other half's
        }
    }
    if (!me.in) return;
    for (int s = 0; s < N; ++s) pa[(size_t)s * c.channels] = s & 1 ? sh.dA[s / 2][tid].y : sh.dA[s / 2][tid].x;
    pd_[0] = dD;
    pd_[c.channels] = dbias;
}

// What a segment hands back when nothing comes from behind it, and its sum of steps: for
// sel_join.  The first segment of a sequence hands back to nobody.
constexpr int CARRY_THREADS = 64;
template <typename T, int NP>
__global__ void __launch_bounds__(CARRY_THREADS) sel_carry_kernel(SelCall c, Segments sg, bool wide) {
    constexpr int P = NP / 2;
    using Stage = StageBC<T, NP, SEL_CHUNK, CARRY_THREADS>;
    __shared__ __align__(16) float4 bc[Stage::BYTES / 16];
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end) || lo == first) return;
    const Mine me = my_channel<CARRY_THREADS>(c, blockIdx.y);
    const int N = c.dstate, d = me.channel;
    const T *B = static_cast<const T *>(c.B) + me.group * N, *C = static_cast<const T *>(c.C) + me.group * N;
    const T *dt = static_cast<const T *>(c.dt) + d, *z = static_cast<const T *>(c.z) + (c.z ? d : 0), *dy = static_cast<const T *>(c.dy) + d;
    float2 A2[P], R[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        A2[p] = make_float2(2 * p < N ? c.A[(size_t)d * N + 2 * p] * LOG2E : 0.f, 2 * p + 1 < N ? c.A[(size_t)d * N + 2 * p + 1] * LOG2E : 0.f);
        R[p] = make_float2(0.f, 0.f);
    }
    const float bias = c.dt_bias ? c.dt_bias[d] : 0.f;
    float steps = 0.f;
    for (int t0 = lo + (hi - 1 - lo) / SEL_CHUNK * SEL_CHUNK; t0 >= lo; t0 -= SEL_CHUNK) {
        const int n = min(SEL_CHUNK, hi - t0);
        Stage stage;
        stage.load(B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, n, N, wide);
        __syncthreads();
        stage.put(bc);
        __syncthreads();
        constexpr int G = 4;
#pragma unroll 1
        for (int t = (n - 1) / G * G; t >= 0; t -= G) {
            float dl[G], e[G];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const int row = t0 + min(t + k, n - 1);
                dl[k] = ld_f32<T>(dt + row * c.ld_dt) + bias, e[k] = ld_f32<T>(dy + (size_t)row * c.channels);
                if (c.softplus) dl[k] = softplus_f(dl[k]);
                if (c.z) e[k] *= silu_v(ld_f32<T>(z + row * c.ld_z));
            }
#pragma unroll
            for (int k = G - 1; k >= 0; --k) {
                if (t + k >= n) continue;
                const float2 d2 = splat(dl[k]), e2 = splat(e[k]);
                steps += dl[k];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float4 v = bc[(t + k) * P + p];
                    const float2 arg = mul2(d2, A2[p]);
                    R[p] = mul2(make_float2(ex2a(arg.x), ex2a(arg.y)), fma2(e2, make_float2(v.z, v.w), R[p]));
                }
            }
        }
    }
    if (!me.in) return;
    float *o = sg.state + (size_t)blockIdx.x * N * c.channels + d;
#pragma unroll
    for (int n = 0; n < NP; ++n)
        if (n < N) o[(size_t)n * c.channels] = n & 1 ? R[n / 2].y : R[n / 2].x;
    sg.steps[(size_t)blockIdx.x * c.channels + d] = steps;
}

// The sums over blocks.  The first row_blocks blocks: dB and dC, a warp per token,
// from the channel tiles of each group; a token of no sequence gets zero gradients.
// The others: dA, dD and dbias over the slots, a thread per element.
template <typename T>
__global__ void __launch_bounds__(256) sel_bwd_sum(SelCall c, Parts parts, int slots, int tiles, int row_blocks) {
    const int N = c.dstate, G = c.groups;
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
#pragma unroll 4
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
#pragma unroll 8
        for (int i = 0; i < slots; ++i) s += parts.a[i * na + u];
        c.dA[u % c.channels * N + u / c.channels] = s;
    } else if (u < na + 2 * c.channels) {
        const long long v = u - na;
        float s = 0.f;
#pragma unroll 8
        for (int i = 0; i < slots; ++i) s += parts.d[(size_t)i * 2 * c.channels + v];
        float *o = v < c.channels ? c.dD : c.dbias;
        if (o) o[v < c.channels ? v : v - c.channels] = s;
    }
}

constexpr int BWD_WARPS_PER_SM = 12;

struct Layout {  // of the workspace, in floats
    int seg, slots, tiles;
    size_t bc, a, d, carried, steps, total;
    Layout(int tokens, int nseq, int channels, int groups, int N) {
        seg = choose_seg(tokens, nseq, channels, BWD_WARPS_PER_SM);
        slots = tokens > 0 ? seg_slots(tokens, nseq, seg) : 0;
        const int threads = N <= 32 ? 128 : 64;
        tiles = (channels / groups + threads - 1) / threads;
        bc = 0;
        a = bc + (size_t)groups * tiles * tokens * 2 * N;
        d = a + (size_t)slots * channels * N;
        carried = d + (size_t)slots * channels * 2;
        steps = carried + (seg == WHOLE ? 0 : (size_t)slots * channels * N);
        total = steps + (seg == WHOLE ? 0 : (size_t)slots * channels);
    }
};

template <typename T> cudaError_t run(const SelCall &c, float *ws, cudaStream_t st) {
    const size_t e = sizeof(T);
    const int per_group = c.channels / c.groups;
    const Layout l(c.seq.tokens, c.seq.nseq, c.channels, c.groups, c.dstate);
    const bool wide = rows_aligned(c.x, c.ld_x, e, 16) && rows_aligned(c.dt, c.ld_dt, e, 16) &&
                      (!c.z || rows_aligned(c.z, c.ld_z, e, 16)) && c.channels * e % 16 == 0 && per_group * e % 16 == 0;
    const bool wb = wide_bc(c);
    const Parts p{ws + l.bc, ws + l.a, ws + l.d};
    const Segments sg{l.seg, l.slots, ws + l.carried, ws + l.steps};
    if (c.seq.nseq > 0 && c.seq.tokens > 0) {
        const cudaError_t err = with_states(c.dstate, [&](auto np) {
            constexpr int TH = bwd_threads<np()>();
            const size_t smem = sizeof(BwdShared<T, np()>);
            cudaError_t r = cudaFuncSetAttribute(sel_bwd_kernel<T, np()>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (r == cudaSuccess && l.seg != WHOLE) {
                sel_carry_kernel<T, np()><<<dim3(l.slots, channel_tiles<CARRY_THREADS>(c)), CARRY_THREADS, 0, st>>>(c, sg, wb);
                r = cudaGetLastError();
                if (r == cudaSuccess) r = launch_sel_join(c, sg, true, st);
            }
            if (r != cudaSuccess) return r;
            sel_bwd_kernel<T, np()><<<dim3(l.slots, channel_tiles<TH>(c)), TH, smem, st>>>(c, sg, p, wide, wb);
            return cudaGetLastError();
        });
        if (err != cudaSuccess) return err;
    }
    const int row_blocks = (c.seq.tokens + 7) / 8, slots = c.seq.nseq > 0 ? l.slots : 0;
    const long long rest = ((long long)c.channels * (c.dstate + 2) + 255) / 256;
    sel_bwd_sum<T><<<(unsigned)(row_blocks + rest), 256, 0, st>>>(c, p, slots, l.tiles, row_blocks);
    return cudaGetLastError();
}

}  // namespace

size_t sel_bwd_workspace(int tokens, int nseq, int channels, int groups, int dstate) {
    return Layout(tokens, nseq, channels, groups, dstate).total * sizeof(float);
}

cudaError_t launch_sel_bwd(const SelCall &c, void *ws, cudaStream_t st) {
    return c.bf16 ? run<__nv_bfloat16>(c, static_cast<float *>(ws), st) : run<float>(c, static_cast<float *>(ws), st);
}

}  // namespace ssd
