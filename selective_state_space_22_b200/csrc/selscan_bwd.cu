// selscan_bwd.cu -- the gradient of the gated Mamba-1 scan on packed sequences.
//
// With a_t = exp(delta_t A), y = p silu(z), p = sum_n C h + D x and dp = dy silu(z):
//   g_t = dp_t C_t + G_{t+1},  G_t = a_t g_t     (the gradient at h_t, and what it hands back)
//   dC_t = sum_d dp_t h_t,  dB_t = sum_d delta_t x_t g_t          (over a group's channels)
//   du_t = sum_n g_t B_t,   q_t = G_t h_{t-1},  dA = sum_t delta_t q_t
//   ddelta_t = x_t du_t + sum_n A q_t,  dx_t = delta_t du_t + D dp_t,  dD = sum_t dp_t x_t
//   dz_t = dy_t p_t silu'(z_t),  ddt_t = ddelta_t softplus'(dt_t + bias),  dbias = sum_t ddt_t.
//
// A thread takes two channels and 8 states and walks its sequence (or segment,
// selscan_seg.cuh) backwards, in chunks of SEL_CHUNK tokens that start where the forward kept the states, and a chunk
// in two halves of SUB tokens.  For each half and state it runs the
// recurrence forwards (a_t and h_{t-1} stay in registers, so the backward walk takes no
// exponential) and then backwards, both channels in one packed operation; the second half
// starts from a state formed again from the first half's tokens, which costs half an
// exponential per state and token and halves the states to keep.
// dB and dC are summed over a warp's channels by matrix instructions (ChannelSum), over
// the block's warps in shared memory, and over blocks by sel_bwd_sum, all in a fixed
// order.  Bound by issue and latency: the registers of a half (step, input and upstream
// gradient of 4 tokens, three sums for each, a_t and h_{t-1}) leave 16 warps to an SM.
// Measured at 64 x 512 tokens, 1024 channels, 16 states, bf16: 1090 us, issue slots 53 % busy.
// Before the sums over channels took each product in two parts it was 990 us; then a form
// that split a chunk's tokens over the lanes of a warp took 1428 us, one with a channel per
// thread and its states paired 1490 us (each step, input and gradient held twice, spilled).
#include "selscan_seg.cuh"

namespace ssd {
namespace {

constexpr int SUB = GROUP, BWD_BLOCKS_PER_SM = 4;
static_assert(SEL_CHUNK == 2 * SUB, "a chunk is two halves");

// Sums over a warp's channels by matrix instructions: D[lane/4][c] += A[lane/4][k] B[k][c],
// where A holds four values of every lane as they are (k: the four lanes of a group, times
// two registers; two rows of A per group) and B is ones where k and c belong together.  An
// instruction thus adds each of the four values over the four lanes of a group; the
// sums of instruction i land in the lanes with lane%4 = i.  Four instructions (the
// gradients of B and C, four tokens each, of two states) fill D, and three shuffles that
// halve the values add the groups of a part (the lanes that hold the same states).
// Each value goes in as two tf32 parts, its first 11 bits and the next 11, so that it keeps
// 2^-22; the sums are float32.  bf16 io needs the second part as float32 io does: with the
// first alone dB and dC shrink by 3.5e-4, and by any amount where channels cancel (forward
// and gradient of 64 x 512 tokens, 1024 channels, bf16: 1268 us so, 1349 us with both).
// The zeros of B turn an infinite (or NaN) value into NaN sums of other tokens and states.
// `spoilt` sees that in the result, and the half's sums are then taken by shuffles.
template <int SPLIT> struct ChannelSum {
    static constexpr int GROUPS = 8 / SPLIT;  // of a part
    float d[4];
    __device__ __forceinline__ void clear() { d[0] = d[1] = d[2] = d[3] = 0.f; }
    static __device__ __forceinline__ void mma(float (&d)[4], const float (&v)[4], float b0, float b1) {
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
              "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
    }
    __device__ __forceinline__ void add(const float (&v)[4], int i, int lane) {
        const float b0 = (lane >> 2) == 2 * i ? 1.f : 0.f, b1 = (lane >> 2) == 2 * i + 1 ? 1.f : 0.f;
        float x[4], y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(__float_as_uint(v[k]) & 0xffffe000u), y[k] = v[k] - x[k];
        mma(d, x, b0, b1);
        mma(d, y, b0, b1);
    }
    __device__ __forceinline__ float spoilt(float so_far) const {  // NaN from the first sum on that is not finite, else zero
        return fmaf(d[0], 0.f, fmaf(d[1], 0.f, fmaf(d[2], 0.f, fmaf(d[3], 0.f, so_far))));
    }
    // Instruction lane%4's sums over the part: out(value, sum) for the values this lane
    // ends with.  d[0..3] are the group's sums of values 0, 2, 1, 3.
    template <typename F> __device__ __forceinline__ void finish(int lane, F &&out) const {
        auto half = [&](float a, float b, bool second, int mask) {  // the kept one, with the other lane's added
            return (second ? b : a) + __shfl_xor_sync(0xffffffffu, second ? a : b, mask);
        };
        constexpr int top = GROUPS == 8 ? 16 : GROUPS == 4 ? 8 : 4;
        const bool odd = lane & top;  // keeps values 1 and 3
        const float a = half(d[0], d[2], odd, top), b = half(d[1], d[3], odd, top);
        if constexpr (GROUPS == 2) {
            out(odd ? 1 : 0, a), out(odd ? 3 : 2, b);
        } else {
            const bool upper = lane & (top / 2);
            float s = half(a, b, upper, top / 2);
            if (GROUPS == 8) s += __shfl_xor_sync(0xffffffffu, s, 4);
            if (GROUPS == 4 || !(lane & 4)) out((odd ? 1 : 0) + (upper ? 2 : 0), s);
        }
    }
};

template <typename T, int NP> struct BwdShared {
    static constexpr int NS = Lanes<NP>::NS, WARPS = SCAN_THREADS / 32, CH = WARPS * Lanes<NP>::CH;
    T x[SEL_CHUNK][CH], dt[SEL_CHUNK][CH], z[SEL_CHUNK][CH], dy[SEL_CHUNK][CH];
    float4 bc[SEL_CHUNK * NP];
    float2 A2[NS][SCAN_THREADS], G[NS][SCAN_THREADS], dA[NS][SCAN_THREADS];
    // the states before the chunk and before its second half; once a state of a half has been
    // read for the last time, hm keeps the G that it met
    float2 h0[NS][SCAN_THREADS], hm[NS][SCAN_THREADS];
    float part[WARPS][SUB][2][NP];                      // a warp's sums: [token][dB, dC][state]
};

struct Parts {   // workspace
    float *bc;   // [channel tiles][tokens][2][dstate]
    float *a;    // [slots][dstate][channels]
    float *d;    // [slots][2][channels]: dD, dbias
};

template <typename T, int NP>
__global__ void __launch_bounds__(SCAN_THREADS, BWD_BLOCKS_PER_SM) sel_bwd_kernel(SelCall c, Segments sg, Parts parts, Access ok) {
    using Sh = BwdShared<T, NP>;
    using L = Lanes<NP>;
    constexpr int NS = L::NS, SPLIT = L::SPLIT, PAIRS = L::PAIRS, CH = Sh::CH, OWN = SUB / SPLIT;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Sh &sh = *reinterpret_cast<Sh *>(smem_raw);
    const Mine me = my_channels<NP>(c, blockIdx.y);
    const int N = c.dstate, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = lane / PAIRS, pair = lane % PAIRS;
    auto state_of = [&](int k) { return k * SPLIT + part; };  // neighbours at the same time: A = -1, -2, .. are alike then
    const int ch = 2 * (warp * PAIRS + pair);  // of the block's
    const size_t step = (size_t)N * c.channels;
    float *const pa = parts.a + blockIdx.x * step, *const pdd = parts.d + (size_t)blockIdx.x * 2 * c.channels;
    const float2 zero = make_float2(0.f, 0.f);
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end)) {  // the same for the whole block
        for (int k = 0; k < NS; ++k)
            if (state_of(k) < N) store_two<float>(pa + (size_t)state_of(k) * c.channels, zero, me, ok.state);
        if (part == 0) store_two<float>(pdd, zero, me, ok.state), store_two<float>(pdd + c.channels, zero, me, ok.state);
        return;
    }
    const int per_group = c.channels / c.groups, tiles = (per_group + CH - 1) / CH;
    const int t_first = me.group * per_group + blockIdx.y % tiles * CH, t_cols = min(CH, (me.group + 1) * per_group - t_first);
    const float2 bias = c.dt_bias ? make_float2(c.dt_bias[me.c0], c.dt_bias[me.c1]) : zero;
    const float2 D = c.D ? make_float2(c.D[me.c0], c.D[me.c1]) : zero;
    for (int k = 0; k < NS; ++k) {
        const int n = state_of(k);
        float2 A2 = zero, G = zero;
        if (n < N) {
            A2 = make_float2(rate(c.A[(size_t)me.c0 * N + n]), rate(c.A[(size_t)me.c1 * N + n]));
            const float *from = sg.state + blockIdx.x * step + (size_t)n * c.channels;
            if (sg.seg != WHOLE) G = make_float2(from[me.c0], from[me.c1]);
        }
        sh.A2[k][tid] = A2, sh.G[k][tid] = G, sh.dA[k][tid] = sh.h0[k][tid] = zero;
    }
    float2 dD = zero, dbias = zero;
    StageBC<T, NP, SEL_CHUNK, true> stage;
    const T *B = static_cast<const T *>(c.B) + me.group * N, *C = static_cast<const T *>(c.C) + me.group * N;
    const int c_first = (lo - first) / SEL_CHUNK, c_last = (hi - 1 - first) / SEL_CHUNK;
    const float *kept = c.chunk_states + (size_t)(first / SEL_CHUNK + i) * step;
    {
        const int t0 = first + c_last * SEL_CHUNK;
        stage.load(B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, min(SEL_CHUNK, hi - t0), N, ok.bc);
    }
    for (int chunk = c_last; chunk >= c_first; --chunk) {
        const int t0 = first + chunk * SEL_CHUNK, n = min(SEL_CHUNK, hi - t0);
        __syncthreads();  // the chunk before has been read
        const RowsOf<T, CH> rows[4] = {{sh.x, static_cast<const T *>(c.x) + t0 * c.ld_x + t_first, c.ld_x},
                                       {sh.dt, static_cast<const T *>(c.dt) + t0 * c.ld_dt + t_first, c.ld_dt},
                                       {sh.dy, static_cast<const T *>(c.dy) + (size_t)t0 * c.channels + t_first, c.channels},
                                       {sh.z, static_cast<const T *>(c.z) + (c.z ? t0 * c.ld_z + t_first : 0), c.ld_z}};
        fetch_rows(rows, c.z ? 4 : 3, n, t_cols, ok.wide, ok.paired);
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            if (state_of(k) >= N) continue;
            const float *from = kept + chunk * step + (size_t)state_of(k) * c.channels;
            if (ok.state) {
                cp8(&sh.h0[k][tid], from + me.c0);
            } else {
                cp4(&sh.h0[k][tid].x, from + me.c0);
                cp4(&sh.h0[k][tid].y, from + me.c1);
            }
        }
        stage.put(sh.bc);
        if (chunk > c_first) {
            const int tp = t0 - SEL_CHUNK;
            stage.load(B + tp * c.ld_b, c.ld_b, C + tp * c.ld_c, c.ld_c, SEL_CHUNK, N, ok.bc);
        }
        cp_wait_all();
        __syncthreads();

        // Row r of a tile for this thread's channels.  Tokens past the end, and channels
        // that the thread has not got (whose places were never written), read as zero.
        auto two = [&](T(*tile)[CH], int r) {
            const float2 v = reinterpret_cast<const Two<T> *>(&tile[r][ch])->f();
            return make_float2(r < n && me.has > 0 ? v.x : 0.f, r < n && me.has > 1 ? v.y : 0.f);
        };
        auto step_of = [&](int r) {
            const float2 v = add2(two(sh.dt, r), bias), s = c.softplus ? softplus2(v) : v;
            return make_float2(r < n && me.has > 0 ? s.x : 0.f, r < n && me.has > 1 ? s.y : 0.f);
        };
        // v[j], which every lane has for its own tokens, to all lanes of the pair: w[token]
        auto spread = [&](const float2 (&v)[OWN], float2 (&w)[SUB]) {
#pragma unroll
            for (int k = 0; k < SUB; ++k) w[k] = SPLIT == 1 ? v[k / SPLIT] : shfl2(v[k / SPLIT], pair + k % SPLIT * PAIRS);
        };
        float2 dl[SUB], u2[SUB], own_dl[OWN], own[OWN];
        float most;  // the lane's largest step
        // a[k] = exp(delta_k A). Decays near one, where the whole warp has them, by the
        // polynomial: the gradient of the state adds up many of their errors (dA 1.2e-6 off
        // with the approximate exponential everywhere, 6.3e-7 so, at 32 sequences of 512
        // tokens; 64 of them took 907 us so, 990 us with it). The state before a second half is four
        // tokens away from one that was kept, and does without.
        auto decays = [&](float2 A2, float2 (&a)[SUB]) {
            if (__all_sync(0xffffffffu, most * fmaxf(fabsf(A2.x), fabsf(A2.y)) <= SMALL_EXP)) {
#pragma unroll
                for (int k = 0; k < SUB; ++k) a[k] = ex2_small(mul2(dl[k], A2));
            } else {
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const float2 x = mul2(dl[k], A2);
                    a[k] = make_float2(ex2a(x.x), ex2a(x.y));
                }
            }
        };
        auto steps_of_half = [&](int k0) {
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int r = k0 + j * SPLIT + part;
                own_dl[j] = step_of(r);
                own[j] = mul2(own_dl[j], two(sh.x, r));
            }
            spread(own_dl, dl);
            spread(own, u2);
            most = 0.f;
#pragma unroll
            for (int k = 0; k < SUB; ++k) most = fmaxf(most, fmaxf(fabsf(dl[k].x), fabsf(dl[k].y)));
        };
        if (n > SUB) {  // the state before the second half
            steps_of_half(0);
#pragma unroll 2
            for (int s = 0; s < NS; ++s) {
                const float2 A2 = sh.A2[s][tid];
                float2 h = sh.h0[s][tid];
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const float2 b = *reinterpret_cast<const float2 *>(sh.bc + k * NP + state_of(s)), arg = mul2(dl[k], A2);
                    h = fma2(make_float2(ex2a(arg.x), ex2a(arg.y)), h, mul2(u2[k], b));
                }
                sh.hm[s][tid] = h;
            }
        }
        for (int half = n > SUB ? 1 : 0; half >= 0; --half) {
            const int k0 = half * SUB;
            float2 dp[SUB], du[SUB], sd[SUB], pre[SUB];
            steps_of_half(k0);
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int r = k0 + j * SPLIT + part;
                own[j] = two(sh.dy, r);
                if (c.z) own[j] = mul2(own[j], silu2(two(sh.z, r)));
            }
            spread(own, dp);
#pragma unroll
            for (int k = 0; k < SUB; ++k) du[k] = sd[k] = pre[k] = zero;
            const float2(*const h_from)[SCAN_THREADS] = half ? sh.hm : sh.h0;
            float spoilt = 0.f;
#pragma unroll 1
            for (int s2 = 0; s2 < NS; s2 += 2) {
                ChannelSum<SPLIT> sums;
                sums.clear();
#pragma unroll
                for (int s = s2; s < s2 + 2; ++s) {
                    const float2 A2 = sh.A2[s][tid];
                    float2 h = h_from[s][tid], a[SUB], hp[SUB];
                    float v[SUB];
                    const float4 *q = sh.bc + k0 * NP + state_of(s);
                    decays(A2, a);
#pragma unroll
                    for (int k = 0; k < SUB; ++k) {
                        const float4 bc = q[k * NP];
                        hp[k] = h;
                        h = fma2(a[k], h, mul2(u2[k], make_float2(bc.x, bc.y)));
                        pre[k] = fma2(make_float2(bc.z, bc.w), h, pre[k]);
                        const float2 e = mul2(dp[k], h);
                        v[k] = e.x + e.y;
                    }
                    sums.add(v, 2 * (s - s2) + 1, lane);
                    const float2 G0 = sh.G[s][tid];  // kept below (a store here cost 6 to 12 % in float32 and at 64 states)
                    float2 G = G0, dA = make_float2(0.f, 0.f);  // of these tokens: one addition to the long sum
#pragma unroll
                    for (int k = SUB - 1; k >= 0; --k) {
                        const float4 bc = q[k * NP];
                        const float2 g = fma2(dp[k], make_float2(bc.z, bc.w), G);
                        G = mul2(a[k], g);
                        const float2 qq = mul2(G, hp[k]);
                        du[k] = fma2(g, make_float2(bc.x, bc.y), du[k]);
                        sd[k] = fma2(A2, qq, sd[k]);
                        dA = fma2(dl[k], qq, dA);
                        const float2 e = mul2(u2[k], g);
                        v[k] = e.x + e.y;
                    }
                    sh.G[s][tid] = G, sh.hm[s][tid] = G0, sh.dA[s][tid] = add2(sh.dA[s][tid], dA);
                    sums.add(v, 2 * (s - s2), lane);
                }
                spoilt = sums.spoilt(spoilt);
                const int which = lane & 1, state = state_of(s2 + ((lane >> 1) & 1));  // what instruction lane%4 summed
                sums.finish(lane, [&](int token, float sum) { sh.part[warp][token][which][state] = sum; });
            }
            if (__any_sync(0xffffffffu, spoilt != 0.f)) {
                // The half again for its sums of dB and dC (and of dA where it holds tokens past
                // the end, whose states count for nothing; it is the first half taken then).
                float2 dl0[SUB], u0[SUB], e[OWN];
#pragma unroll
                for (int j = 0; j < OWN; ++j) e[j] = own[j];
                steps_of_half(0);
#pragma unroll
                for (int k = 0; k < SUB; ++k) dl0[k] = dl[k], u0[k] = u2[k];
                steps_of_half(k0);
#pragma unroll
                for (int j = 0; j < OWN; ++j) own[j] = e[j];
#pragma unroll 1
                for (int s = 0; s < NS; ++s) {
                    const float2 A2 = sh.A2[s][tid];
                    float2 h = sh.h0[s][tid], G = sh.hm[s][tid], a[SUB], hp[SUB], dA = zero;
                    auto put = [&](int token, int which, float2 v2) {
                        float v = v2.x + v2.y;
#pragma unroll
                        for (int o = 1; o < PAIRS; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                        if (pair == 0) sh.part[warp][token][which][state_of(s)] = v;
                    };
                    auto bc = [&](int token) { return sh.bc[token * NP + state_of(s)]; };
                    if (half)
#pragma unroll
                        for (int k = 0; k < SUB; ++k) {
                            const float2 arg = mul2(dl0[k], A2);
                            h = fma2(make_float2(ex2a(arg.x), ex2a(arg.y)), h, mul2(u0[k], make_float2(bc(k).x, bc(k).y)));
                        }
                    decays(A2, a);
#pragma unroll
                    for (int k = 0; k < SUB; ++k) {
                        hp[k] = h;
                        h = fma2(a[k], h, mul2(u2[k], make_float2(bc(k0 + k).x, bc(k0 + k).y)));
                        put(k, 1, mul2(dp[k], h));
                    }
#pragma unroll
                    for (int k = SUB - 1; k >= 0; --k) {
                        const float2 g = fma2(dp[k], make_float2(bc(k0 + k).z, bc(k0 + k).w), G);
                        G = mul2(a[k], g);
                        if (k0 + k < n) dA = fma2(dl[k], mul2(G, hp[k]), dA);
                        put(k, 0, mul2(u2[k], g));
                    }
                    if (k0 + SUB > n) sh.dA[s][tid] = dA;
                }
            }
            sum_parts<SPLIT>(du, part);
            sum_parts<SPLIT>(sd, part);
            if (c.z) sum_parts<SPLIT>(pre, part);
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int r = k0 + j * SPLIT + part;
                const float2 xv = two(sh.x, r), dyv = two(sh.dy, r), e = own[j];
                float2 ddt = fma2(xv, du[j], mul2(sd[j], splat(0.6931471805599453f)));  // A was scaled by log2 e
                if (c.softplus) ddt = mul2(ddt, sigmoid2(add2(two(sh.dt, r), bias)));
                if (r < n) {
                    const size_t o = (size_t)(t0 + r) * c.channels;
                    store_two<T>(static_cast<T *>(c.dx) + o, fma2(own_dl[j], du[j], mul2(D, e)), me, ok.paired);
                    store_two<T>(static_cast<T *>(c.ddt) + o, ddt, me, ok.paired);
                    dD = fma2(e, xv, dD);
                    dbias = add2(dbias, ddt);
                    if (c.z) {
                        const float2 zv = two(sh.z, r), s = sigmoid2(zv), p = fma2(D, xv, pre[j]);
                        const float2 one = splat(1.f), slope = mul2(s, fma2(zv, fma2(s, splat(-1.f), one), one));  // silu'
                        store_two<T>(static_cast<T *>(c.dz) + o, mul2(mul2(dyv, p), slope), me, ok.paired);
                    }
                }
            }
            __syncthreads();  // every warp's sums are there
            for (int u = tid; u < SUB * 2 * NP; u += SCAN_THREADS) {
                const int t = u / (2 * NP), k = u % (2 * NP), s = k % NP;
                float v = (&sh.part[0][0][0][0])[u];
#pragma unroll
                for (int w = 1; w < Sh::WARPS; ++w) v += (&sh.part[w][0][0][0])[u];
                if (s < N && k0 + t < n) parts.bc[((size_t)blockIdx.y * c.seq.tokens + t0 + k0 + t) * 2 * N + (k / NP) * N + s] = v;
            }
            __syncthreads();  // before the other half's
        }
    }
    for (int k = 0; k < NS; ++k)
        if (state_of(k) < N) store_two<float>(pa + (size_t)state_of(k) * c.channels, sh.dA[k][tid], me, ok.state);
#pragma unroll
    for (int o = PAIRS; o < 32; o *= 2) {
        dD = add2(dD, make_float2(__shfl_xor_sync(0xffffffffu, dD.x, o), __shfl_xor_sync(0xffffffffu, dD.y, o)));
        dbias = add2(dbias, make_float2(__shfl_xor_sync(0xffffffffu, dbias.x, o), __shfl_xor_sync(0xffffffffu, dbias.y, o)));
    }
    if (part == 0) store_two<float>(pdd, dD, me, ok.state), store_two<float>(pdd + c.channels, dbias, me, ok.state);
}

// What a segment hands back when nothing comes from behind it, and its sum of steps: for
// sel_join.  The first segment of a sequence hands back to nobody.
template <typename T, int NP>
__global__ void __launch_bounds__(SCAN_THREADS) sel_carry_kernel(SelCall c, Segments sg, Access ok) {
    using L = Lanes<NP>;
    constexpr int NS = L::NS, SPLIT = L::SPLIT, PAIRS = L::PAIRS, OWN = GROUP / SPLIT;
    using Stage = StageBC<T, NP, SEL_CHUNK, true>;
    __shared__ __align__(16) float4 bc[SEL_CHUNK * NP];
    int i, first, lo, hi, end;
    if (!segment(c.seq, sg.seg, blockIdx.x, i, first, lo, hi, end) || lo == first) return;
    const Mine me = my_channels<NP>(c, blockIdx.y);
    const int N = c.dstate, lane = threadIdx.x & 31, part = lane / PAIRS, pair = lane % PAIRS;
    auto state_of = [&](int k) { return k * SPLIT + part; };
    const T *B = static_cast<const T *>(c.B) + me.group * N, *C = static_cast<const T *>(c.C) + me.group * N;
    const T *dt = static_cast<const T *>(c.dt), *z = static_cast<const T *>(c.z), *dy = static_cast<const T *>(c.dy);
    float2 A2[NS], R[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int n = min(state_of(k), N - 1);
        A2[k] = make_float2(rate(c.A[(size_t)me.c0 * N + n]), rate(c.A[(size_t)me.c1 * N + n]));
        R[k] = make_float2(0.f, 0.f);
    }
    const float2 bias = c.dt_bias ? make_float2(c.dt_bias[me.c0], c.dt_bias[me.c1]) : make_float2(0.f, 0.f);
    float2 steps = make_float2(0.f, 0.f);
    // A group of tokens at a time, the next one's rows and the next chunk's B and C on their
    // way (without, the kernel took 216 us, 91 us so, for 5925 tokens of 1658
    // channels of 4 states).
    Two<T> nd[OWN], ny[OWN], nz[OWN];
    auto fetch = [&](int g) {
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const int row = min(lo + g * GROUP + j * SPLIT + part, hi - 1);
            nd[j] = load_two(dt + row * c.ld_dt, me, ok.paired);
            ny[j] = load_two(dy + (size_t)row * c.channels, me, ok.paired);
            if (c.z) nz[j] = load_two(z + row * c.ld_z, me, ok.paired);
        }
    };
    Stage stage;
    auto load_bc = [&](int chunk) {
        const int t0 = lo + chunk * SEL_CHUNK;
        stage.load(B + t0 * c.ld_b, c.ld_b, C + t0 * c.ld_c, c.ld_c, min(SEL_CHUNK, hi - t0), N, ok.bc);
    };
    constexpr int GROUPS = SEL_CHUNK / GROUP;
    const int last = (hi - 1 - lo) / GROUP;
    load_bc(last / GROUPS);
    fetch(last);
#pragma unroll 1
    for (int g = last, staged = -1; g >= 0; --g) {
        if (g / GROUPS != staged) {
            staged = g / GROUPS;
            __syncthreads();  // the chunk behind has been read
            stage.put(bc);
            __syncthreads();
            if (staged > 0) load_bc(staged - 1);
        }
        float2 dl[OWN], e[OWN], d2[GROUP], e2[GROUP];
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            dl[j] = add2(nd[j].f(), bias);
            e[j] = ny[j].f();
            if (c.softplus) dl[j] = softplus2(dl[j]);
            if (c.z) e[j] = mul2(e[j], silu2(nz[j].f()));
            if (lo + g * GROUP + j * SPLIT + part >= hi) dl[j] = e[j] = make_float2(0.f, 0.f);
            steps = add2(steps, dl[j]);
        }
        if (g > 0) fetch(g - 1);
#pragma unroll
        for (int k = 0; k < GROUP; ++k) {
            const int from = pair + k % SPLIT * PAIRS;
            d2[k] = SPLIT == 1 ? dl[k / SPLIT] : shfl2(dl[k / SPLIT], from);
            e2[k] = SPLIT == 1 ? e[k / SPLIT] : shfl2(e[k / SPLIT], from);
            most = fmaxf(most, fmaxf(fabsf(d2[k].x), fabsf(d2[k].y)));
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            float2 a[GROUP];
            if (__all_sync(0xffffffffu, most * fmaxf(fabsf(A2[s].x), fabsf(A2[s].y)) <= SMALL_EXP)) {
#pragma unroll
                for (int k = 0; k < GROUP; ++k) a[k] = ex2_small(mul2(d2[k], A2[s]));
            } else {
#pragma unroll
                for (int k = 0; k < GROUP; ++k) {
                    const float2 x = mul2(d2[k], A2[s]);
                    a[k] = make_float2(ex2a(x.x), ex2a(x.y));
                }
            }
#pragma unroll
            for (int k = GROUP - 1; k >= 0; --k) {
                const float4 v = bc[(g % GROUPS * GROUP + k) * NP + state_of(s)];
                R[s] = mul2(a[k], fma2(e2[k], make_float2(v.z, v.w), R[s]));
            }
        }
    }
    float *o = sg.state + (size_t)blockIdx.x * N * c.channels;
#pragma unroll
    for (int k = 0; k < NS; ++k)
        if (state_of(k) < N) store_two<float>(o + (size_t)state_of(k) * c.channels, R[k], me, ok.state);
#pragma unroll
    for (int k = PAIRS; k < 32; k *= 2)
        steps = add2(steps, make_float2(__shfl_xor_sync(0xffffffffu, steps.x, k), __shfl_xor_sync(0xffffffffu, steps.y, k)));
    if (part == 0) store_two<float>(sg.steps + (size_t)blockIdx.x * c.channels, steps, me, ok.state);
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
        double s = 0.;
#pragma unroll 8
        for (int i = 0; i < slots; ++i) s += parts.a[i * na + u];
        c.dA[u % c.channels * N + u / c.channels] = (float)s;
    } else if (u < na + 2 * c.channels) {
        const long long v = u - na;
        double s = 0.;
#pragma unroll 8
        for (int i = 0; i < slots; ++i) s += parts.d[(size_t)i * 2 * c.channels + v];
        float *o = v < c.channels ? c.dD : c.dbias;
        if (o) o[v < c.channels ? v : v - c.channels] = (float)s;
    }
}

// Warps counted as of 32 channels (64 of up to 8 states): counting the 16 that 32 and 64
// states have cuts less, and took 6 to 12 % more at 4096 tokens of 1024 channels.
constexpr int BWD_WARPS_PER_SM = 16;

struct Layout {  // of the workspace, in floats
    int seg, slots, tiles;
    size_t bc, a, d, carried, steps, total;
    Layout(int tokens, int nseq, int channels, int groups, int N) {
        const int split = N <= 8 ? 1 : N <= 16 ? 2 : 4, ch = 2 * SCAN_THREADS / split;  // as Lanes
        seg = choose_seg(tokens, nseq, channels, split == 1 ? 64 : 32, BWD_WARPS_PER_SM);
        slots = tokens > 0 ? seg_slots(tokens, nseq, seg) : 0;
        tiles = (channels / groups + ch - 1) / ch;
        bc = 0;
        a = bc + (size_t)groups * tiles * tokens * 2 * N;
        d = a + (size_t)slots * channels * N;
        carried = d + (size_t)slots * channels * 2;
        steps = carried + (seg == WHOLE ? 0 : (size_t)slots * channels * N);
        total = steps + (seg == WHOLE ? 0 : (size_t)slots * channels);
    }
};

template <typename T> cudaError_t run(const SelCall &c, float *ws, cudaStream_t st) {
    const Layout l(c.seq.tokens, c.seq.nseq, c.channels, c.groups, c.dstate);
    const Parts p{ws + l.bc, ws + l.a, ws + l.d};
    const Segments sg{l.seg, l.slots, ws + l.carried, ws + l.steps};
    const Access ok(c);
    if (c.seq.nseq > 0 && c.seq.tokens > 0) {
        const cudaError_t err = with_states(c.dstate, [&](auto np) {
            const dim3 grid(l.slots, channel_tiles<np()>(c));
            constexpr size_t smem = sizeof(BwdShared<T, np()>);
            cudaError_t r = cudaSuccess;
            if (smem > 48 << 10) r = cudaFuncSetAttribute(sel_bwd_kernel<T, np()>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (r == cudaSuccess && l.seg != WHOLE) {
                sel_carry_kernel<T, np()><<<grid, SCAN_THREADS, 0, st>>>(c, sg, ok);
                r = cudaGetLastError();
                if (r == cudaSuccess) r = launch_sel_join(c, sg, true, st);
            }
            if (r != cudaSuccess) return r;
            sel_bwd_kernel<T, np()><<<grid, SCAN_THREADS, smem, st>>>(c, sg, p, ok);
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
