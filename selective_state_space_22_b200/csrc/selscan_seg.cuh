// selscan_seg.cuh -- what the forward and backward selective scans share: the cut of
// sequences into segments, the staging of B and C, and the join of segments.
//
// A thread walks the recurrence of some states of a channel (backwards: of two channels),
// two values in the halves of a float2, so that every operation but the exponential is a
// packed one; the lanes that share a channel's states take turns at the work per channel
// and token (step size, gate).  Where the
// (sequence, channel) pairs do not fill the GPU, sequences are cut into segments of
// `seg` tokens: a first pass runs every segment but a sequence's last from zero and
// keeps its end state and its sum of steps, sel_join carries the states from segment
// to segment, and the full pass then starts each segment from its state.
//
// Segment j of sequence i is slot cu[i] / seg + i + j: slots of different sequences
// never meet, and tokens / seg + nseq of them hold every call.
#pragma once

#include <type_traits>

#include "mixer.cuh"

namespace ssd {

constexpr int WHOLE = 1 << 30;  // seg: sequences are not cut, slot = sequence

struct Segments {
    int seg, slots;
    float *state;   // [slots][dstate][channels]: end state (or carried gradient) from zero, then the one to start from
    float *steps;   // [slots][channels]: sum of delta
};

inline int seg_slots(int tokens, int nseq, int seg) { return seg == WHOLE ? nseq : tokens / seg + nseq; }

// The cut, of `per_warp` channels to a warp: none once there are half of `warps_per_sm`
// warps for each SM, else segments so short that there are all, but of 32 tokens at least
// (a multiple of 16, so that kept states fall on segment starts).  8 x 256 tokens of 256
// channels, forward and gradient, 16 states: 159 us with 64 at least, 105 us with 32, 87 us
// with 16, which takes 8 % more for one sequence of 4096 tokens.
inline int choose_seg(int tokens, int nseq, int channels, int per_warp, int warps_per_sm) {
    const long long want = 148LL * warps_per_sm, per_token = (channels + per_warp - 1) / per_warp;
    if (nseq * per_token * 2 >= want) return WHOLE;
    const long long seg = (tokens * per_token / want + 15) / 16 * 16;
    return seg < 32 ? 32 : (int)seg;
}

// What slot s stands for: false when it is no segment.
__device__ __forceinline__ bool segment(const Packed &p, int seg, int s, int &i, int &first, int &lo, int &hi, int &end) {
    if (seg == WHOLE) {
        i = s;
        if (!seq_rows(p, i, lo, end)) return false;
        first = lo, hi = end;
        return lo < end;
    }
    int a = 0, b = p.nseq;  // the last sequence whose slots start at or before s
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (p.cu[m] / seg + m <= s) a = m; else b = m;
    }
    i = a;
    if (!seq_rows(p, i, first, end)) return false;
    const int j = s - (first / seg + i);
    if (j < 0 || (long long)first + (long long)j * seg >= end) return false;
    lo = first + j * seg;
    hi = min(lo + seg, end);
    return true;
}

// Backwards, how dstate (padded to NP) states are shared out: NS to a lane, SPLIT <= 4
// lanes to a channel pair, lane = pair + PAIRS * part.  GROUP tokens are taken at a time, so that
// each lane has a whole number of them to prepare.
constexpr int GROUP = 4;
template <int NP> struct Lanes {
    static constexpr int NS = NP < 8 ? NP : NP <= 32 ? 8 : 16, SPLIT = NP / NS, PAIRS = 32 / SPLIT, CH = 64 / SPLIT;  // CH: channels of a warp
};
constexpr int SCAN_THREADS = 128;  // of a block: 64 measured 10 % more at 64 x 512 tokens (B and C staged for fewer channels), 256 7 %

__device__ __forceinline__ void cp16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp8(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp4(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// n rows of `cols` channels of K tensors into their tiles [..][CH]: by asynchronous copies
// of 16 or 4 bytes where rows divide into them (they land by cp_wait_all), else through
// registers, four rows' elements of all tensors on their way at a time.  (An element at a
// time through registers, 19 sequences of 753 tokens, 1565 channels of 8 states in float32
// took 366 us, 203 us so.)
template <typename T, int CH> struct RowsOf {
    T (*to)[CH];
    const T *src;
    long long ld;
};
template <int BYTES, typename T, int CH, int K>
__device__ __forceinline__ void copy_rows(const RowsOf<T, CH> (&a)[K], int used, int n, int cols) {
    constexpr int E = BYTES / (int)sizeof(T), PER = CH / E;
#pragma unroll
    for (int q = 0; q < K; ++q) {
        if (q >= used) break;
#pragma unroll 2
        for (int u = threadIdx.x; u < n * PER; u += SCAN_THREADS) {
            const int r = u / PER, k = u % PER * E;
            if (k >= cols) continue;
            if constexpr (BYTES == 16) cp16(&a[q].to[r][k], a[q].src + r * a[q].ld + k);
            if constexpr (BYTES == 4) cp4(&a[q].to[r][k], a[q].src + r * a[q].ld + k);
        }
    }
}
template <typename T, int CH, int K>
__device__ __forceinline__ void fetch_rows(const RowsOf<T, CH> (&a)[K], int used, int n, int cols, bool wide, bool paired) {
    if (wide) {
        copy_rows<16>(a, used, n, cols);
    } else if (sizeof(T) == 4 || paired) {
        copy_rows<4>(a, used, n, cols);
    } else {
        constexpr int U = 2;
        for (int u0 = threadIdx.x; u0 < n * CH; u0 += U * SCAN_THREADS) {
            T v[K][U];
#pragma unroll
            for (int q = 0; q < K; ++q)
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int u = u0 + j * SCAN_THREADS, r = u / CH, k = u % CH;
                    if (q < used && r < n && k < cols) v[q][j] = a[q].src[r * a[q].ld + k];
                }
#pragma unroll
            for (int q = 0; q < K; ++q)
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int u = u0 + j * SCAN_THREADS, r = u / CH, k = u % CH;
                    if (q < used && r < n && k < cols) a[q].to[r][k] = v[q][j];
                }
        }
    }
}

// B and C of TT tokens in shared memory, for 16-byte reads that are the same for all
// lanes with those states: of token t, states 2 p and 2 p + 1 as (B, B', C, C'), or with
// TWICE state n as (B, B, C, C) for two channels at once.
// Fetched a run ahead: `load` takes the rows into registers as they lie in
// memory, `put` writes them out once the buffer is free.  Tokens past the run's end and
// states past N are zero.
template <typename T, int NP, int TT, bool TWICE> struct StageBC {
    static constexpr int QUADS = TT * NP / 4, PER = (QUADS + SCAN_THREADS - 1) / SCAN_THREADS;  // of B, and of C
    struct alignas(4 * sizeof(T)) Quad {
        T v[4];
    };
    Quad b[PER], c[PER];
    static __device__ __forceinline__ Quad get(const T *p, int left, bool wide) {
        Quad q;
        if (wide) {
            if (left > 0) return *reinterpret_cast<const Quad *>(p);
            left = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) st_f32<T>(&q.v[i], i < left ? ld_f32<T>(p + i) : 0.f);
        return q;
    }
    // n tokens from row 0 of B and C; wide: rows are aligned vectors of four and N a multiple of 4
    __device__ __forceinline__ void load(const T *B, long long lb, const T *C, long long lc, int n, int N, bool wide) {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int at = u * SCAN_THREADS + threadIdx.x, t = at / (NP / 4), s = at % (NP / 4) * 4;
            const int left = t < n && at < QUADS ? N - s : 0;
            b[u] = get(B + (left > 0 ? t * lb + s : 0), left, wide);
            c[u] = get(C + (left > 0 ? t * lc + s : 0), left, wide);
        }
    }
    __device__ __forceinline__ void put(float4 *to) const {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int at = u * SCAN_THREADS + threadIdx.x;
            if (at >= QUADS) break;
            float fb[4], fc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fb[i] = ld_f32<T>(&b[u].v[i]), fc[i] = ld_f32<T>(&c[u].v[i]);
            if constexpr (TWICE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) to[4 * at + i] = make_float4(fb[i], fb[i], fc[i], fc[i]);
            } else {
                to[2 * at] = make_float4(fb[0], fb[1], fc[0], fc[1]);
                to[2 * at + 1] = make_float4(fb[2], fb[3], fc[2], fc[3]);
            }
        }
    }
};

// A thread's channel pair: its first channel, the second (the first again where the
// group ends), and how many of the two it has (0 to 2).
struct Mine {
    int group, c0, c1, has;
};
template <int NP> __device__ __forceinline__ Mine my_channels(const SelCall &c, int tile) {
    using L = Lanes<NP>;
    constexpr int CH = SCAN_THREADS / 32 * L::CH;  // channels of a block
    const int per_group = c.channels / c.groups, tiles = (per_group + CH - 1) / CH, g = tile / tiles;
    const int k = tile % tiles * CH + 2 * ((threadIdx.x >> 5) * L::PAIRS + (threadIdx.x & 31) % L::PAIRS);
    const int first = min(k, (per_group - 1) & ~1);  // threads past the group follow along on its last pair
    return {g, g * per_group + first, g * per_group + min(first + 1, per_group - 1), max(0, min(2, per_group - k))};
}
template <int NP> inline int channel_tiles(const SelCall &c) {
    constexpr int CH = SCAN_THREADS / 32 * Lanes<NP>::CH;
    return c.groups * ((c.channels / c.groups + CH - 1) / CH);
}

// Two neighbouring values of a row.  paired: one aligned access.
template <typename T> struct alignas(2 * sizeof(T)) Two {
    T a, b;
    __device__ __forceinline__ float2 f() const { return make_float2(ld_f32<T>(&a), ld_f32<T>(&b)); }
};
template <typename T> __device__ __forceinline__ Two<T> load_two(const T *row, const Mine &me, bool paired) {
    if (paired) return *reinterpret_cast<const Two<T> *>(row + me.c0);
    return {row[me.c0], row[me.c1]};
}
template <typename T> __device__ __forceinline__ void store_two(T *row, float2 v, const Mine &me, bool paired) {
    Two<T> t;
    st_f32<T>(&t.a, v.x), st_f32<T>(&t.b, v.y);
    if (paired) {
        if (me.has) *reinterpret_cast<Two<T> *>(row + me.c0) = t;
    } else {
        if (me.has > 0) row[me.c0] = t.a;
        if (me.has > 1) row[me.c1] = t.b;
    }
}
__device__ __forceinline__ float2 shfl2(float2 v, int lane) {
    return make_float2(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane));
}
// v[k] summed over the SPLIT lanes of a channel pair: a lane of part s ends with token
// j SPLIT + s in v[j].
template <int SPLIT, int K> __device__ __forceinline__ void sum_parts(float2 (&v)[K], int part) {
    constexpr int PAIRS = 32 / SPLIT;
#pragma unroll
    for (int j = 0; j < K / SPLIT; ++j) {
        float2 t[SPLIT];
#pragma unroll
        for (int u = 0; u < SPLIT; ++u) t[u] = v[j * SPLIT + u];
#pragma unroll
        for (int n = SPLIT / 2; n > 0; n /= 2)
#pragma unroll
            for (int u = 0; u < n; ++u) {
                const float2 keep = part & n ? t[u + n] : t[u], give = part & n ? t[u] : t[u + n];
                t[u] = add2(keep, make_float2(__shfl_xor_sync(0xffffffffu, give.x, n * PAIRS), __shfl_xor_sync(0xffffffffu, give.y, n * PAIRS)));
            }
        v[j] = t[0];
    }
}

// Whether every row of x, dt and z (and with them y and the gradients, which are
// contiguous) divides into aligned pieces of so many bytes from each group's start on.
inline bool rows_in(const SelCall &c, size_t bytes) {
    const size_t e = c.bf16 ? 2 : 4;
    return c.channels / c.groups * e % bytes == 0 && rows_aligned(c.x, c.ld_x, e, bytes) && rows_aligned(c.dt, c.ld_dt, e, bytes) &&
           (!c.z || rows_aligned(c.z, c.ld_z, e, bytes));
}
struct Access {
    bool wide, paired, state, bc;  // 16-byte pieces of rows, pairs of channels, pairs of float32, quads of B and C
    explicit Access(const SelCall &c) {
        const size_t e = c.bf16 ? 2 : 4;
        wide = rows_in(c, 16), paired = rows_in(c, 2 * e), state = c.channels / c.groups % 2 == 0;
        bc = c.dstate % 4 == 0 && rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
    }
};
// The states that segments start from, in place of the ones they end with from zero:
// forwards h_{j+1} = exp(A steps_j) h_j + S_j from the sequence's initial state,
// backwards the same from the last segment, from zero.
cudaError_t launch_sel_join(const SelCall &c, const Segments &s, bool backwards, cudaStream_t st);

// Calls f with dstate padded to 4, 8, 16, 32 or 64 (padding states stay zero).
template <typename F> cudaError_t with_states(int N, F &&f) {
    if (N <= 4) return f(std::integral_constant<int, 4>{});
    if (N <= 8) return f(std::integral_constant<int, 8>{});
    if (N <= 16) return f(std::integral_constant<int, 16>{});
    if (N <= 32) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 64>{});
}

}  // namespace ssd
