// selscan_seg.cuh -- what the forward and backward selective scans share: the cut of
// sequences into segments, the staging of B and C, and the join of segments.
//
// A thread walks the recurrence of one channel, its states in registers two to a
// float2, so that every operation but the exponential is a packed one.  Where the
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

// The cut: none once there are `warps_per_sm` warps for each SM, else segments so
// short that there are, but of 64 tokens at least (a multiple of 16, so that kept
// states fall on segment starts).
inline int choose_seg(int tokens, int nseq, int channels, int warps_per_sm) {
    const long long want = 148LL * warps_per_sm, per_token = (channels + 31) / 32;
    if (nseq * per_token * 2 >= want) return WHOLE;
    const long long seg = (tokens * per_token / want + 15) / 16 * 16;
    return seg < 64 ? 64 : (int)seg;
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

// B and C of TT tokens in shared memory: token t, states 2 p and 2 p + 1 as
// (B, B, C, C), so that one 16-byte read, the same for all lanes, feeds a pair of
// states.  Fetched a run ahead: `load` takes the rows into registers as they lie in
// memory, `put` writes them out once the buffer is free.  Tokens past the run's end and
// states past N are zero.
template <typename T, int NP, int TT, int THREADS> struct StageBC {
    static constexpr int QUADS = TT * NP / 4, PER = (QUADS + THREADS - 1) / THREADS;  // of B, and of C
    static constexpr int BYTES = TT * NP * 8;
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
            const int at = u * THREADS + threadIdx.x, t = at / (NP / 4), s = at % (NP / 4) * 4;
            const int left = t < n && at < QUADS ? N - s : 0;
            b[u] = get(B + (left > 0 ? t * lb + s : 0), left, wide);
            c[u] = get(C + (left > 0 ? t * lc + s : 0), left, wide);
        }
    }
    __device__ __forceinline__ void put(float4 *to) const {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int at = u * THREADS + threadIdx.x;
            if (at >= QUADS) break;
            float fb[4], fc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fb[i] = ld_f32<T>(&b[u].v[i]), fc[i] = ld_f32<T>(&c[u].v[i]);
            to[2 * at] = make_float4(fb[0], fb[1], fc[0], fc[1]);
            to[2 * at + 1] = make_float4(fb[2], fb[3], fc[2], fc[3]);
        }
    }
};

// Channels of block `tile` of THREADS: first channel, group, and whether this thread has one.
struct Mine {
    int group, channel;
    bool in;
};
template <int THREADS> __device__ __forceinline__ Mine my_channel(const SelCall &c, int tile) {
    const int per_group = c.channels / c.groups, tiles = (per_group + THREADS - 1) / THREADS;
    const int g = tile / tiles, k = tile % tiles * THREADS + threadIdx.x;
    return {g, g * per_group + min(k, per_group - 1), k < per_group};
}
template <int THREADS> inline int channel_tiles(const SelCall &c) {
    return c.groups * ((c.channels / c.groups + THREADS - 1) / THREADS);
}

inline bool wide_bc(const SelCall &c) {
    const size_t e = c.bf16 ? 2 : 4;
    return c.dstate % 4 == 0 && rows_aligned(c.B, c.ld_b, e, 4 * e) && rows_aligned(c.C, c.ld_c, e, 4 * e);
}

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
