// selscan_tile.cuh -- what the forward and backward selective scans share: the
// split of a chunk over a warp, and the staging of its rows in shared memory.
//
// A warp holds 32 / TL channels; the TL lanes of a channel hold consecutive runs
// of `len` = 4, 8 or 16 tokens each (chosen per chunk so that short sequences waste
// little).  Token r of a chunk is item r % len of lane r / len.
// Within its run a lane walks the recurrence in registers; runs are joined by a
// scan over the lanes of (decay, state) pairs.  One exponential per state and
// token is all the recurrence needs, whatever the split.
#pragma once

#include "mixer.cuh"

namespace ssd {

constexpr int SEL_WARPS = 8;

__device__ __forceinline__ void cp16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A tile of SEG rows x CB channels of T: row r at r * CB * sizeof(T) plus 16 bytes
// per lane run before it, so that the lanes of a warp, which read rows a run
// apart, hit different banks.
template <typename T, int SEG, int CB, int TL> struct RowTile {
    static constexpr int BYTES = SEG * CB * (int)sizeof(T) + 16 * TL;
    static __device__ __forceinline__ T *row(unsigned char *base, int r, int run) {
        return reinterpret_cast<T *>(base + r * (CB * (int)sizeof(T)) + run * 16);
    }
    // Rows 0 .. n-1 of src (row stride ld, `cols` channels) into the tile.  wide:
    // every row start is 16-byte aligned and cols * sizeof(T) a multiple of 16.
    static __device__ __forceinline__ void fetch(unsigned char *base, const T *src, long long ld, int n, int cols, int len,
                                                 bool wide) {
        const int sh = 31 - __clz(len);
        if (wide) {
            constexpr int E = 16 / (int)sizeof(T), PER = CB / E;
            for (int u = threadIdx.x; u < n * PER; u += SEL_WARPS * 32) {
                const int r = u / PER, k = (u % PER) * E;
                if (k < cols) cp16(row(base, r, r >> sh) + k, src + r * ld + k);
            }
        } else {
            for (int u = threadIdx.x; u < n * CB; u += SEL_WARPS * 32) {
                const int r = u / CB, k = u % CB;
                if (k < cols) row(base, r, r >> sh)[k] = src[r * ld + k];
            }
        }
    }
    // The reverse, for results.
    static __device__ __forceinline__ void flush(unsigned char *base, T *dst, long long ld, int n, int cols, int len, bool wide) {
        const int sh = 31 - __clz(len);
        if (wide) {
            constexpr int E = 16 / (int)sizeof(T), PER = CB / E;
            for (int u = threadIdx.x; u < n * PER; u += SEL_WARPS * 32) {
                const int r = u / PER, k = (u % PER) * E;
                if (k < cols)
                    *reinterpret_cast<uint4 *>(dst + r * ld + k) = *reinterpret_cast<const uint4 *>(row(base, r, r >> sh) + k);
            }
        } else {
            for (int u = threadIdx.x; u < n * CB; u += SEL_WARPS * 32) {
                const int r = u / CB, k = u % CB;
                if (k < cols) dst[r * ld + k] = row(base, r, r >> sh)[k];
            }
        }
    }
};

// B and C of a chunk, per state n, in the order the lanes read them: quad q of
// lane run l (4 tokens) at (q * TL + l) * 4, so that a warp's 16-byte reads of one
// quad are consecutive.  bf16: B in the low and C in the high half of a word.
template <typename T, int SEG, int TL> struct BCTile {
    static constexpr bool PACK = sizeof(T) == 2;
    static constexpr int STATE_WORDS = PACK ? SEG : 2 * SEG;
    static __device__ __forceinline__ int at(int r, int len) {
        const int l = r >> (31 - __clz(len)), i = r - l * len;
        return ((i >> 2) * TL + l) * 4 + (i & 3);
    }
    static __device__ __forceinline__ void put(uint32_t *bc, int s, int o, float b, float c) {
        if constexpr (PACK) {
            bc[s * STATE_WORDS + o] = pack_bf16(b, c);  // exact: both came from bf16
        } else {
            bc[s * STATE_WORDS + o] = __float_as_uint(b);
            bc[s * STATE_WORDS + SEG + o] = __float_as_uint(c);
        }
    }
    // Rows of N states per token (n tokens, row strides lb and lc) into the tile;
    // the tokens up to TL * len read as zero.  wide: rows are aligned vectors of four.
    static __device__ __forceinline__ void fetch(uint32_t *bc, const T *B, long long lb, const T *C, long long lc, int n, int N,
                                                 int len, bool wide) {
        const int all = TL * len;
        if (wide) {
            const int per = N >> 2;
            for (int u = threadIdx.x; u < all * per; u += SEL_WARPS * 32) {
                const int r = u / per, s = (u - r * per) * 4, o = at(r, len);
                float b[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
                if (r < n) load_v<T, 4, true>(B + r * lb + s, b), load_v<T, 4, true>(C + r * lc + s, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) put(bc, s + i, o, b[i], c[i]);
            }
        } else {
            for (int u = threadIdx.x; u < all * N; u += SEL_WARPS * 32) {
                const int r = u / N, s = u - r * N;
                put(bc, s, at(r, len), r < n ? ld_f32<T>(B + r * lb + s) : 0.f, r < n ? ld_f32<T>(C + r * lc + s) : 0.f);
            }
        }
    }
    // B and C of quad q of lane run l for state s, as two pairs of tokens each.
    static __device__ __forceinline__ void quad(const uint32_t *bc, int s, int q, int l, float2 *b, float2 *c) {
        const uint32_t *p = bc + s * STATE_WORDS + (q * TL + l) * 4;
        if constexpr (PACK) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            b[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.y << 16));
            b[1] = make_float2(__uint_as_float(v.z << 16), __uint_as_float(v.w << 16));
            c[0] = make_float2(__uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y & 0xffff0000u));
            c[1] = make_float2(__uint_as_float(v.z & 0xffff0000u), __uint_as_float(v.w & 0xffff0000u));
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(p), u = *reinterpret_cast<const float4 *>(p + SEG);
            b[0] = make_float2(v.x, v.y), b[1] = make_float2(v.z, v.w);
            c[0] = make_float2(u.x, u.y), c[1] = make_float2(u.z, u.w);
        }
    }
};



}  // namespace ssd
