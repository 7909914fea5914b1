// mixer.cuh -- arguments and helpers of the mixer-block operators: the short
// causal convolution and the selective scan on packed sequences and on single
// tokens (with their gradients), and the norms before and after a block.
//
// Packed sequences: the tokens of all sequences of a call lie one after another;
// sequence i holds rows cu[i] .. cu[i+1]-1 (device memory).  cu and the slot
// numbers are only known on the device, so the kernels check them there: a
// sequence whose bounds or slot are out of range is skipped and the device error
// word says so (ssd_get_device_status).
#pragma once

#include "ssd_internal.cuh"

namespace ssd {

struct Packed {
    const int *cu;                  // [nseq + 1]
    int nseq, tokens;               // tokens: rows of the packed tensors
    const int *slots;               // [nseq] or NULL: sequence i uses slot i
    int nslots;                     // slots of the state cache (0: no cache)
    const unsigned char *has_init;  // [nseq] or NULL: every sequence starts from zero
    int *dev_error;
};

__device__ __forceinline__ void raise_bad_index(int *dev_error) { atomicCAS(dev_error, DEV_OK, DEV_BAD_INDEX); }

// Sequence i's rows; false (and flagged) when they do not lie in the tensor.
__device__ __forceinline__ bool seq_rows(const Packed &p, int i, int &lo, int &hi) {
    lo = p.cu[i], hi = p.cu[i + 1];
    if (lo < 0 || hi < lo || hi > p.tokens) {
        raise_bad_index(p.dev_error);
        return false;
    }
    return true;
}

// Slot of sequence (or batch row) i: -1 for a padded entry (a negative number in
// `slots`), -2 for one out of range or already named by an earlier sequence of
// the call (flagged: two sequences cannot share a state, the first one has it).
// Called by a whole warp, so that the look at the earlier entries is 32 wide.
__device__ __forceinline__ int slot_of(const int *slots, int nslots, int i, int *dev_error) {
    const int s = slots ? slots[i] : i;
    if (s < 0) return -1;
    bool bad = s >= nslots;
    if (slots) {
        const int lane = threadIdx.x & 31;
        bool same = false;
        for (int j = lane; j < i; j += 32) same |= slots[j] == s;
        bad |= __any_sync(0xffffffffu, same) != 0;
    }
    if (bad) {
        raise_bad_index(dev_error);
        return -2;
    }
    return s;
}

// ------------------------------------------------------------- scalar functions
__device__ __forceinline__ float ex2a(float v) {  // 2^v, relative error about 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float LOG2E = 1.4426950408889634f;
// A in powers of two, and finite: a step of nothing (a token past the end) is a decay of
// one then, and any other of zero, also where A is -infinity.
__device__ __forceinline__ float rate(float A) { return fabsf(A) <= 1e38f ? A * LOG2E : A < 0.f ? -3e38f : A; }

__device__ __forceinline__ float rcpa(float v) {  // 1/v, 1 ulp; subnormal results are zero
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + e^-v): past v = -88 the exponential is infinite and the result zero
// (its value there is below 1e-38).
__device__ __forceinline__ float sigmoid_f(float v) { return rcpa(1.f + ex2a(-LOG2E * v)); }
__device__ __forceinline__ float silu_v(float v) { return v * sigmoid_f(v); }
// ln(1 + e^v) = max(v, 0) + ln(1 + t), t = e^-|v|: no overflow, and small steps (v
// far below zero) keep their relative precision.  ln(1 + t) = 2 artanh(s) with
// s = t / (2 + t) <= 1/3, by artanh's series: seven terms leave 1.4e-8.
__device__ __forceinline__ float softplus_f(float v) {
    const float t = ex2a(-LOG2E * fabsf(v)), s = t * rcpa(2.f + t), q = s * s;
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(q, p, 1.f / 9.f);
    p = fmaf(q, p, 1.f / 7.f);
    p = fmaf(q, p, 1.f / 5.f);
    p = fmaf(q, p, 1.f / 3.f);
    p = fmaf(q, p, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// ------------------------------------------------------------- packed pairs
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// 2^x for |x| <= SMALL_EXP by its Taylor polynomial (the first term left out is below
// 8e-9): decays near one come out to within an ulp, where the approximate exponential is
// off by up to about 2^-22, mostly to the same side.
constexpr float SMALL_EXP = 1.f;
__device__ __forceinline__ float2 ex2_small(float2 x) {
    float2 p = fma2(x, splat(1.0178086009e-7f), splat(1.3215486790e-6f));  // ln2^9 / 9!, ln2^8 / 8!
    p = fma2(x, p, splat(1.5252733804e-5f));
    p = fma2(x, p, splat(1.5403530393e-4f));
    p = fma2(x, p, splat(1.3333558146e-3f));
    p = fma2(x, p, splat(9.6181291076e-3f));
    p = fma2(x, p, splat(5.5504108665e-2f));
    p = fma2(x, p, splat(2.4022650696e-1f));
    p = fma2(x, p, splat(6.9314718056e-1f));
    return fma2(x, p, splat(1.f));
}
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 e = mul2(v, splat(-LOG2E)), d = add2(make_float2(ex2a(e.x), ex2a(e.y)), splat(1.f));
    return mul2(v, make_float2(rcpa(d.x), rcpa(d.y)));
}

__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 e = mul2(v, splat(-LOG2E)), d = add2(make_float2(ex2a(e.x), ex2a(e.y)), splat(1.f));
    return make_float2(rcpa(d.x), rcpa(d.y));
}
__device__ __forceinline__ float2 softplus2(float2 v) {  // softplus_f of each
    const float2 e = mul2(make_float2(fabsf(v.x), fabsf(v.y)), splat(-LOG2E));
    const float2 t = make_float2(ex2a(e.x), ex2a(e.y)), d = add2(t, splat(2.f));
    const float2 s = mul2(t, make_float2(rcpa(d.x), rcpa(d.y))), q = mul2(s, s);
    float2 p = fma2(q, splat(1.f / 13.f), splat(1.f / 11.f));
    p = fma2(q, p, splat(1.f / 9.f));
    p = fma2(q, p, splat(1.f / 7.f));
    p = fma2(q, p, splat(1.f / 5.f));
    p = fma2(q, p, splat(1.f / 3.f));
    p = fma2(q, p, splat(1.f));
    return fma2(add2(s, s), p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// V consecutive elements <-> floats, one access of V * sizeof(T) bytes where WIDE
// (the caller has checked the alignment), else V accesses.
template <typename T, int V, bool WIDE> __device__ __forceinline__ void load_v(const T *p, float (&v)[V]) {
    if constexpr (WIDE && sizeof(T) == 2 && V == 8) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else if constexpr (WIDE && sizeof(T) == 2 && V == 4) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else if constexpr (WIDE && sizeof(T) == 2 && V == 2) {
        const uint32_t q = *reinterpret_cast<const uint32_t *>(p);
        v[0] = __uint_as_float(q << 16), v[1] = __uint_as_float(q & 0xffff0000u);
    } else if constexpr (WIDE && sizeof(T) == 4 && V == 2) {
        const float2 q = *reinterpret_cast<const float2 *>(p);
        v[0] = q.x, v[1] = q.y;
    } else if constexpr (WIDE && sizeof(T) == 4 && V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = ld_f32<T>(p + i);
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 q = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&q);
}
template <typename T, int V, bool WIDE> __device__ __forceinline__ void store_v(T *p, const float (&v)[V]) {
    if constexpr (WIDE && sizeof(T) == 2 && V == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else if constexpr (WIDE && sizeof(T) == 2 && V == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else if constexpr (WIDE && sizeof(T) == 2 && V == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[1]);
    } else if constexpr (WIDE && sizeof(T) == 4 && V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    } else if constexpr (WIDE && sizeof(T) == 4 && V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) st_f32<T>(p + i, v[i]);
    }
}

// Whether a base and a row stride (in elements) keep every row aligned to `bytes`.
inline bool rows_aligned(const void *p, long long ld, size_t elem, size_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * elem % bytes == 0;
}

// ------------------------------------------------------------- calls
struct ConvCall {
    const void *in;  // [tokens, channels], row stride ld
    long long ld;
    const float *w, *bias;  // [channels, width], [channels] or NULL
    void *xo, *bo, *co;     // outputs (forward) or their gradients (backward)
    void *state;            // [nslots, channels, width - 1] or NULL
    void *dx;               // backward: [tokens, channels]
    float *dw, *db;         // backward
    bool bf16;
    int cx, cb, width, silu;
    Packed seq;
};
cudaError_t launch_conv_varlen(const ConvCall &c, cudaStream_t st);
cudaError_t launch_conv_update(const ConvCall &c, int batch, cudaStream_t st);
size_t conv_bwd_workspace(int tokens, int channels, int width);
cudaError_t launch_conv_bwd(const ConvCall &c, float *ws, cudaStream_t st);

struct SelCall {
    const void *x, *dt, *z, *B, *C;                 // [tokens, channels] (z or NULL), [tokens, groups, dstate]
    long long ld_x, ld_dt, ld_z, ld_b, ld_c;        // row strides
    const float *A, *D, *dt_bias;                   // [channels, dstate], [channels] or NULL
    float *state;                                   // [nslots, channels, dstate] or NULL
    float *chunk_states;                            // [tokens / SEL_CHUNK + nseq, dstate, channels] or NULL
    void *y;                                        // [tokens, channels]
    const void *dy;                                 // backward
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *dbias;
    bool bf16;
    int softplus, channels, groups, dstate;
    Packed seq;
};
constexpr int SEL_CHUNK = 8;  // tokens between kept states
constexpr int SEL_MAX_DSTATE = 64;  // states of a channel in registers
size_t sel_fwd_workspace(int tokens, int nseq, int channels, int dstate);
cudaError_t launch_sel_varlen(const SelCall &c, float *ws, cudaStream_t st);
cudaError_t launch_sel_update(const SelCall &c, int batch, cudaStream_t st);
size_t sel_bwd_workspace(int tokens, int nseq, int channels, int groups, int dstate);
cudaError_t launch_sel_bwd(const SelCall &c, void *ws, cudaStream_t st);

constexpr int NORM_MAX_WIDTH = 8192;  // channels of a normalised group (registers of 512 threads)
struct NormCall {
    const void *x, *z, *res;      // rows (z, res or NULL)
    long long ld_x, ld_z, ld_res;
    const float *w, *scale;       // [width], [width] or NULL
    void *out, *res_out;          // [rows, width]
    const void *dout, *dres;      // backward
    void *dx, *dz, *dres_out;
    float *dw, *dscale;
    bool bf16, res_bf16;
    int rows, width, groups, norm_first;
    float eps;
};
cudaError_t launch_norm_before(const NormCall &c, cudaStream_t st);
cudaError_t launch_norm_after(const NormCall &c, cudaStream_t st);
size_t norm_bwd_workspace(int rows, int width);
cudaError_t launch_norm_before_bwd(const NormCall &c, float *ws, cudaStream_t st);
cudaError_t launch_norm_after_bwd(const NormCall &c, float *ws, cudaStream_t st);

// The current device's error word of bounds and slots (set by kernels, read by
// ssd_get_device_status; a wait that gave up has a word of its own); NULL with ssd_last_error set when it cannot be had.
int *device_error_word();

}  // namespace ssd
