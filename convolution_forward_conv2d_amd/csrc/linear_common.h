// linear_common.h -- pieces shared by the feed-forward kernels (linear and
// gated layers, their gradients, the root-mean-square norm): element types,
// activations, guarded vector loads and stores, and the product's arguments.
#pragma once

#include <stdint.h>

#include <type_traits>

#include <hip/hip_runtime.h>

#include "mfma_common.h"
#include "kernels.h"

namespace miconv {

typedef int i32x8 __attribute__((ext_vector_type(8)));

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct Bf16 { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ Bf16 from_f32<Bf16>(float v)
{
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)v)};      // round to nearest even, NaN kept
}

// ------------------------------------------------------------------ guarded vectors of eight
//
// Eight consecutive elements, of which the first nv exist.  A whole vector is
// one or two 16-byte accesses at any element alignment (gfx950 splits an
// unaligned one itself); a row's ragged end goes element by element, so
// nothing past the row is read or written.

template <class T> __device__ __forceinline__ void load8(const T* p, int nv, float (&v)[8])
{
    if (nv >= 8) {
        T t[8];
        __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < nv ? to_f32(p[i]) : 0.0f;
    }
}

template <class T> __device__ __forceinline__ void store8(T* p, int nv, const float (&v)[8])
{
    if (nv >= 8) {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
        __builtin_memcpy(p, t, sizeof(t));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nv) p[i] = from_f32<T>(v[i]);
    }
}

// The 16-byte piece at p of which the first nv elements exist.
template <int E> __device__ __forceinline__ u32x4 load_piece(const uint8_t* p, int nv)
{
    u32x4 v = {0, 0, 0, 0};
    if (nv >= 16 / E) {
        __builtin_memcpy(&v, p, 16);
    } else if (nv > 0) {
#pragma unroll
        for (int i = 0; i < 16 / E; ++i)
            if (i < nv) {
                uint32_t x;
                if constexpr (E == 4) x = *reinterpret_cast<const uint32_t*>(p + 4 * i);
                else if constexpr (E == 2) x = *reinterpret_cast<const uint16_t*>(p + 2 * i);
                else x = p[i];
                v[i * E / 4] |= x << (8 * (i * E % 4));
            }
    }
    return v;
}

// ------------------------------------------------------------------ activations
//
// All in fp32.  e^x is 2^(x log2 e) on the hardware's exponential and 1/x its
// reciprocal, each within 1 ulp.  Rounding x log2 e to fp32 puts e^x off by up
// to |x| 2^-24 of itself more: that is below 2^-17 where bf16 outputs round to
// 2^-8, but not for fp32 ones (EXACT), which put what the rounding took back.
// e^x is then within 2^-22 of itself, SiLU within 2^-21, and the tanh GELU
// within 2^-21 (1 + |a|), a the logistic function's argument, which fp32 itself
// holds no better.  What is below 2^-126 becomes zero.
//
// A cross entropy's loss and lse are fp32 for bf16 tensors too, and their tiles' sums (loss_tile.h, loss_run8) still take
// the shorter form: an argument of size d puts its term off by 1.23 d 2^-24 (the rounding, and log2 e's own), and over up to
// 96 terms, the nearest of which is 1, the d weigh 2.6 at most ((n - 1) d e^-d / (1 + (n - 1) e^-d) is largest at d - 1 = (n
// - 1) e^-d, where it is d - 1), so that a sum is off by less than 2^-22 of itself, as the longer form's terms may be.  Sums
// of longer rows, in memory, and what joins runs take the longer one.  In the tiles it costs 29 us of 154 (4096 x 50021
// of 256 features; of 4096 33 of 1142).
//
// The normal distribution function of the exact GELU: fp32 tensors use erff,
// whose complement 1 + erf(x) is within 2^-24 (of 1, not of itself).  bf16 ones
// take its tail as the bell times a polynomial of 1 / (1 + 0.292 |z|), fitted
// for this: the polynomial is within 6.2e-8 of the tail in all and within 6.1e-5
// (2^-14) relative to it up to |z| = 14, where the bell ends, so outputs far
// below zero keep bf16's precision too, at a third of erff's instructions (the
// epilogue of an e4m3 product of depth 4096 would otherwise spend half as long
// in erff as in its matrix instructions).

template <bool EXACT> __device__ __forceinline__ float exponential(float x)
{
    const float e = __builtin_amdgcn_exp2f(x * 1.44269504f);
    if constexpr (!EXACT) return e;
    // past 128 e is 0 or infinite already, and the rest of the argument no small number
    const float c = fminf(fmaxf(x, -128.0f), 128.0f), p = c * 1.44269504f;
    const float rest = fmaf(c, 1.92596303e-8f, fmaf(c, 1.44269504f, -p));      // of x log2 e, past p
    return e * fmaf(rest, 0.693147181f, 1.0f);
}
template <bool EXACT> __device__ __forceinline__ float logistic(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + exponential<EXACT>(-x));
}

// Phi(-|z|), the normal distribution's tail, and its bell e^(-z^2/2).
__device__ __forceinline__ float normal_tail(float z, float& bell)
{
    bell = __builtin_amdgcn_exp2f(z * (z * -0.721347520444482f));
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.292f * fabsf(z));
    return t * (0.11744149f + t * (0.10390588f + t * (0.1709076f + t * (-0.076288655f + t * (0.27079475f + t * -0.086761124f))))) * bell;
}

// (Phi(z), e^(-z^2/2)): the normal distribution function and its bell.
template <bool EXACT> __device__ __forceinline__ void normal_cdf(float z, float& phi, float& bell)
{
    if constexpr (EXACT) {
        bell = exponential<EXACT>(-0.5f * z * z);
        phi = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
    } else {
        const float half = normal_tail(z, bell);
        phi = z >= 0.0f ? 1.0f - half : half;                  // a NaN is in half already
    }
}

template <bool EXACT> __device__ __forceinline__ float act_value(int act, float z)
{
    switch (act) {
    case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case ACT_GELU: {
        float phi, bell;
        if constexpr (EXACT) {
            normal_cdf<EXACT>(z, phi, bell);
            return z * phi;
        }
        // z Phi(z) = max(z, 0) - |z| tail(|z|); past 16 the tail is below 2^-180, and infinity times it no number
        const float tail = normal_tail(z, bell);
        return fmaxf(z, 0.0f) - fminf(fabsf(z), 16.0f) * tail;
    }
    case ACT_GELU_TANH:       // 0.5 z (1 + tanh(u)) = z * logistic(2 u)
        return z * logistic<EXACT>(1.59576912160573f * (z + 0.044715f * z * z * z));
    case ACT_SILU: return z * logistic<EXACT>(z);
    default: return z;
    }
}

// Value and derivative at z.
template <bool EXACT> __device__ __forceinline__ void act_both(int act, float z, float& value, float& slope)
{
    switch (act) {
    case ACT_RELU:
        value = z > 0.0f ? z : (z != z ? z : 0.0f);
        slope = z > 0.0f ? 1.0f : 0.0f;
        break;
    case ACT_GELU: {
        float phi, bell;
        normal_cdf<EXACT>(z, phi, bell);
        value = z * phi;
        slope = phi + z * bell * 0.398942280401433f;
        break;
    }
    case ACT_GELU_TANH: {
        const float p = logistic<EXACT>(1.59576912160573f * (z + 0.044715f * z * z * z));
        value = z * p;
        // past 64 p is 0 or 1 to the last bit, and z^2 may overflow
        const float c = fminf(fmaxf(z, -64.0f), 64.0f);
        slope = p + c * p * (1.0f - p) * 1.59576912160573f * (1.0f + 0.134145f * c * c);
        break;
    }
    case ACT_SILU: {
        const float p = logistic<EXACT>(z);
        value = z * p;
        slope = p + value * (1.0f - p);
        break;
    }
    default: value = z; slope = 1.0f;
    }
}

// ------------------------------------------------------------------ the product's arguments
//
// raw[i, j] = sum_k A(i, k) B(j, k), rows i < M, and an epilogue.  Each
// operand is stored along k ("k-major": element (r, k) at r * ld + k) or
// across it (element (r, k) at k * ld + r).  All pitches in bytes.
struct ProductArgs {
    const uint8_t* a;
    const uint8_t* b;
    const uint8_t* b2;        // gated forward: the second weights; two k segments: the second segment's B
    int64_t lda, ldb, ldb2;
    int M;                    // rows of A
    int N;                    // output columns
    int K;                    // reduction length of one segment
    // linear_fast.h reads whole 16-byte pieces: the lengths its operands are padded to, zeros past the real ones
    int a_K;                  // columns of k-major operands, >= K
    int a_rows, b_rows;       // columns of operands stored across k, >= M and >= N
    int k_segments;           // 1, or 2: A's columns [k_pitch, k_pitch + K) meet b2
    int k_pitch;
    int m_pitch;              // rows at or past m_pitch are rows of the second output y2 (EPI_PLAIN)
    int m_valid;              // rows of each output
    // epilogue
    int act;
    void* y;
    void* y2;
    int64_t ldy, ldy2;        // elements, as every pitch below
    const void* bias;
    const void* residual;
    int64_t ldr;
    const float* x_scale;
    const float* w_scale;
    const float* w2_scale;
    void* pre;                // the product before the activation (gated: gate), or null
    void* pre2;               // gated: up
    int64_t ldp, ldp2;
    // reduction split over blockIdx.z: partial sums, fp32, [split][M][part_ld]
    int splits;
    float* part;
    int64_t part_ld;
};

// A product of a loss's kinds.
struct LossProductArgs : ProductArgs {
    LossArgs loss;
    int y_columns;            // EPI_LOGITS_GRAD: y is dz, whose columns up to y_columns are written, zeros past N
    float* sums;              // its column sums over each wave's rows, or null
    // EPI_SUM: one of several products of dz that add up to y.  Their sum so far, fp32, rows of ld_sum: the first writes it, the
    // last adds to it and writes y instead
    float* sum;
    int64_t ld_sum;
    bool sum_first, sum_last;
    int cus;                  // the device's compute units (linear_chain.h)
};

enum Epilogue : int { EPI_PLAIN = 0, EPI_LINEAR = 1, EPI_GATED = 2, EPI_LOSS = 3, EPI_LOGITS_GRAD = 4, EPI_SUM = 5, EPI_STORE = 6 };
template <int EPI> using ArgsOf = std::conditional_t<(EPI >= EPI_LOSS), LossProductArgs, ProductArgs>;

// A gated layer's raw columns come in blocks of 32, 16 of the gate's and the
// same 16 of the other product's, so both meet in one workgroup (and one wave)
// whatever its tile.
__host__ __device__ inline int gated_raw_columns(int n) { return (n + 15) / 16 * 32; }

// Eight values; the branch is outside the loop: eight independent chains inside.
template <bool EXACT> __device__ __forceinline__ void activate8(int act, float (&v)[8])
{
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value<EXACT>(ACT_RELU, v[i]);
        break;
    case ACT_GELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value<EXACT>(ACT_GELU, v[i]);
        break;
    case ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value<EXACT>(ACT_GELU_TANH, v[i]);
        break;
    case ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value<EXACT>(ACT_SILU, v[i]);
        break;
    default: break;
    }
}

// A scale s = part * 2^power.  The product of a row's and a column's scale can leave fp32's normal range where the sum
// times both does not, so the parts (in [1/2, 1)) are multiplied first and the powers applied last, with one rounding
// more only where the result is subnormal; anywhere else the bits are those of sum * (x_scale * w_scale).
struct Scale {
    float part;
    int power;
};
__device__ __forceinline__ Scale split_scale(float s)
{
    return Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
__device__ __forceinline__ float scaled(float v, Scale a, Scale b)
{
    return __builtin_ldexpf(v * (a.part * b.part), a.power + b.power);
}

// ------------------------------------------------------------------ cross entropy
//
// z the logits of a row, t its target, a the smoothing's share:
//   lse = log sum_j e^z_j      loss = lse - (1 - a) z_t - a mean(z)
//   dz_j = gain (e^(z_j - lse) - (1 - a) [j = t] - a / classes),  gain = dloss / count
// A row without a target (loss.ignore) has neither loss nor gradient, whatever its logits; a target that is no class
// makes both no number; a row of which a bias of -infinity leaves no class has no gradient.
struct LossRow {
    float lse, gain;
    int at;                   // the target's column in this product, outside it if it is not there; NO_GRADIENT
};
constexpr int NO_GRADIENT = INT32_MIN;
__device__ __forceinline__ int loss_column(const LossArgs& p, int64_t target)
{
    return target >= 0 && target < p.classes ? (int)target - p.first : -1;
}
// dz is rounded to the tensors' type for the matrix instructions of its products, half a step of each of its values.  It is
// held in units of what it is where a row's target has no share yet, (1 - a + a / classes) dloss / count, and what is made
// of it multiplied by that: -1 takes no rounding in bf16, where a unit of 1 rounds the largest term of every row the same
// way, by as much as 2^-8 (dx and dw of 4096 x 50021 random logits were 3.0e-3 off in all, and are 1.7e-3 now, their own
// rounding).  A target with a probability p has -1 + p, which is rounded again: dx and dw are 2.2e-3 off for p spread over 0
// to 0.4 or 0 to 1, 3.3e-3 if every row's is the same 0.5, 2.2e-3 at 0.9; rows with a dloss each have that in dz, 2.3 to
// 2.5e-3 whatever p is.  (dz in 32 bits would leave 1.66e-3, the outputs' rounding.)  fp32 needs no unit.
template <bool EXACT> __device__ __forceinline__ float loss_unit(const LossArgs& p)
{
    if constexpr (EXACT) return 1.0f;
    float unit = 1.0f - p.smooth + p.smooth / (float)p.classes;
    if (!p.dloss_rows) unit *= *p.dloss;
    if (p.count) unit /= *p.count;
    return fabsf(unit) >= 0x1p-126f && fabsf(unit) < __builtin_inff() ? unit : 1.0f;
}
__device__ __forceinline__ LossRow loss_row(const LossArgs& p, int m, float unit)
{
    const int64_t target = p.target[m];
    LossRow r;
    r.lse = p.lse[m];
    r.gain = p.dloss[p.dloss_rows ? m : 0];
    if (p.count) r.gain = *p.count > 0.0f ? r.gain / *p.count : 0.0f;
    r.gain /= unit;
    if (target < 0 || target >= p.classes) r.gain = __builtin_nanf("");
    r.at = target == p.ignore || r.lse == -__builtin_inff() ? NO_GRADIENT : loss_column(p, target);
    return r;
}
template <bool EXACT> __device__ __forceinline__ float loss_gradient(const LossRow& r, float z, bool hit, float goal, float every)
{
    const float v = (exponential<EXACT>(z - r.lse) - (hit ? goal : every)) * r.gain;
    return r.at != NO_GRADIENT ? v : 0.0f;
}

// Statistics of eight logits n..n+7 of row m, as loss_tile.h's of a tile's columns.
template <bool EXACT> __device__ __forceinline__ void loss_run8(const LossProductArgs& p, int m, int n, float (&z)[8])
{
    using In = std::conditional_t<EXACT, float, Bf16>;
    const int nv = p.N - n, at = loss_column(p.loss, p.loss.target[m]);
    float bias[8] = {};
    if (p.bias) load8(static_cast<const In*>(p.bias) + n, nv, bias);
    float most = -__builtin_inff(), sum = 0.0f, total = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z[i] += bias[i];
        if (i < nv) most = fmaxf(most, z[i]), total += z[i];
        if (n + i == at) p.loss.hit[m] = z[i];
    }
    const float from = most == -__builtin_inff() ? 0.0f : most;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += i < nv ? exponential<EXACT>(z[i] - from) : 0.0f;
    const int64_t to = (int64_t)(p.loss.part_first + n / 8) * p.M + m;
    reinterpret_cast<float2*>(p.loss.part)[to] = float2{most, sum};
    if (p.loss.part_z) p.loss.part_z[to] = total;
}

// Eight finished columns n..n+7 of row m: v the raw sums (u the second product's).
template <class Out, int EPI>
__device__ __forceinline__ void finish8(const ArgsOf<EPI>& p, int m, int n, float (&v)[8], float (&u)[8])
{
    constexpr bool EXACT = sizeof(Out) == 4;
    if constexpr (EPI == EPI_PLAIN) {
        const bool second = m >= p.m_pitch;
        const int r = second ? m - p.m_pitch : m;
        if (r >= p.m_valid || n >= p.N) return;
        Out* y = second ? static_cast<Out*>(p.y2) + (int64_t)r * p.ldy2 : static_cast<Out*>(p.y) + (int64_t)r * p.ldy;
        store8(y + n, p.N - n, v);
        return;
    }
    if constexpr (EPI == EPI_LOSS) {
        // few rows: eight columns are a run
        if (m < p.M && n < p.N) loss_run8<EXACT>(p, m, n, v);
        return;
    }
    if constexpr (EPI == EPI_SUM) {
        if (m >= p.M || n >= p.N) return;
        if (!p.sum_first) {
            load8(p.sum + (int64_t)m * p.ld_sum + n, p.N - n, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
        if (!p.sum_last) {
            store8(p.sum + (int64_t)m * p.ld_sum + n, p.N - n, v);
            return;
        }
        const float unit = loss_unit<EXACT>(p.loss);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= unit;
        store8(static_cast<Out*>(p.y) + (int64_t)m * p.ldy + n, p.N - n, v);
        return;
    }
    if (m >= p.M || n >= p.N) return;
    const int nv = p.N - n;
    if (p.x_scale) {
        const Scale xs = split_scale(p.x_scale[m]);
        float ws[8];
        load8(p.w_scale + n, nv, ws);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = scaled(v[i], xs, split_scale(ws[i]));
        if constexpr (EPI == EPI_GATED) {
            load8(p.w2_scale + n, nv, ws);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = scaled(u[i], xs, split_scale(ws[i]));
        }
    }
    if constexpr (EPI == EPI_LINEAR) {
        if (p.bias) {
            float b[8];
            load8(static_cast<const Out*>(p.bias) + n, nv, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
    }
    if (p.pre) store8(static_cast<Out*>(p.pre) + (int64_t)m * p.ldp + n, nv, v);
    if constexpr (EPI == EPI_GATED) {
        if (p.pre2) store8(static_cast<Out*>(p.pre2) + (int64_t)m * p.ldp2 + n, nv, u);
    }
    activate8<EXACT>(p.act, v);
    if constexpr (EPI == EPI_GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= u[i];
    } else if (p.residual) {
        float r[8];
        load8(static_cast<const Out*>(p.residual) + (int64_t)m * p.ldr + n, nv, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8(static_cast<Out*>(p.y) + (int64_t)m * p.ldy + n, nv, v);
}

// ------------------------------------------------------------------ matrix instructions
//
// A step of the reduction is 128 bytes of every row, in two halves of 64.  For
// 32 rows and one half, lane l holds two 16-byte vectors f[0], f[1] of row
// l % 32: the bytes 32 t + 16 (l / 32) of the half.  One mfma() consumes both
// for a 32 x 32 block: v_mfma_f32_32x32x16_bf16 twice, 32x32x2_f32 eight times
// or 32x32x64 in e4m3 once (32x32x16_bf16 four times).  Each instruction pairs lane groups of the two
// operands by position, so the order in which it walks k does not matter as
// long as both operands share it.  `rows` gives D's rows and `cols` its columns:
// value i of lane l is D[8 (i/4) + 4 (l/32) + i%4][l % 32].

struct MulBf16 {
    static constexpr int E = 2;                                // bytes per element
    using Out = Bf16;
    __device__ static f32x16 mfma(const u32x4* rows, const u32x4* cols, f32x16 c)
    {
#pragma unroll
        for (int t = 0; t < 2; ++t)
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, rows[t]),
                                                        __builtin_bit_cast(bf16x8, cols[t]), c, 0, 0, 0);
        return c;
    }
    // for 16 rows and one half, lane l holds one vector: the bytes 16 (l / 16) of the half of row l % 16
    using Block = f32x4;
    static constexpr int T = 16;                               // large tiles' blocks: T x T
    __device__ static f32x4 block(const u32x4* rows, const u32x4* cols, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, rows[0]),
                                                       __builtin_bit_cast(bf16x8, cols[0]), c, 0, 0, 0);
    }
    // one vector a lane, of row l % 16, for 16 x 16 (the lane groups and a vector's elements walk k in one order)
    __device__ static f32x4 mac16(u32x4 rows, u32x4 cols, f32x4 c) { return block(&rows, &cols, c); }
};

// The same with outputs in fp32.
struct MulBf16F32 : MulBf16 {
    using Out = float;
};

struct MulF32 {
    static constexpr int E = 4;
    using Out = float;
    using Block = f32x16;
    static constexpr int T = 32;
    __device__ static f32x16 block(const u32x4* rows, const u32x4* cols, f32x16 c) { return mfma(rows, cols, c); }
    __device__ static f32x16 mfma(const u32x4* rows, const u32x4* cols, f32x16 c)
    {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(rows[t][e]), __uint_as_float(cols[t][e]), c,
                                                         0, 0, 0);
        return c;
    }
    __device__ static f32x4 mac16(u32x4 rows, u32x4 cols, f32x4 c)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(rows[e]), __uint_as_float(cols[e]), c, 0, 0, 0);
        return c;
    }
};

// e4m3 comes in two forms.  The e4m3 instructions (32x32x64 here, 32x32x16 the
// same) keep only about 13 bits of each product below the largest one they add:
// on uniformly drawn bit patterns a sum of 64 was off by up to 2^-11.6 of its
// largest term, whatever the accumulator.  The default therefore widens to bf16
// (exact) in registers and adds in fp32; SHORT takes the e4m3 instruction, for
// callers that ask for its rate.
template <class OutT, bool SHORT> struct MulE4m3 {
    static constexpr int E = 1;
    using Out = OutT;
    __device__ static bf16x8 widen(uint32_t lo, uint32_t hi)
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    using Block = f32x16;
    static constexpr int T = 32;
    __device__ static f32x16 block(const u32x4* rows, const u32x4* cols, f32x16 c) { return mfma(rows, cols, c); }
    __device__ static f32x16 mfma(const u32x4* rows, const u32x4* cols, f32x16 c)
    {
        if constexpr (SHORT) {
            const i32x8 a = {(int)rows[0][0], (int)rows[0][1], (int)rows[0][2], (int)rows[0][3],
                             (int)rows[1][0], (int)rows[1][1], (int)rows[1][2], (int)rows[1][3]};
            const i32x8 b = {(int)cols[0][0], (int)cols[0][1], (int)cols[0][2], (int)cols[0][3],
                             (int)cols[1][0], (int)cols[1][1], (int)cols[1][2], (int)cols[1][3]};
            // formats 0, 0: e4m3; block scales 0 selects the unscaled instruction
            return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(rows[t][e], rows[t][e + 1]),
                                                            widen(cols[t][e], cols[t][e + 1]), c, 0, 0, 0);
        return c;
    }
    __device__ static f32x4 mac16(u32x4 rows, u32x4 cols, f32x4 c)
    {
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(rows[e], rows[e + 1]), widen(cols[e], cols[e + 1]), c,
                                                        0, 0, 0);
        return c;
    }
};

}  // namespace miconv
