// loss_tile.h -- a tile of logits in a wave's registers reduced to its rows' softmax statistics, or turned into the
// loss's gradient, without passing through memory.
//
// The wave holds FM x FN blocks of T rows x T columns: lane l has row l % T of
// each, and of its columns those that column_of() says.
#pragma once

#include "linear_common.h"

namespace miconv {

// Column in a block of value e of lane l.
template <int T> __device__ __forceinline__ int column_of(int e, int lane)
{
    return T == 32 ? 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3) : 4 * (lane >> 4) + e;
}

template <class In, class Block, int FM, int FN>
__device__ __forceinline__ void add_bias(const ProductArgs& p, Block (&acc)[FM][FN], int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4;
    if (!p.bias) return;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int n = j0 + T * j + column_of<T>(e, lane);
            const float b = n < p.N ? to_f32(static_cast<const In*>(p.bias)[n]) : 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[i][j][e] += b;
        }
}

// Each row's largest logit of these columns and the sum of e^(z - largest), [run][row]: run = the wave's columns; with
// smoothing the sum of z; the target's logit where it is among them.
template <bool EXACT, class Block, int FM, int FN>
__device__ __forceinline__ void loss_wave(const LossProductArgs& p, Block (&acc)[FM][FN], int m0, int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4, W = T * FN;
    using In = typename std::conditional<EXACT, float, Bf16>::type;
    if (j0 >= p.N) return;
    add_bias<In>(p, acc, j0, lane);
    const bool cut = j0 + W > p.N;
    const float least = -__builtin_inff();
    const int64_t run = p.loss.part_first + j0 / W;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + T * i + lane % T;
        if (m0 + T * i >= p.M) break;
        const int at = m < p.M ? loss_column(p.loss, p.loss.target[m]) : -1;
        if (at >= j0 && at < j0 + W) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (j0 + T * j + column_of<T>(e, lane) == at) p.loss.hit[m] = acc[i][j][e];
        }
        float sum_z = 0.0f;
        if (p.loss.part_z) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) sum_z += acc[i][j][e];         // columns past N are zeros
#pragma unroll
            for (int o = T; o < 64; o <<= 1) sum_z += __shfl_xor(sum_z, o);
        }
        if (cut) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (j0 + T * j + column_of<T>(e, lane) >= p.N) acc[i][j][e] = least;
        }
        float most = least;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) most = fmaxf(most, acc[i][j][e]);  // a NaN stays in the sum
#pragma unroll
        for (int o = T; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o));
        // a row with no class left here has largest -infinity: its terms are e^-infinity, not e^(-infinity + infinity)
        const float from = most == least ? 0.0f : most;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) sum += exponential<EXACT>(acc[i][j][e] - from);
#pragma unroll
        for (int o = T; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
        if (lane < T && m < p.M) {
            const int64_t to = run * p.M + m;
            reinterpret_cast<float2*>(p.loss.part)[to] = float2{most, sum};
            if (p.loss.part_z) p.loss.part_z[to] = sum_z;
        }
    }
}

// The logits' gradient in their place, zeros past N; and of each column the sum over the wave's rows, [rows of a wave][column].
template <bool EXACT, class Block, int FM, int FN>
__device__ __forceinline__ void gradient_wave(const LossProductArgs& p, Block (&acc)[FM][FN], int m0, int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4, W = T * FN;
    using In = typename std::conditional<EXACT, float, Bf16>::type;
    add_bias<In>(p, acc, j0, lane);
    const float every = p.loss.smooth / (float)p.loss.classes, goal = 1.0f - p.loss.smooth + every;
    const bool cut = j0 + W > p.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        LossRow r = loss_row(p.loss, min(m0 + T * i + lane % T, p.M - 1));
        r.counts = r.counts && m0 + T * i + lane % T < p.M;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int n = j0 + T * j + column_of<T>(e, lane);
                const float v = loss_gradient<EXACT>(r, acc[i][j][e], n, goal, every);
                acc[i][j][e] = cut && n >= p.N ? 0.0f : v;
            }
    }
    if (!p.sums || m0 >= p.M) return;
    float* sums = p.sums + (int64_t)(m0 / (T * FM)) * p.N;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) s += acc[i][j][e];
#pragma unroll
            for (int o = 1; o < T; o <<= 1) s += __shfl_xor(s, o);
            const int n = j0 + T * j + column_of<T>(e, lane);
            if (lane % T == 0 && n < p.N) sums[n] = s;
        }
}

}  // namespace miconv
