// loss_tile.h -- a tile of logits in a wave's registers reduced to its rows' softmax statistics, or turned into the
// loss's gradient, without passing through memory.
//
// The wave holds FM x FN blocks of T rows x T columns: lane l has row l % T of
// each; its value e of block j is column j0 + lane_column() + column_of(j, e).
// Rows are taken one after the other and compared by the distance from the
// lane's first column, against constants: masks of all columns at once, and all
// rows' values, would not fit the registers beside a tile's sums.
//
// The statistics add 4.4 us to a tile of 256 x 256: 57 us of 156 to 4096 x 50021 of
// 256 features, 46 of 1205 of 4096.  No one unit's time: without its exponentials
// a tile takes 1.2 us less, without the permutes that join lanes 0.6, without
// writing the runs 0.6, without the targets 0.4, without the largest's comparisons
// 0.15, without permutes, exponentials and comparisons together 2.2; the rest is
// the latency of one row block's chain after the other's.
#pragma once

#include "linear_common.h"

namespace miconv {

template <int T> __device__ __forceinline__ int lane_column(int lane) { return 4 * (lane / T); }
template <int T> __device__ constexpr int column_of(int j, int e) { return T * j + (T == 32 ? 8 * (e >> 2) + (e & 3) : e); }

template <class In, class Block, int FM, int FN>
__device__ __forceinline__ void add_bias(const ProductArgs& p, Block (&acc)[FM][FN], int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4;
    if (!p.bias) return;
    const int n0 = j0 + lane_column<T>(lane), left = p.N - n0;
    const In* bias = static_cast<const In*>(p.bias) + n0;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float b = column_of<T>(j, e) < left ? to_f32(bias[column_of<T>(j, e)]) : 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[i][j][e] += b;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Each row's largest logit of these columns and the sum of e^(z - largest), [run][row]: run = the wave's columns; with
// smoothing the sum of z; the target's logit where it is among them.
template <bool EXACT, class Block, int FM, int FN>
__device__ __forceinline__ void loss_wave(const LossProductArgs& p, Block (&acc)[FM][FN], int m0, int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4, W = T * FN;
    using In = typename std::conditional<EXACT, float, Bf16>::type;
    if (j0 >= p.N || m0 >= p.M) return;
    add_bias<In>(p, acc, j0, lane);
    const float least = -__builtin_inff();
    const int n0 = j0 + lane_column<T>(lane), left = p.N - n0;
    const int64_t run = (int64_t)(p.loss.part_first + j0 / W) * p.M;
    int at[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) at[i] = loss_column(p.loss, p.loss.target[min(m0 + T * i + lane % T, p.M - 1)]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + T * i + lane % T;
        if (at[i] >= j0 && at[i] < j0 + W && m < p.M) {
            const int here = at[i] - n0;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (here == column_of<T>(j, e)) p.loss.hit[m] = acc[i][j][e];
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
        if (j0 + W > p.N) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (column_of<T>(j, e) >= left) acc[i][j][e] = least;
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
            reinterpret_cast<float2*>(p.loss.part)[run + m] = float2{most, sum};
            if (p.loss.part_z) p.loss.part_z[run + m] = sum_z;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The logits' gradient in their place, zeros past N; and of each column the sum over the wave's rows, [rows of a wave][column].
template <bool EXACT, class Block, int FM, int FN>
__device__ __forceinline__ void gradient_wave(const LossProductArgs& p, Block (&acc)[FM][FN], int m0, int j0, int lane)
{
    constexpr int T = sizeof(Block) == sizeof(f32x16) ? 32 : 16, V = sizeof(Block) / 4, W = T * FN;
    using In = typename std::conditional<EXACT, float, Bf16>::type;
    if (m0 >= p.M) return;
    add_bias<In>(p, acc, j0, lane);
    const float every = p.loss.smooth / (float)p.loss.classes, goal = 1.0f - p.loss.smooth + every;
    const int n0 = j0 + lane_column<T>(lane), left = p.N - n0;
    const float unit = loss_unit<EXACT>(p.loss);
    LossRow rows[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + T * i + lane % T;
        rows[i] = loss_row(p.loss, min(m, p.M - 1), unit);
        if (m >= p.M) rows[i].at = NO_GRADIENT;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int here = (int)((uint32_t)rows[i].at - (uint32_t)n0);     // of NO_GRADIENT 2^30 at least: no column
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[i][j][e] = loss_gradient<EXACT>(rows[i], acc[i][j][e], here == column_of<T>(j, e), goal, every);
        if (j0 + W > p.N) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (column_of<T>(j, e) >= left) acc[i][j][e] = 0.0f;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!p.sums) return;
    float* sums = p.sums + (int64_t)(m0 / (T * FM)) * p.N + n0;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) s += acc[i][j][e];
#pragma unroll
            for (int o = 1; o < T; o <<= 1) s += __shfl_xor(s, o);
            if (lane % T == 0 && column_of<T>(j, e) < left) sums[column_of<T>(j, e)] = s * unit;
            __builtin_amdgcn_sched_barrier(0);
        }
}

}  // namespace miconv
